// The selective scan's recurrence over a sequence, as one kernel in four modes: with outputs,
// and, without them, the states that the segmented forward and the backward start from.
//
//   h_t[n] = exp(u_t A[n]) h_{t-1}[n] + u_t x_t B_t[n]  per channel,  y_t = sum_n C_t[n] h_t[n] + D x_t
//
// Each (token, channel, state) costs one exponential and six operations and no state leaves
// the chip, so on-chip throughput bounds it: instruction issue first, then the shared-memory
// pipe (operands into registers) and the exponentials.
//
// A thread holds 2 channels by 4 states in registers (arithmetic on packed pairs of states);
// LN lanes share a channel pair (4 LN = N rounded up).  Per token it reads 4 B, 4 C and two
// (u, u x): 48 bytes for 8 states.  One channel by 4 states reads 40 bytes for 4 and is bound by
// the shared-memory pipe; 2 by 8 reads less per state but needs as many instructions and halves
// the warps, which the recurrence needs to cover its latencies.  (bf16 B and C kept as they come
// halve the reads, but unpacking them at every use costs more: 557 -> 602 us, 32768 tokens.)
// A CTA of four warps takes CPB = 256 / LN channels of one sequence and walks its tokens in tiles
// staged in shared memory as fp32 (softplus once per token and channel) while the next ones are
// on their way: tiles of 16, and y goes back through shared memory, so rows are written as they
// are read.  The backward's checkpoints take tiles of 8 in two halves: between two barriers a warp
// stages the next tile and computes the one at hand, and warps drift apart in what they do.
// (With outputs that costs, for what is done once a tile then counts twice: 227 -> 246 us at
// 8 x 2048 x 2048 x 16 in bf16, when parts of y were still stored between the loads; 195 us now, with
// the shared-memory pipe at 71 % on the SMs that hold two of the 256 CTAs, 60 % on average.)
#pragma once

#include <type_traits>

#include "layer_common.cuh"

namespace qd {
namespace ssm {

constexpr int kScanThreads = 128;
constexpr int kTile = 16;             // tokens staged at a time
constexpr int kChunk = 8;             // tokens between the backward's checkpoints, which are staged at a time there

__host__ __device__ constexpr int padded_states(int N) { return N <= 8 ? 8 : N <= 16 ? 16 : N <= 32 ? 32 : N <= 64 ? 64 : 128; }

// Channel blocks never cross a group of channels that share B and C.
__host__ __device__ inline int channel_blocks(int D, int G, int CPB) { return G * ((D / G + CPB - 1) / CPB); }

struct ChannelBlock {
    int group, first, count;          // its group, its first channel and how many it has
    __device__ __forceinline__ ChannelBlock(const SsmArgs &a, int block, int CPB) {
        const int per = a.D / a.G, nb = (per + CPB - 1) / CPB;
        group = block / nb;
        const int at = (block % nb) * CPB;
        first = group * per + at;
        count = min(CPB, per - at);
    }
};

// Tokens cut into S segments of `len` (a multiple of `align`, the tile): one when `ctas` CTAs
// already number `enough`, else about `want` CTAs in all, of at least `least` tokens.  What a segment
// spends on joining those before it is not counted: at 512 segments (1 x 32768 tokens x 16 channels x 16 states,
// bf16) the forward takes 84 us and the backward 209, as long as with 128 channels and 293 segments (84, 199).
struct Split {
    int S, len;
};
inline Split split_tokens(int64_t ctas, int T, int64_t enough, int64_t want, int least, int align) {
    Split s{1, T > 0 ? T : 1};
    if (ctas <= 0 || ctas >= enough) return s;
    int64_t S = want / ctas, most = T / least;
    if (S > most) S = most;
    if (S < 2) return s;
    s.len = (int)(((T + S - 1) / S + align - 1) / align * align);
    s.S = (int)(((int64_t)T + s.len - 1) / s.len);     // T + len passes 2^31
    return s;
}

// More dynamic shared memory than a launch gets without asking.
template <typename K> cudaError_t allow_smem(K kernel, size_t bytes) {
    return bytes <= 48 * 1024 ? cudaSuccess
                              : cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

// Whether a lane of the warp holds a rate A above 0: its states grow, by more than fp32 holds over many tokens.
__device__ __forceinline__ bool rates_grow(const f32x2 (&A2)[2][2]) {
    bool up = false;
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            float lo, hi;
            unpk(A2[c][p], lo, hi);
            up = up || lo > 0.f || hi > 0.f;
        }
    return __any_sync(0xffffffffu, up);
}

__device__ __forceinline__ int seq_len(const int *lens, int b, int T) { return lens ? min(max(lens[b], 0), T) : T; }

// Where a token's channel pair p lies in a row of staged pairs: even and odd ones apart, so that a
// thread's two neighbouring pairs are written, and a warp's read, without bank conflicts.
__host__ __device__ constexpr int pair_at(int p, int PAIRS) { return p / 2 + (p & 1) * (PAIRS / 2 + 4); }
__host__ __device__ constexpr int pair_row(int PAIRS) { return PAIRS + 4; }

// u = softplus(delta + bias), or the sum, of VEC channels.
template <int VEC> __device__ __forceinline__ void step_sizes(float (&u)[VEC], const float (&bias)[VEC], int softplus) {
#pragma unroll
    for (int k = 0; k < VEC; ++k) u[k] += bias[k];
    if (softplus) {
        float e0, e1, none = 0.f;
        if constexpr (VEC == 1) softplus2(u[0], none, e0, e1);
        else
#pragma unroll
            for (int k = 0; k + 1 < VEC; k += 2) softplus2(u[k], u[k + 1], e0, e1);
    }
}

// A tile of TILE tokens on its way from global to shared memory: NA token arrays and B and C.  The raw
// tile arrives by asynchronous copies, some tiles ahead, in one of STAGES buffers; every thread
// then reads back what it copied itself (so its own wait is enough), converts it and stages it
// for the CTA.  An access is V neighbouring channels of a token, or V states of its B or C: 4, or for
// odd shapes 2 (bf16) or 1; single bf16 values are below what a copy can move and are read when they
// are staged.  What is beyond the sequence, the block's channels or N arrives as zero.
template <typename T, int THREADS, int TILE, int CPB, int NP, int NA, int V, int STAGES> struct Staging {
    static constexpr bool ASYNC = V * sizeof(T) >= 4;
    static constexpr int ROW = CPB / V;                                // accesses a token
    static constexpr int PER = (TILE * ROW + THREADS - 1) / THREADS;
    static constexpr bool EVEN = PER * THREADS == TILE * ROW;          // every thread has PER of them
    static constexpr int GROW = NP / V, GALL = 2 * TILE * GROW;        // accesses of B a token; of both in all
    static constexpr int GPER = (GALL + THREADS - 1) / THREADS;
    static_assert(THREADS % ROW == 0);                                 // a thread's channels are the same every time
    static constexpr int STAGE = ASYNC ? (NA * TILE * CPB + 2 * TILE * NP) : 0;    // elements of a raw tile
    static constexpr size_t BYTES = (size_t)STAGES * STAGE * sizeof(T);
    using Vec = Pack<T, V>;

    __device__ __forceinline__ static int tok(int i) { return (threadIdx.x + i * THREADS) / ROW; }
    __device__ __forceinline__ static int chan() { return threadIdx.x % ROW * V; }
    // B or C, token and first state of group access i
    struct Group {
        int e, which, t, k;
        __device__ __forceinline__ Group(int i) {
            e = threadIdx.x + i * THREADS;
            which = e / (TILE * GROW);
            t = e % (TILE * GROW) / GROW;
            k = e % GROW * V;
        }
    };

    // The parameter p (or 0) of the thread's channels.
    __device__ __forceinline__ static void param(const float *p, const ChannelBlock &cb, float (&f)[V]) {
        const int c = chan();
#pragma unroll
        for (int k = 0; k < V; ++k) f[k] = p && c + k < cb.count ? p[cb.first + c + k] : 0.f;
    }
    // Whether the whole tile at t0 is real: no padding, no channels beyond the block's.
    __device__ __forceinline__ static bool full(const ChannelBlock &cb, int t0, int n) { return t0 + TILE <= n && cb.count == CPB; }

    // A thread's place in the arrays, moved from tile to tile: addresses are worked out once.  (g is indexed
    // with B or C as the thread has it, so the compiler keeps the cursor in local memory: 56 or 64 bytes.)
    struct Cursor {
        const T *p[NA], *g[2], *own;                                   // tokens; the tile's B and C; this thread's if it has one access
        size_t rows;                                                   // from one token access of a tile to the next
        int group_row;
        __device__ __forceinline__ Cursor(const SsmArgs &a, const ChannelBlock &cb, int b, int t0, const void *const (&src)[NA]) {
            rows = (size_t)(THREADS / ROW) * a.D;
            group_row = a.G * a.N;
            const ptrdiff_t at = ((ptrdiff_t)b * a.T + t0 + tok(0)) * a.D + cb.first + chan();
#pragma unroll
            for (int j = 0; j < NA; ++j) p[j] = (const T *)src[j] + at;
            const ptrdiff_t ga = (((ptrdiff_t)b * a.T + t0) * a.G + cb.group) * a.N;
            g[0] = (const T *)a.Bm + ga;
            g[1] = (const T *)a.Cm + ga;
            const Group q(0);
            own = g[q.which ? 1 : 0] + (ptrdiff_t)q.t * group_row + q.k;
        }
        __device__ __forceinline__ void move(const SsmArgs &a, int tiles) {
#pragma unroll
            for (int j = 0; j < NA; ++j) p[j] += (ptrdiff_t)tiles * TILE * a.D;
            const ptrdiff_t by = (ptrdiff_t)tiles * TILE * group_row;
            g[0] += by;
            g[1] += by;
            own += by;
        }
        // where group access q of the cursor's tile lies
        __device__ __forceinline__ const T *group(const Group &q) const {
            return GPER == 1 ? own : g[q.which] + (ptrdiff_t)q.t * group_row + q.k;
        }
    };
    // Starts the copies of the cursor's tile, which is at t0, into buffer `buf` (one group of copies,
    // empty where `any` is false) and moves the cursor by `step` tiles.
    __device__ __forceinline__ static void issue(Cursor &at, T *raw, int buf, const SsmArgs &a, const ChannelBlock &cb, int t0, bool any,
                                                 int n, bool both, int step) {
        if constexpr (ASYNC) {
            T *to = raw + (size_t)buf * STAGE + threadIdx.x * V;
            if (any) {
                if (full(cb, t0, n)) {
#pragma unroll
                    for (int j = 0; j < NA; ++j) {
#pragma unroll
                        for (int i = 0; i < PER; ++i)
                            if (EVEN || tok(i) < TILE) copy_async<V * sizeof(T)>(to + j * TILE * CPB + i * THREADS * V, at.p[j] + i * at.rows);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < PER; ++i) {
                        if (tok(i) >= TILE) break;
                        const bool on = t0 + tok(i) < n && chan() < cb.count;
#pragma unroll
                        for (int j = 0; j < NA; ++j)
                            copy_async<V * sizeof(T)>(to + j * TILE * CPB + i * THREADS * V, on ? at.p[j] + i * at.rows : (const T *)a.x, on);
                    }
                }
#pragma unroll
                for (int i = 0; i < GPER; ++i) {
                    const Group q(i);
                    const bool on = t0 + q.t < n && q.k < a.N;
                    if (q.e < (both ? GALL : GALL / 2))
                        copy_async<V * sizeof(T)>(to + NA * TILE * CPB + i * THREADS * V, on ? at.group(q) : (const T *)a.Bm, on);
                }
                at.move(a, step);
            }
            copies_issued();
        }
    }
    // Access i of token array j (src) of the tile at t0, in buffer `buf`.
    __device__ __forceinline__ static void get(const T *raw, int buf, int j, int i, const SsmArgs &a, const ChannelBlock &cb, int b,
                                               int t0, int n, const void *src, float (&f)[V]) {
        Vec v;
        if constexpr (ASYNC) {
            v.load(raw + (size_t)buf * STAGE + j * TILE * CPB + (threadIdx.x + i * THREADS) * V);
        } else {
            const int t = tok(i), c = chan();
            v.zero();
            if (t0 + t < n && c < cb.count) v.load((const T *)src + ((size_t)b * a.T + t0 + t) * a.D + cb.first + c);
        }
        v.get(f);
    }
    // put(which, t, k, f) for the V states from k of B (0) or C (1) of token t that this thread has
    // copied (or reads now): for the CTA to lay B and C out in its own way.
    template <typename F>
    __device__ __forceinline__ static void get_groups(const T *raw, int buf, const SsmArgs &a, const ChannelBlock &cb, int b, int t0,
                                                      int n, bool both, F put) {
#pragma unroll
        for (int i = 0; i < GPER; ++i) {
            const Group q(i);
            if (q.e >= (both ? GALL : GALL / 2)) break;
            Vec v;
            float f[V];
            if constexpr (ASYNC) {
                v.load(raw + (size_t)buf * STAGE + NA * TILE * CPB + q.e * V);
            } else {
                v.zero();
                if (t0 + q.t < n && q.k < a.N)
                    v.load((const T *)(q.which ? a.Cm : a.Bm) + (((size_t)b * a.T + t0 + q.t) * a.G + cb.group) * a.N + q.k);
            }
            v.get(f);
            put(q.which, q.t, q.k, f);
        }
    }
};

enum ScanMode {
    kOutputs,           // y and the final state
    kEnds,              // the end and the sum of u of every segment but the last (segmented forward)
    kCheckpoints,       // the state entering every chunk (backward, one segment)
    kSegCheckpoints     // the same from a zero state per segment, and what joins segments (backward)
};

// Workspace arrays of the modes; states are [.., B, D, NP].
struct ScanWs {
    float *start;       // [1]: S0 or zero.  Read back by the outputs, so that S_final may be S0
    float *E, *U;       // [S]: a segment's end (from zero; segment 0 from S0) and its sum of u
    float *R;           // [S]: sum_t (prod_{s<=t} a_s) C_t dy_t over a segment
    float *chk, *ucum;  // [chunks]: the state entering a chunk, and u summed from the segment's start
};

// A sum over n is split over LN lanes.  Shuffles join it down to PARTS lanes, which leave their
// parts in shared memory for whoever writes the result: joining all of it by shuffles costs a
// tenth of the instructions more.
__host__ __device__ constexpr int sum_parts(int LN) { return LN < 4 ? LN : 4; }
// Row of the parts of y, free of bank conflicts.
__host__ __device__ constexpr int scan_row(int LN) { return 256 / LN + (LN == 2 ? 16 : LN <= 8 ? 8 : 4); }

// Tiles and shared memory of a mode.
template <typename T, int LN, int VEC, int MODE> struct ScanSize {
    static constexpr bool OUT = MODE == kOutputs, SEG = MODE == kSegCheckpoints;
    static constexpr int PAIRS = kScanThreads / LN, CPB = 2 * PAIRS, NP = 4 * LN;
    static constexpr bool DRIFT = SEG || MODE == kCheckpoints;
    static constexpr int TILE = DRIFT ? kChunk : kTile, HALVES = DRIFT ? 2 : 1;
    static constexpr int AHEAD = DRIFT ? 3 : sizeof(T) == 4 ? 1 : 2;   // tiles on their way (fp32: as many as leave room for four CTAs)
    static constexpr int STAGES = AHEAD + 1;
    using St = Staging<T, kScanThreads, TILE, CPB, NP, SEG ? 3 : 2, VEC, STAGES>;
    static constexpr int SU = TILE * pair_row(PAIRS);                  // float4
    static constexpr int SG = TILE * NP * (OUT || SEG ? 2 : 1);        // floats, as below
    static constexpr int SY = OUT ? TILE * sum_parts(LN) * scan_row(LN) : SEG ? TILE * CPB : 0;
    static constexpr size_t BYTES = St::BYTES + HALVES * (SU * 4 + SG + SY) * sizeof(float);
};

template <typename T, int LN, int VEC, int MODE>
__global__ void __launch_bounds__(kScanThreads, 4) scan_kernel(SsmArgs a, Split sp, ScanWs w) {
    constexpr int PAIRS = kScanThreads / LN, CPB = 2 * PAIRS, NP = 4 * LN;
    constexpr bool OUT = MODE == kOutputs, SEG = MODE == kSegCheckpoints, CHK = SEG || MODE == kCheckpoints;
    constexpr bool BOTH = OUT || SEG;                                  // C is needed
    constexpr int PARTS = sum_parts(LN), NL = LN / PARTS, YS = scan_row(LN);
    using Z = ScanSize<T, LN, VEC, MODE>;
    using St = typename Z::St;
    constexpr int TILE = Z::TILE, AHEAD = Z::AHEAD, STAGES = Z::STAGES, PER = St::PER, SU = Z::SU, SG = Z::SG, SY = Z::SY;
    extern __shared__ float4 smem4[];
    T *raw = reinterpret_cast<T *>(smem4);                             // [STAGES] tiles on their way
    float4 *su = smem4 + St::BYTES / 16;                               // [HALVES][TILE][pair_row] (u0, u1, u0 x0, u1 x1)
    float *sB = reinterpret_cast<float *>(su + Z::HALVES * SU);        // [HALVES] B and (BOTH) C, [TILE][NP] each
    float *sy = sB + Z::HALVES * SG;                                   // [HALVES] OUT: parts of y, [TILE][PARTS][YS]; SEG: dy, [TILE][CPB]

    const int lane = threadIdx.x & 31, ln = threadIdx.x % LN, pr = threadIdx.x / LN, seg = blockIdx.y;
    const int nblk = channel_blocks(a.D, a.G, CPB), b = blockIdx.x / nblk;
    const ChannelBlock cb(a, blockIdx.x % nblk, CPB);
    const int D = a.D, N = a.N, c0 = 2 * pr;
    const int n = seq_len(a.lens, b, a.T);
    const int t_begin = seg * sp.len, t_stop = min(t_begin + sp.len, a.T), t_end = min(t_stop, n);
    const size_t bd = (size_t)b * D + cb.first + c0, all = (size_t)a.B * D;

    f32x2 A2[2][2], h[2][2], P[2][2], R[2][2];                         // A log2(e); pairs of states
    const bool from_S0 = a.S0 && seg == 0 && (MODE != kOutputs || sp.S == 1);
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            float av[2], hv[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int k = ln * 4 + 2 * p + j;
                const bool on = c0 + c < cb.count && k < N;
                av[j] = on ? a.A[(size_t)(cb.first + c0 + c) * N + k] * kLog2e : 0.f;
                hv[j] = on && from_S0 ? a.S0[(bd + c) * N + k] : 0.f;
            }
            A2[c][p] = pk(av[0], av[1]);
            h[c][p] = pk(hv[0], hv[1]);
            if (SEG) {
                P[c][p] = pk(1.f, 1.f);
                R[c][p] = 0;
            }
        }
    // four states of a channel as they lie in the workspace
    auto put_state = [&](float *base, size_t row, int c, const f32x2(&v)[2]) {
        if (c0 + c < cb.count) *reinterpret_cast<ulonglong2 *>(base + (row + c) * NP + ln * 4) = make_ulonglong2(v[0], v[1]);
    };
    if (MODE == kEnds && seg == 0) {
        put_state(w.start, bd, 0, h[0]);
        put_state(w.start, bd, 1, h[1]);
    }
    const bool up = (SEG || (OUT && sp.S > 1)) && rates_grow(A2);
    if (OUT && sp.S > 1) {                                             // fold the segments before this one
        auto fold = [&](auto careful) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                if (c0 + c >= cb.count) continue;
                for (int s = seg > 0 ? 0 : -1; s < max(seg, 0); ++s) {
                    const float *src = s < 0 ? w.start : w.E + s * all * NP;
                    const ulonglong2 e = *reinterpret_cast<const ulonglong2 *>(src + (bd + c) * NP + ln * 4);
                    const float U = s < 0 ? 0.f : w.U[s * all + bd + c];
                    const f32x2 UU = pk(U, U);
                    h[c][0] = carry2<careful.value>(UU, A2[c][0], h[c][0], e.x);
                    h[c][1] = carry2<careful.value>(UU, A2[c][1], h[c][1], e.y);
                }
            }
        };
        if (up || !a.softplus) fold(std::true_type{});
        else fold(std::false_type{});
    }

    float bias[VEC], skip[VEC];
    St::param(a.delta_bias, cb, bias);
    if (OUT) St::param(a.Dskip, cb, skip);
    auto cursor = [&] {
        if constexpr (SEG) return typename St::Cursor(a, cb, b, t_begin, {a.x, a.delta, a.dy});
        else return typename St::Cursor(a, cb, b, t_begin, {a.x, a.delta});
    };
    typename St::Cursor at = cursor();
    T *y = OUT ? (T *)a.y + ((size_t)b * a.T + t_begin + St::tok(0)) * D + cb.first + St::chan() : nullptr;
    f32x2 U = 0;                                                       // of the two channels
    bool back = false;                                                 // SEG: a step size below 0 has been staged

    auto issue = [&](int t0, int slot) { St::issue(at, raw, slot, a, cb, t0, t0 < t_end, n, BOTH, 1); };
    // the tile at t0, arrived in `slot`, to half `half` of the staging arrays
    auto stage = [&](int t0, int slot, int half) {
        const bool full = St::full(cb, t0, n);
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int t = St::tok(i), c = St::chan();
            if (!St::EVEN && t >= TILE) break;
            float u[VEC], x[VEC];
            St::get(raw, slot, 0, i, a, cb, b, t0, n, a.x, x);
            St::get(raw, slot, 1, i, a, cb, b, t0, n, a.delta, u);
            step_sizes<VEC>(u, bias, a.softplus);
            if (SEG && !a.softplus) {
#pragma unroll
                for (int k = 0; k < VEC; ++k) back = back || u[k] < 0.f;
            }
            if (!full && !(t0 + t < n && c < cb.count)) {              // of the padding nothing counts
#pragma unroll
                for (int k = 0; k < VEC; ++k) u[k] = 0.f;
            }
            float4 *row = su + half * SU + t * pair_row(PAIRS);
            if constexpr (VEC > 1) {
#pragma unroll
                for (int k = 0; k < VEC; k += 2)
                    row[pair_at((c + k) / 2, PAIRS)] = make_float4(u[k], u[k + 1], u[k] * x[k], u[k + 1] * x[k + 1]);
            } else {
                float *to = reinterpret_cast<float *>(row + pair_at(c / 2, PAIRS)) + (c & 1);
                to[0] = u[0];
                to[2] = u[0] * x[0];
            }
            if constexpr (SEG) {
                float g[VEC];
                St::get(raw, slot, 2, i, a, cb, b, t0, n, a.dy, g);
#pragma unroll
                for (int k = 0; k < VEC; ++k) sy[half * SY + t * CPB + c + k] = g[k];
            }
        }
        St::get_groups(raw, slot, a, cb, b, t0, n, BOTH, [&](int which, int t, int k, const float (&f)[VEC]) {
            Pack<float, VEC> v;
            v.set(f);
            v.store(sB + half * SG + (which * TILE + t) * NP + k);
        });
    };
    // the rows of y of the tile at t0 and the next place in y
    auto finish = [&](int t0, int slot, int half) {
        const bool full = St::full(cb, t0, n);
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int t = St::tok(i), c = St::chan();
            if (!full && (t0 + t >= t_stop || c >= cb.count)) continue;
            if (!St::EVEN && t >= TILE) continue;
            float f[VEC], x[VEC];
            St::get(raw, slot, 0, i, a, cb, b, t0, n, a.x, x);
#pragma unroll
            for (int q = 0; q < PARTS; ++q) {
                Pack<float, VEC> part;
                float g[VEC];
                part.load(sy + half * SY + (t * PARTS + q) * YS + c);
                part.get(g);
#pragma unroll
                for (int k = 0; k < VEC; ++k) f[k] = q ? f[k] + g[k] : g[k];
            }
            if (a.Dskip) {
#pragma unroll
                for (int k = 0; k < VEC; ++k) f[k] = fmaf(skip[k], x[k], f[k]);
            }
            if (!full && t0 + t >= n) {
#pragma unroll
                for (int k = 0; k < VEC; ++k) f[k] = 0.f;
            }
            typename St::Vec o;
            o.set(f);
            o.store(y + i * at.rows);
        }
        y += (size_t)TILE * D;
    };

    // the kChunk tokens from `from` on of the staged tile, the first of them token tc.  GROWS (SEG, from the
    // first tile on that has what may grow): R takes the products P from the sums of u.
    auto compute = [&](auto growing, int tc, int from, int half) {
        constexpr bool GROWS = growing.value;
        if (CHK) {                                                     // tc is a checkpoint of the segment
            const size_t row = (size_t)(tc / kChunk) * all + bd;
            put_state(w.chk, row, 0, h[0]);
            put_state(w.chk, row, 1, h[1]);
            if (SEG && ln == 0) {
                float u0, u1;
                unpk(U, u0, u1);
                if (c0 < cb.count) w.ucum[row] = u0;
                if (c0 + 1 < cb.count) w.ucum[row + 1] = u1;
            }
        }
        const float4 *mine = su + half * SU + from * pair_row(PAIRS) + pair_at(pr, PAIRS);
        const float *gB = sB + half * SG + from * NP + ln * 4, *gC = gB + TILE * NP;
        float *part = sy + half * SY + (from * PARTS + ln % PARTS) * YS + c0;
        float v[kChunk][2];                                            // parts of y, stored after the last load: a store
                                                                       // to shared memory would hold up the loads behind it
#pragma unroll
        for (int t = 0; t < kChunk; ++t) {
            const float4 q = mine[t * pair_row(PAIRS)];
            const ulonglong2 Bq = *reinterpret_cast<const ulonglong2 *>(gB + t * NP);
            const ulonglong2 Cq = BOTH ? *reinterpret_cast<const ulonglong2 *>(gC + t * NP) : ulonglong2{};
            const f32x2 Bv[2] = {Bq.x, Bq.y}, Cv[2] = {Cq.x, Cq.y};
            if (MODE == kEnds || SEG) U = add2(U, pk(q.x, q.y));
            const f32x2 uu[2] = {pk(q.x, q.x), pk(q.y, q.y)}, ux[2] = {pk(q.z, q.z), pk(q.w, q.w)};
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                f32x2 acc = 0;
                const float g = SEG ? sy[half * SY + (from + t) * CPB + c0 + c] : 0.f;
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    const f32x2 av = decay2(uu[c], A2[c][p]);
                    h[c][p] = fma2(av, h[c][p], mul2(ux[c], Bv[p]));
                    if (OUT) acc = p ? fma2(Cv[p], h[c][p], acc) : mul2(Cv[p], h[c][p]);
                    if (SEG && GROWS) {
                        float u0, u1;
                        unpk(U, u0, u1);
                        R[c][p] = carry2<true>(c ? pk(u1, u1) : pk(u0, u0), A2[c][p], mul2(pk(g, g), Cv[p]), R[c][p]);
                    } else if (SEG) {
                        P[c][p] = mul2(P[c][p], av);
                        R[c][p] = fma2(P[c][p], mul2(pk(g, g), Cv[p]), R[c][p]);
                    }
                }
                if (OUT) v[t][c] = sum2(acc);
            }
            if (OUT) lane_reduce<2, NL, PARTS>(v[t], lane);
        }
        if constexpr (OUT) {
#pragma unroll
            for (int t = 0; t < kChunk; ++t) {
                if constexpr (NL == 1) *reinterpret_cast<float2 *>(part + t * PARTS * YS) = make_float2(v[t][0], v[t][1]);
                else if (reduced_owner<2, NL, PARTS>(lane)) part[t * PARTS * YS + reduced_first<2, NL, PARTS>(lane)] = v[t][0];
            }
        }
    };

    auto later = [](int slot, int by) { return slot + by < STAGES ? slot + by : slot + by - STAGES; };
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) issue(t_begin + i * TILE, i);
    int slot = 0;                                                      // of the tile at hand
    if constexpr (!Z::DRIFT) {
        for (int t0 = t_begin; t0 < t_end; t0 += TILE, slot = later(slot, 1)) {
            issue(t0 + AHEAD * TILE, later(slot, AHEAD));
            if constexpr (St::ASYNC) copies_done<AHEAD>();
            stage(t0, slot, 0);
            __syncthreads();
#pragma unroll 1
            for (int from = 0; from < TILE; from += kChunk) compute(std::false_type{}, t0 + from, from, 0);
            __syncthreads();
            if (OUT) finish(t0, slot, 0);
        }
    } else {
        bool grows = up;                                               // from here on, for all of the CTA
        auto staged = [&] {
            if (SEG && !a.softplus) grows |= __syncthreads_or(back) != 0;
            else __syncthreads();
        };
        if (t_begin < t_end) {
            if constexpr (St::ASYNC) copies_done<AHEAD - 1>();
            stage(t_begin, 0, 0);
        }
        staged();
        int half = 0;
        for (int t0 = t_begin; t0 < t_end; t0 += TILE, slot = later(slot, 1), half ^= 1) {
            issue(t0 + AHEAD * TILE, later(slot, AHEAD));
            if (t0 + TILE < t_end) {
                if constexpr (St::ASYNC) copies_done<AHEAD - 1>();
                stage(t0 + TILE, later(slot, 1), half ^ 1);
            }
            if constexpr (SEG) {
                if (grows) compute(std::true_type{}, t0, 0, half);
                else compute(std::false_type{}, t0, 0, half);
            } else {
                compute(std::false_type{}, t0, 0, half);
            }
            staged();
        }
    }
    if constexpr (OUT) {                                               // whole tiles of padding
        const int done = t_begin < t_end ? t_begin + (t_end - t_begin + TILE - 1) / TILE * TILE : t_begin;
        for (int64_t e = threadIdx.x; e < (int64_t)max(t_stop - done, 0) * cb.count; e += kScanThreads)
            ((T *)a.y)[((size_t)b * a.T + done + e / cb.count) * D + cb.first + e % cb.count] = from_f<T>(0.f);
    }
    if (OUT && a.S_final && seg == sp.S - 1) {
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                float v[2];
                unpk(h[c][p], v[0], v[1]);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int k = ln * 4 + 2 * p + j;
                    if (c0 + c < cb.count && k < N) a.S_final[(bd + c) * N + k] = v[j];
                }
            }
    }
    if (MODE == kEnds || SEG) {
        const size_t row = seg * all + bd;
        put_state(w.E, row, 0, h[0]);
        put_state(w.E, row, 1, h[1]);
        if (SEG) {
            put_state(w.R, row, 0, R[0]);
            put_state(w.R, row, 1, R[1]);
        }
        if (ln == 0) {
            float u0, u1;
            unpk(U, u0, u1);
            if (c0 < cb.count) w.U[row] = u0;
            if (c0 + 1 < cb.count) w.U[row + 1] = u1;
        }
    }
}

template <typename T, int LN, int VEC, int MODE>
cudaError_t run_scan(const SsmArgs &a, const Split &sp, const ScanWs &w, cudaStream_t s, int *nlaunch) {
    constexpr int CPB = 2 * kScanThreads / LN;
    constexpr size_t smem = ScanSize<T, LN, VEC, MODE>::BYTES;
    const cudaError_t e = allow_smem(scan_kernel<T, LN, VEC, MODE>, smem);
    if (e != cudaSuccess) return e;
    const unsigned nblk = (unsigned)(a.B * channel_blocks(a.D, a.G, CPB));
    scan_kernel<T, LN, VEC, MODE><<<dim3(nblk, MODE == kEnds ? sp.S - 1 : sp.S), kScanThreads, smem, s>>>(a, sp, w);
    const cudaError_t r = cudaGetLastError();
    if (r == cudaSuccess) *nlaunch += 1;
    return r;
}

// Elements of an access: what divides the channels of a group and the states, and starts every
// access on a multiple of its own size.
template <typename T> int access_size(const SsmArgs &a) {
    const int per = a.D / a.G;
    return per % 4 == 0 && a.N % 4 == 0 ? 4 : sizeof(T) == 2 && per % 2 == 0 && a.N % 2 == 0 ? 2 : 1;
}
template <typename T, int LN, int MODE>
cudaError_t run_scan(const SsmArgs &a, const Split &sp, const ScanWs &w, cudaStream_t s, int *nlaunch) {
    const int v = access_size<T>(a);
    if (v == 4) return run_scan<T, LN, 4, MODE>(a, sp, w, s, nlaunch);
    if constexpr (sizeof(T) == 2)
        if (v == 2) return run_scan<T, LN, 2, MODE>(a, sp, w, s, nlaunch);
    return run_scan<T, LN, 1, MODE>(a, sp, w, s, nlaunch);
}

template <typename T, int MODE>
cudaError_t run_scan(const SsmArgs &a, const Split &sp, const ScanWs &w, cudaStream_t s, int *nlaunch) {
    switch (padded_states(a.N)) {
        case 8: return run_scan<T, 2, MODE>(a, sp, w, s, nlaunch);
        case 16: return run_scan<T, 4, MODE>(a, sp, w, s, nlaunch);
        case 32: return run_scan<T, 8, MODE>(a, sp, w, s, nlaunch);
        case 64: return run_scan<T, 16, MODE>(a, sp, w, s, nlaunch);
        default: return run_scan<T, 32, MODE>(a, sp, w, s, nlaunch);
    }
}

// CTAs of the scan along sequences and channels.
inline int64_t scan_ctas(int B, int D, int G, int N) {
    return (int64_t)B * channel_blocks(D, G, 2 * kScanThreads * 4 / padded_states(N));
}

}  // namespace ssm
}  // namespace qd
