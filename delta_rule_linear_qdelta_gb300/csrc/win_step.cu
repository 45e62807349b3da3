// One token of windowed attention against a cache of sinks + window slots, and the filling of such a cache from
// a prompt.  Token p of a sequence has slot p while p < sinks + window, later ones the ring's: slot
// sinks + (p - sinks) % window.  So the slots in use hold what the token at position p sees: itself, the
// window - 1 before it and the sinks.
#include "mixers.cuh"

namespace qd {
namespace {

constexpr int kThreads = 128, kWarps = kThreads / 32;

__device__ __forceinline__ int slot_of(int p, int sinks, int window) {
    return p < sinks || p - sinks < window ? p : sinks + (p - sinks) % window;
}

// How the slots of one (sequence, key head, tile of its queries) are cut: `splits` CTAs of `per` slots.
struct Plan {
    int qtiles, splits, per;
};

// What a CTA works on.
struct Work {
    int b, hk, q0, nq;        // sequence, key head, its first query head and their number
    int split, at, held;      // the token's slot; slots in use, the token's among them (0: an idle sequence)
    int s0, s1;               // the CTA's slots
};
__device__ __forceinline__ Work work_of(const WinArgs &a, const Plan &p, int queries) {
    const int r = a.H / a.Hkv, slots = a.sinks + a.window;
    Work w;
    int u = blockIdx.x;
    w.split = u % p.splits;
    u /= p.splits;
    const int qt = u % p.qtiles;
    u /= p.qtiles;
    w.hk = u % a.Hkv;
    w.b = u / a.Hkv;
    w.q0 = w.hk * r + qt * queries;
    w.nq = min(queries, r - qt * queries);
    const int pos = a.pos[w.b];
    w.at = pos < 0 ? -1 : slot_of(pos, a.sinks, a.window);
    w.held = pos < 0 ? 0 : pos < slots ? pos + 1 : slots;
    w.s0 = w.split * p.per;                                 // (at most slots: it fits)
    w.s1 = w.held - w.s0 > p.per ? w.s0 + p.per : w.held;
    return w;
}

// The workspace where slots are cut: for each (row, split) its part of o, then its maximum (times log2 e) and sum.
__device__ __forceinline__ float *part_o(const WinArgs &a, const Plan &p, size_t row, int split) {
    return static_cast<float *>(a.ws) + (row * p.splits + split) * a.d;
}
__device__ __forceinline__ float *part_ml(const WinArgs &a, const Plan &p, size_t row, int split) {
    return static_cast<float *>(a.ws) + (size_t)a.B * a.H * p.splits * a.d + (row * p.splits + split) * 2;
}

// Joins PARTS parts of each of w.nq queries in shared memory (ml: maximum and sum, acc: rows of LD floats) and
// writes the output, or the CTA's part of it where slots are cut.
template <typename T, int PARTS, int QUERIES, int LD>
__device__ __forceinline__ void join(const WinArgs &a, const Plan &p, const Work &w, const float (&ml)[PARTS][QUERIES][2],
                                     const float (&acc)[PARTS][QUERIES][LD]) {
    for (int u = threadIdx.x; u < w.nq * a.d; u += kThreads) {
        const int q = u / a.d, c = u % a.d;
        float m = -INFINITY, l = 0.f, y = 0.f;
#pragma unroll
        for (int i = 0; i < PARTS; ++i) m = fmaxf(m, ml[i][q][0]);
#pragma unroll
        for (int i = 0; i < PARTS; ++i) {
            const float f = ml[i][q][1] == 0.f ? 0.f : exp2_fast(ml[i][q][0] - m);
            l = fmaf(f, ml[i][q][1], l);
            y = fmaf(f, acc[i][q][c], y);
        }
        const size_t row = (size_t)w.b * a.H + w.q0 + q;
        if (p.splits == 1) {
            static_cast<T *>(a.o)[row * a.d + c] = from_f<T>(w.held ? y / l : 0.f);
        } else {
            part_o(a, p, row, w.split)[c] = y;
            if (c == 0) part_ml(a, p, row, w.split)[0] = m, part_ml(a, p, row, w.split)[1] = l;
        }
    }
}

// One CTA a (sequence, head): joins the parts of its splits, four threads a column over every fourth of them.
// (One thread a column, loads one after the other: 20 us for 103 splits in the place of 4.)
constexpr int kMostSplits = 3 * kSMs, kJoinThreads = 4 * 128;

template <typename T> __global__ void __launch_bounds__(kJoinThreads) win_join_kernel(WinArgs a, Plan p) {
    __shared__ float weight[kMostSplits], most[kJoinThreads / 32], part[4][128], part_l[4][128];
    const size_t row = blockIdx.x;
    const int tid = threadIdx.x, c = tid & 127, k = tid >> 7;
    const float *ml = part_ml(a, p, row, 0), *acc = part_o(a, p, row, 0);
    const float2 own = tid < p.splits ? *reinterpret_cast<const float2 *>(ml + 2 * tid) : make_float2(-INFINITY, 0.f);
    float m = own.x;
#pragma unroll
    for (int off = 16; off; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    if ((tid & 31) == 0) most[tid >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kJoinThreads / 32; ++i) m = fmaxf(m, most[i]);
    // an empty part (sum 0) has no say, a NaN one has
    if (tid < p.splits) weight[tid] = own.y == 0.f ? 0.f : exp2_fast(own.x - m);
    __syncthreads();
    float l = 0.f, y = 0.f;
#pragma unroll 8
    for (int i = k; i < p.splits; i += 4) {
        l = fmaf(weight[i], ml[2 * i + 1], l);
        if (c < a.d) y = fmaf(weight[i], acc[(size_t)i * a.d + c], y);
    }
    part[k][c] = y;
    part_l[k][c] = l;
    __syncthreads();
    if (tid < a.d) {
        l = (part_l[0][c] + part_l[1][c]) + (part_l[2][c] + part_l[3][c]);
        y = (part[0][c] + part[1][c]) + (part[2][c] + part[3][c]);
        static_cast<T *>(a.o)[row * a.d + c] = from_f<T>(l == 0.f ? 0.f : y / l);      // (l = 0: an idle sequence)
    }
}

// ------------------------------------------------------------------ bf16: scores and sums by warp-level products
// Memory bound (the cache is read once: 2.15 GB for 512 sequences of 2052 slots, 4 key heads of 128), so the
// products only have to keep out of the way: with up to 16 queries against a slot they are 16x8x16 ones, far below
// a tcgen05 tile, and their fragments come straight from global memory, 16 bytes a lane.  That takes two
// permutations, which the sums do not see: lane (g, t) holds elements 32 j + 8 t .. + 7 of a key's row in the
// place of the fragment's two pairs, the queries' rows the same way; and for the values it holds columns
// 64 i + 8 g .. + 7 of slots 2 t, 2 t + 1, 2 t + 8, 2 t + 9, whose pairs of slots are then put together by column.
//     S^T (16 slots x 8 queries) = K Q^T,   O^T (16 columns x 8 queries) += V^T P^T
// P^T is S^T's layout transposed (movmatrix).  A warp walks every fourth tile of 16 slots; a tile's keys and values
// are under way while the tile before is computed.  The maximum is renewed, and sums rescaled, only when a score
// passes it.  Measured there: 315 us, the copy rate (101 %); one sequence of 32772 slots: 12.3 us and 5.6 for the join.

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ uint32_t word(const uint4 &v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

template <int DP, int NQ> __global__ void __launch_bounds__(kThreads) win_step_mma_kernel(WinArgs a, Plan plan) {
    constexpr int J = DP / 32, I = DP / 64;
    __shared__ float ml[kWarps][8 * NQ][2], acc[kWarps][8 * NQ][DP + 1];
    typedef __nv_bfloat16 T;
    const Work w = work_of(a, plan, 8 * NQ);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const size_t row = (size_t)a.Hkv * a.d, slots = (size_t)a.sinks + a.window;
    const size_t cache = (w.b * slots * a.Hkv + w.hk) * a.d, own = ((size_t)w.b * a.Hkv + w.hk) * a.d;
    T *K = static_cast<T *>(a.K) + cache, *V = static_cast<T *>(a.V) + cache;
    const T *k = static_cast<const T *>(a.k) + own, *v = static_cast<const T *>(a.v) + own;
    const uint4 none = make_uint4(0u, 0u, 0u, 0u);

    uint4 q[NQ][J], kr[2][J], vr[4][I];
#pragma unroll
    for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int j = 0; j < J; ++j)
            q[n][j] = 8 * n + g < w.nq && 32 * j + 8 * t < a.d
                          ? *reinterpret_cast<const uint4 *>(static_cast<const T *>(a.q) + ((size_t)w.b * a.H + w.q0 + 8 * n + g) * a.d + 32 * j + 8 * t)
                          : none;
    auto load_k = [&](int s) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int r = s + g + 8 * u;                    // the token's own row may not be in the cache yet
            const T *from = (r == w.at ? k : K + r * row) + 8 * t;
#pragma unroll
            for (int j = 0; j < J; ++j)
                kr[u][j] = r < w.s1 && 32 * j + 8 * t < a.d ? __ldcs(reinterpret_cast<const uint4 *>(from + 32 * j)) : none;
        }
    };
    auto load_v = [&](int s) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int r = s + 2 * t + (u & 1) + 8 * (u >> 1);
            const T *from = (r == w.at ? v : V + r * row) + 8 * g;
#pragma unroll
            for (int i = 0; i < I; ++i)
                vr[u][i] = r < w.s1 && 64 * i + 8 * g < a.d ? __ldcs(reinterpret_cast<const uint4 *>(from + 64 * i)) : none;
        }
    };
    float o[NQ][4 * I][4], m[NQ][2], l[NQ][2];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
        m[n][0] = m[n][1] = -INFINITY;
        l[n][0] = l[n][1] = 0.f;
#pragma unroll
        for (int i = 0; i < 4 * I; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[n][i][e] = 0.f;
    }
    const float scale = a.scale * kLog2e;
    int s = w.s0 + 16 * warp;
    if (s < w.s1) {
        load_k(s);
        load_v(s);
    }
    if (w.at >= w.s0 && w.at < w.s1 && w.q0 == w.hk * (a.H / a.Hkv)) {   // the token's row into its slot
        const int c = 8 * (threadIdx.x & 15);
        if (threadIdx.x < 32 && c < a.d) {
            const T *from = (threadIdx.x < 16 ? k : v) + c;
            *reinterpret_cast<uint4 *>((threadIdx.x < 16 ? K : V) + w.at * row + c) = *reinterpret_cast<const uint4 *>(from);
        }
    }
    for (; s < w.s1; s += 16 * kWarps) {
        float c[NQ][4];
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
            c[n][0] = c[n][1] = c[n][2] = c[n][3] = 0.f;
#pragma unroll
            for (int j = 0; j < J; ++j) {
                mma_bf16(c[n], kr[0][j].x, kr[1][j].x, kr[0][j].y, kr[1][j].y, q[n][j].x, q[n][j].y);
                mma_bf16(c[n], kr[0][j].z, kr[1][j].z, kr[0][j].w, kr[1][j].w, q[n][j].z, q[n][j].w);
            }
        }
        const int next = s + 16 * kWarps;
        if (next < w.s1) load_k(next);
        uint32_t b[NQ][2];
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
#pragma unroll
            for (int e = 0; e < 4; ++e) c[n][e] = s + g + 8 * (e >> 1) < w.s1 ? scale * c[n][e] : -INFINITY;
            float hi0 = fmaxf(c[n][0], c[n][2]), hi1 = fmaxf(c[n][1], c[n][3]);
            if (__any_sync(0xffffffffu, hi0 > m[n][0] || hi1 > m[n][1])) {
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) {
                    hi0 = fmaxf(hi0, __shfl_xor_sync(0xffffffffu, hi0, off));
                    hi1 = fmaxf(hi1, __shfl_xor_sync(0xffffffffu, hi1, off));
                }
                hi0 = fmaxf(hi0, m[n][0]);
                hi1 = fmaxf(hi1, m[n][1]);
                const float f0 = exp2_fast(m[n][0] - hi0), f1 = exp2_fast(m[n][1] - hi1);
                m[n][0] = hi0;
                m[n][1] = hi1;
                l[n][0] *= f0;
                l[n][1] *= f1;
#pragma unroll
                for (int i = 0; i < 4 * I; ++i) {
                    o[n][i][0] *= f0;
                    o[n][i][1] *= f1;
                    o[n][i][2] *= f0;
                    o[n][i][3] *= f1;
                }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                c[n][e] = exp2_fast(c[n][e] - m[n][e & 1]);
                l[n][e & 1] += c[n][e];
            }
            b[n][0] = transpose8(pack2(c[n][0], c[n][1]));  // probabilities are held in bf16 (half a step, 2^-8, as the values)
            b[n][1] = transpose8(pack2(c[n][2], c[n][3]));
        }
#pragma unroll
        for (int i = 0; i < I; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t r0 = word(vr[0][i], e), r1 = word(vr[1][i], e), r2 = word(vr[2][i], e), r3 = word(vr[3][i], e);
                const uint32_t a0 = __byte_perm(r0, r1, 0x5410), a1 = __byte_perm(r0, r1, 0x7632);
                const uint32_t a2 = __byte_perm(r2, r3, 0x5410), a3 = __byte_perm(r2, r3, 0x7632);
#pragma unroll
                for (int n = 0; n < NQ; ++n) mma_bf16(o[n][4 * i + e], a0, a1, a2, a3, b[n][0], b[n][1]);
            }
        if (next < w.s1) load_v(next);
    }
#pragma unroll
    for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], off);
            const int query = 8 * n + 2 * t + e;
            if (g == 0) ml[warp][query][0] = m[n][e], ml[warp][query][1] = l[n][e];
#pragma unroll
            for (int i = 0; i < 4 * I; ++i) {
                const int col = 64 * (i / 4) + 8 * g + 2 * (i % 4);
                acc[warp][query][col] = o[n][i][e];
                acc[warp][query][col + 1] = o[n][i][2 + e];
            }
        }
    __syncthreads();
    join<T>(a, plan, w, ml, acc);
}

// ------------------------------------------------------------------ fp32
// Eight lanes hold a slot's row, so that a dot product takes three shuffles, and keep the maximum, the sum and the
// values' sums of the slots that they see; the CTA's 16 groups of lanes are joined at the end.  A CTA has up to NQ of
// the queries that share a key head.
constexpr int kGroups = kThreads / 8;

template <int DP, int NQ> __global__ void __launch_bounds__(kThreads) win_step_f32_kernel(WinArgs a, Plan plan) {
    constexpr int C = DP / 32;                              // accesses of four floats a lane
    __shared__ float ml[kGroups][NQ][2], acc[kGroups][NQ][DP + 1];
    const Work w = work_of(a, plan, NQ);
    const int group = threadIdx.x >> 3, lane = threadIdx.x & 7;
    const size_t row = (size_t)a.Hkv * a.d, slots = (size_t)a.sinks + a.window;
    const size_t cache = (w.b * slots * a.Hkv + w.hk) * a.d, own = ((size_t)w.b * a.Hkv + w.hk) * a.d;
    float *K = static_cast<float *>(a.K) + cache, *V = static_cast<float *>(a.V) + cache;
    const float *k = static_cast<const float *>(a.k) + own, *v = static_cast<const float *>(a.v) + own;
    const float4 none = make_float4(0.f, 0.f, 0.f, 0.f);
    auto get = [&](float4 (&x)[C], const float *from, bool on) {
#pragma unroll
        for (int c = 0; c < C; ++c)
            x[c] = on && 32 * c + 4 * lane < a.d ? *reinterpret_cast<const float4 *>(from + 32 * c + 4 * lane) : none;
    };
    float4 q[NQ][C], o[NQ][C];
    float m[NQ], l[NQ];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
        get(q[n], static_cast<const float *>(a.q) + ((size_t)w.b * a.H + w.q0 + n) * a.d, n < w.nq);
        m[n] = -INFINITY;
        l[n] = 0.f;
#pragma unroll
        for (int c = 0; c < C; ++c) o[n][c] = none;
    }
    if (w.at >= w.s0 && w.at < w.s1 && w.q0 == w.hk * (a.H / a.Hkv) && (int)threadIdx.x < a.d) {
        K[w.at * row + threadIdx.x] = k[threadIdx.x];
        V[w.at * row + threadIdx.x] = v[threadIdx.x];
    }
    const float scale = a.scale * kLog2e;
    for (int s = w.s0; s < w.s1; s += kGroups) {            // (the whole warp goes round: shuffles)
        const int r = s + group;
        const bool on = r < w.s1;
        float4 kx[C], vx[C];
        get(kx, r == w.at ? k : K + r * row, on);
        get(vx, r == w.at ? v : V + r * row, on);
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
            float x = 0.f;
#pragma unroll
            for (int c = 0; c < C; ++c)
                x = fmaf(q[n][c].x, kx[c].x, fmaf(q[n][c].y, kx[c].y, fmaf(q[n][c].z, kx[c].z, fmaf(q[n][c].w, kx[c].w, x))));
#pragma unroll
            for (int off = 4; off; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
            if (!on) continue;
            x *= scale;
            if (x > m[n]) {
                const float f = exp2_fast(m[n] - x);
                m[n] = x;
                l[n] *= f;
#pragma unroll
                for (int c = 0; c < C; ++c) o[n][c] = make_float4(f * o[n][c].x, f * o[n][c].y, f * o[n][c].z, f * o[n][c].w);
            }
            const float e = exp2_fast(x - m[n]);
            l[n] += e;
#pragma unroll
            for (int c = 0; c < C; ++c) {
                o[n][c].x = fmaf(e, vx[c].x, o[n][c].x);
                o[n][c].y = fmaf(e, vx[c].y, o[n][c].y);
                o[n][c].z = fmaf(e, vx[c].z, o[n][c].z);
                o[n][c].w = fmaf(e, vx[c].w, o[n][c].w);
            }
        }
    }
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
        if (lane == 0) ml[group][n][0] = m[n], ml[group][n][1] = l[n];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            float *to = &acc[group][n][32 * c + 4 * lane];
            to[0] = o[n][c].x, to[1] = o[n][c].y, to[2] = o[n][c].z, to[3] = o[n][c].w;
        }
    }
    __syncthreads();
    join<float>(a, plan, w, ml, acc);
}

// Queries of a CTA: 8 or 16 of bf16, up to 4 of fp32.  Slots are cut while the CTAs would leave SMs without
// three of them, at least 192 to a CTA but the last (three tiles of 16 for each of four warps, or twelve rows for each of 16 groups).
int queries_of(int r, int dtype) { return dtype == kBF16 ? (r > 8 ? 16 : 8) : (r >= 4 ? 4 : r >= 2 ? 2 : 1); }
Plan plan_of(int N, int H, int Hkv, int window, int sinks, int dtype) {
    const int r = H / Hkv, slots = window + sinks, least = 256;
    Plan p;
    p.qtiles = (r + queries_of(r, dtype) - 1) / queries_of(r, dtype);
    const long long ctas = (long long)N * Hkv * p.qtiles, most = (slots + least - 1) / least;
    const long long want = (kMostSplits + ctas - 1) / ctas;
    p.splits = (int)(want < most ? want : most);
    p.per = ((slots + p.splits - 1) / p.splits + 63) / 64 * 64;
    p.splits = (slots + p.per - 1) / p.per;
    return p;
}

template <int DP> cudaError_t run_step(const WinArgs &a, const Plan &p, int dtype, cudaStream_t s) {
    const unsigned grid = (unsigned)((size_t)a.B * a.Hkv * p.qtiles * p.splits);
    const int queries = queries_of(a.H / a.Hkv, dtype);
    if (dtype == kBF16) {
        if (queries == 8) win_step_mma_kernel<DP, 1><<<grid, kThreads, 0, s>>>(a, p);
        else win_step_mma_kernel<DP, 2><<<grid, kThreads, 0, s>>>(a, p);
    } else {
        if (queries == 1) win_step_f32_kernel<DP, 1><<<grid, kThreads, 0, s>>>(a, p);
        else if (queries == 2) win_step_f32_kernel<DP, 2><<<grid, kThreads, 0, s>>>(a, p);
        else win_step_f32_kernel<DP, 4><<<grid, kThreads, 0, s>>>(a, p);
    }
    return cudaGetLastError();
}

// 16 bytes a thread; slots without a token are left as they are.
template <typename T> __global__ void win_fill_kernel(WinArgs a) {
    constexpr int VEC = 16 / sizeof(T);
    const int slots = a.sinks + a.window;
    const size_t row = (size_t)a.Hkv * a.d, per_row = row / VEC;          // (row: up to 2^36 elements)
    const size_t u = (size_t)blockIdx.x * blockDim.x + threadIdx.x, all = (size_t)a.B * slots * per_row;
    if (u >= all) return;
    const int b = (int)(u / (slots * per_row)), s = (int)(u / per_row % slots);
    const size_t c = u % per_row * VEC;
    const int n = a.past + real_tokens(a.lens, b, a.T);
    int p = s;
    if (s >= a.sinks && n > slots) {                        // the last token whose slot this is
        const int count = n - a.sinks, r = s - a.sinks;
        p = a.sinks + count - 1 - (count - 1 - r) % a.window;
    }
    if (p >= n) return;
    const size_t from = ((size_t)b * (a.past + a.T) + p) * row + c, to = ((size_t)b * slots + s) * row + c;
    Pack<T, VEC> x, y;
    x.load(static_cast<const T *>(a.k) + from);
    y.load(static_cast<const T *>(a.v) + from);
    x.store(static_cast<T *>(a.K) + to);
    y.store(static_cast<T *>(a.V) + to);
}

}  // namespace

size_t win_step_workspace(int N, int H, int Hkv, int d, int window, int sinks, int dtype) {
    const Plan p = plan_of(N, H, Hkv, window, sinks, dtype);
    return p.splits == 1 ? 0 : sizeof(float) * (size_t)N * H * p.splits * (d + 2);
}

cudaError_t launch_win_step(const WinArgs &a, int dtype, cudaStream_t s, int *n) {
    const Plan p = plan_of(a.B, a.H, a.Hkv, a.window, a.sinks, dtype);
    cudaError_t e = a.d > 64 ? run_step<128>(a, p, dtype, s) : run_step<64>(a, p, dtype, s);
    if (e != cudaSuccess) return e;
    *n += 1;
    if (p.splits > 1) {
        const unsigned rows = (unsigned)((size_t)a.B * a.H);
        if (dtype == kBF16) win_join_kernel<__nv_bfloat16><<<rows, kJoinThreads, 0, s>>>(a, p);
        else win_join_kernel<float><<<rows, kJoinThreads, 0, s>>>(a, p);
        e = cudaGetLastError();
        if (e == cudaSuccess) *n += 1;
    }
    return e;
}

cudaError_t launch_win_fill(const WinArgs &a, int dtype, cudaStream_t s, int *n) {
    const size_t vec = dtype == kBF16 ? 8 : 4, all = (size_t)a.B * (a.sinks + a.window) * ((size_t)a.Hkv * a.d / vec);
    const unsigned grid = (unsigned)((all + 255) / 256);
    if (dtype == kBF16) win_fill_kernel<__nv_bfloat16><<<grid, 256, 0, s>>>(a);
    else win_fill_kernel<float><<<grid, 256, 0, s>>>(a);
    *n += 1;
    return cudaGetLastError();
}

}  // namespace qd
