// Backward of the selective state space scan (ssm_scan.cuh has the forward's formulas).  With
// g = dy and the gradient dh_t of L with respect to h_t,
//
//   dh_t = C_t g_t + a_{t+1} dh_{t+1}   (+ dS_final at the last token),   r_t = dh_t a_t h_{t-1}
//   dx = u sum_n dh B + D g,  du = sum_n A r + x sum_n dh B,  ddelta = du softplus'
//   dA = sum_{b,t} u r,  dB = sum_d dh u x,  dC = sum_d g h,  dD = sum g x,  dS0 = a_1 dh_1
//
// Launches:
//  1. the forward recurrence again, leaving the state entering every chunk of 8 tokens in the
//     workspace (8 bytes per token and channel at N = 16).  Few channels over many tokens: the
//     tokens are cut into segments as in the forward; each starts from zero and also leaves its
//     end E, its sum of u and R, the gradient that its own tokens send to the state entering it,
//     R = sum_t (prod_{s<=t} a_s) C_t g_t.
//  2. gradients: a CTA walks its segment's chunks backwards.  Per chunk it recomputes the 8
//     states into registers from the checkpoint, then runs dh down the tokens.  Sums over n
//     join over the LN lanes of a channel; sums over channels (dB, dC) over the channels of a
//     warp by shuffles, over the CTA's warps through shared memory.
//  3. the sums over CTAs: dB, dC over the channel blocks, and dA, dD, d bias over sequences
//     and segments; in a fixed order, so results do not change from run to run.
// Bound by the shared-memory pipe and instruction issue: two exponentials and about 20 operations
// per (token, channel, state) in launch 2, one and 4 in launch 1, or one and 7 where it works on
// segments (R and its products).  4 x 4096 tokens x 1024 channels x 16 states, bf16: 360 us, of which
// launch 1 (segments) takes 100, launch 2 243 and the sums 17.  Launch 2 keeps 8 tokens' states in 216
// registers, so 8 warps share an SM.  (Two halves of what it stages, with one barrier a chunk as in
// launch 1, took 371 us in all against 364: the code that is then there twice is slower.)
// States that may grow: carry2 joins segments, see there.
#include "layer_common.cuh"
#include "ssm_scan.cuh"

namespace qd {
namespace {

using namespace ssm;

constexpr int kStages = 3;
constexpr int kGradThreads = 128, kGradWarps = kGradThreads / 32, kSumThreads = 256;

// Everything in the workspace, in floats from its start.
struct BwdWs {
    Split sp;
    int nck, nb;                      // checkpoints a sequence; channel blocks a group
    int rows;                         // rows of dA/dD/dbias partials
    size_t chk, ucum, E, U, R, dbc, par, total;
};

__host__ __device__ constexpr int grad_lanes(int N) { return padded_states(N) / 4; }
__host__ __device__ constexpr int grad_channels(int N) { return 2 * kGradThreads / grad_lanes(N); }

BwdWs bwd_ws(int B, int T, int D, int G, int N) {
    BwdWs w;
    const size_t NP = padded_states(N), bd = (size_t)B * D;
    w.nb = channel_blocks(D, G, grad_channels(N)) / G;
    // One segment when the CTAs fill every SM's two places; otherwise two rounds of them (4 x 4096 x
    // 1024 channels: 414 us in one round, 364 in two, 363 in three; 3 x 517 x 770, ragged: 98, 71, 77).
    w.sp = split_tokens((int64_t)B * G * w.nb, T, 2 * kSMs, 4 * kSMs, 8 * kChunk, kChunk);
    w.nck = (T + kChunk - 1) / kChunk;
    w.rows = B * w.sp.S;
    const bool multi = w.sp.S > 1;
    size_t at = 0;
    auto take = [&](size_t n) { const size_t p = at; at += (n + 63) / 64 * 64; return p; };
    w.chk = take((size_t)w.nck * bd * NP);
    w.ucum = take(multi ? (size_t)w.nck * bd : 0);
    w.E = take(multi ? w.sp.S * bd * NP : 0);
    w.U = take(multi ? w.sp.S * bd : 0);
    w.R = take(multi ? w.sp.S * bd * NP : 0);
    w.dbc = take((size_t)B * T * G * w.nb * 2 * NP);
    w.par = take((size_t)w.rows * D * (N + 2));
    w.total = at;
    return w;
}

// Launch 2.  A thread holds 2 channels by 4 states, LN lanes share a channel pair, CL = 32 / LN
// pairs make a warp.  dB and dC of a token are sums over the warp's channels of 4 states each:
// they are joined like lane_reduce, but a lane keeps its four states in the order n ^ m, m two
// of its channel bits, so what it gives away is always its upper half and nothing has to be
// selected; B and C lie in shared memory in all four orders.  The sums over n behind dx and
// ddelta are left as parts in shared memory for the thread that writes the rows.
// Row of the parts: float4 (s1 of both channels, s2 of both) of pair p at pair_at(p).  This length
// and order_size bring the lanes that shared memory serves at once to different banks.
__host__ __device__ constexpr int part_row(int LN) { return pair_row(kGradThreads / LN) + (LN == 2 ? 2 : 1); }
// From B (or C) in one order to the next.
__host__ __device__ constexpr int order_size(int NP) { return kChunk * NP + 8; }

template <typename T, int LN, int VEC>
__global__ void __launch_bounds__(kGradThreads, 2) grads_kernel(SsmArgs a, BwdWs w, float *ws) {
    constexpr int PAIRS = kGradThreads / LN, CPB = 2 * PAIRS, NP = 4 * LN, CL = 32 / LN;
    constexpr int PARTS = sum_parts(LN), NL = LN / PARTS, PR = part_row(LN);
    using St = Staging<T, kGradThreads, kChunk, CPB, NP, 3, VEC, kStages>;
    constexpr int PER = St::PER;
    extern __shared__ float4 smem4[];
    T *raw = reinterpret_cast<T *>(smem4);                             // [kStages] chunks on their way
    float4 *su = smem4 + St::BYTES / 16;                               // [kChunk][pair_row] (u0, u1, u0 x0, u1 x1)
    float4 *sp = su + kChunk * pair_row(PAIRS);                        // [kChunk][PARTS][PR] parts of the sums over n
    float2 *sg = reinterpret_cast<float2 *>(sp + kChunk * PARTS * PR); // [kChunk][PAIRS] (g0, g1)
    float *ss = reinterpret_cast<float *>(sg + kChunk * PAIRS);        // [kChunk][CPB] softplus'
    float *sB = ss + kChunk * CPB;                                     // [4 orders][kChunk][NP]
    float *sC = sB + 4 * order_size(NP);
    float *sr = sC + 4 * order_size(NP);                                  // [warps][kChunk][2 NP] (dB, dC)

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, ln = tid % LN, pr = tid / LN, seg = blockIdx.y;
    const int cl = lane / LN, m = (CL >= 2 ? (cl & 1) * 2 : 0) + (CL >= 4 ? cl >> 1 & 1 : 0);
    const int nblk = channel_blocks(a.D, a.G, CPB), b = blockIdx.x / nblk, blk = blockIdx.x % nblk;
    const ChannelBlock cb(a, blk, CPB);
    const int D = a.D, N = a.N, S = w.sp.S, c0 = 2 * pr;
    const int n = seq_len(a.lens, b, a.T);
    const int t_begin = seg * w.sp.len, t_stop = min(t_begin + w.sp.len, a.T), t_end = min(t_stop, n);
    const size_t bd = (size_t)b * D + cb.first + c0, all = (size_t)a.B * D;

    // four states of a channel in the lane's order
    auto order = [&](float4 v, f32x2(&to)[2]) {
        if (m & 2) v = make_float4(v.z, v.w, v.x, v.y);
        if (m & 1) v = make_float4(v.y, v.x, v.w, v.z);
        to[0] = pk(v.x, v.y);
        to[1] = pk(v.z, v.w);
    };
    // a parameter or state [.., N] of channel c, by single accesses: once per segment
    auto gather = [&](const float *base, size_t row, int c, f32x2(&to)[2]) {
        float f[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int k = ln * 4 + (i ^ m);
            f[i] = base && c0 + c < cb.count && k < N ? base[row * N + k] : 0.f;
        }
        to[0] = pk(f[0], f[1]);
        to[1] = pk(f[2], f[3]);
    };
    auto scatter = [&](float *base, size_t row, int c, const f32x2(&v)[2]) {
        float f[4];
        unpk(v[0], f[0], f[1]);
        unpk(v[1], f[2], f[3]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int k = ln * 4 + (i ^ m);
            if (c0 + c < cb.count && k < N) base[row * N + k] = f[i];
        }
    };
    // the same of a workspace array [.., NP]
    auto fetch = [&](size_t base, size_t row, int c, f32x2(&to)[2]) {
        order(*reinterpret_cast<const float4 *>(ws + base + (row + c) * NP + ln * 4), to);
    };

    f32x2 A2[2][2], dh[2][2], dA[2][2], hin[2][2];                     // A log2(e); dh: what reaches the state from the right
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        gather(a.A, cb.first + c0 + c, c, A2[c]);
        gather(a.dS_final, bd + c, c, dh[c]);
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            A2[c][p] = mul2(A2[c][p], pk(kLog2e, kLog2e));
            dA[c][p] = hin[c][p] = 0;
        }
    }
    const bool up = S > 1 && (!a.softplus || rates_grow(A2));
    if (S > 1) {
        auto fold = [&](auto careful) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                if (c0 + c >= cb.count) continue;
                for (int s = S - 1; s > seg; --s) {
                    const float U = ws[w.U + s * all + bd + c];
                    f32x2 r[2];
                    fetch(w.R, s * all + bd, c, r);
#pragma unroll
                    for (int p = 0; p < 2; ++p) dh[c][p] = carry2<careful.value>(pk(U, U), A2[c][p], dh[c][p], r[p]);
                }
                for (int s = 0; s < seg; ++s) {
                    const float U = ws[w.U + s * all + bd + c];
                    f32x2 e[2];
                    fetch(w.E, s * all + bd, c, e);
#pragma unroll
                    for (int p = 0; p < 2; ++p) hin[c][p] = carry2<careful.value>(pk(U, U), A2[c][p], hin[c][p], e[p]);
                }
            }
        };
        if (up) fold(std::true_type{});
        else fold(std::false_type{});
    }
    float bias[VEC], skip[VEC], dDs[VEC], dbs[VEC];                    // of the channels this thread writes
    St::param(a.delta_bias, cb, bias);
    St::param(a.Dskip, cb, skip);
#pragma unroll
    for (int k = 0; k < VEC; ++k) dDs[k] = dbs[k] = 0.f;
    const int chunks = t_begin < t_end ? (t_end - t_begin + kChunk - 1) / kChunk : 0;
    typename St::Cursor at(a, cb, b, t_begin + (chunks - 1) * kChunk, {a.x, a.delta, a.dy});
    // the c-th chunk of the segment, none (and no copies) before the first
    auto issue = [&](int c, int buf) { St::issue(at, raw, buf, a, cb, t_begin + c * kChunk, c >= 0, n, true, -1); };
    issue(chunks - 1, 0);
    issue(chunks - 2, 1);
    // this thread's first row of dx and ddelta, and the CTA's of the partial dB and dC, of the chunk at hand
    const int last = t_begin + (chunks - 1) * kChunk;
    size_t out = ((size_t)b * a.T + last + St::tok(0)) * D + cb.first + St::chan();
    const size_t dbc_row = (size_t)a.G * w.nb * 2 * NP;
    float *dbc = ws + w.dbc + ((size_t)b * a.T + last) * dbc_row + ((size_t)cb.group * w.nb + blk % w.nb) * 2 * NP;
    // the checkpoint of the next chunk is on its way while one is computed
    float4 ck_h[2];
    float ck_u[2];
    const int c1 = min(c0 + 1, cb.count - 1), cz = min(c0, cb.count - 1);
    const float *ck_at = ws + w.chk + ((size_t)(last / kChunk) * all + (size_t)b * D + cb.first + cz) * NP + ln * 4;
    const float *cu_at = ws + w.ucum + (size_t)(last / kChunk) * all + (size_t)b * D + cb.first + cz;
    auto checkpoint = [&] {
        ck_h[0] = *reinterpret_cast<const float4 *>(ck_at);
        ck_h[1] = *reinterpret_cast<const float4 *>(ck_at + (c1 - cz) * NP);
        if (seg > 0) {
            ck_u[0] = cu_at[0];
            ck_u[1] = cu_at[c1 - cz];
        }
        ck_at -= all * NP;
        cu_at -= all;
    };
    if (chunks) checkpoint();
    int buf = 0;
    for (int chunk = chunks - 1; chunk >= 0; --chunk, buf = buf + 1 < kStages ? buf + 1 : 0) {
        const int t0 = t_begin + chunk * kChunk;
        issue(chunk - 2, buf + 2 < kStages ? buf + 2 : buf + 2 - kStages);
        if constexpr (St::ASYNC) copies_done<2>();
        const bool full = St::full(cb, t0, n);
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int t = St::tok(i), c = St::chan();
            if (t >= kChunk) break;
            float u[VEC], x[VEC], g[VEC], sig[VEC];
            St::get(raw, buf, 0, i, a, cb, b, t0, n, a.x, x);
            St::get(raw, buf, 1, i, a, cb, b, t0, n, a.delta, u);
            St::get(raw, buf, 2, i, a, cb, b, t0, n, a.dy, g);
#pragma unroll
            for (int k = 0; k < VEC; k += 2) {
                float e0 = 0.f, e1 = 0.f, none = 0.f, &u1 = k + 1 < VEC ? u[k + 1 < VEC ? k + 1 : k] : none;
                u[k] += bias[k];
                if (k + 1 < VEC) u1 += bias[k + 1 < VEC ? k + 1 : k];
                const float r0 = u[k], r1 = u1;
                if (a.softplus) softplus2(u[k], u1, e0, e1);
                sig[k] = a.softplus ? softplus_grad(r0, e0) : 1.f;
                if (k + 1 < VEC) sig[k + 1 < VEC ? k + 1 : k] = a.softplus ? softplus_grad(r1, e1) : 1.f;
            }
            if (!full && !(t0 + t < n && c < cb.count)) {              // of the padding nothing counts
#pragma unroll
                for (int k = 0; k < VEC; ++k) u[k] = 0.f;
            }
            if constexpr (VEC > 1) {
#pragma unroll
                for (int k = 0; k < VEC; k += 2)
                    su[t * pair_row(PAIRS) + pair_at((c + k) / 2, PAIRS)] = make_float4(u[k], u[k + 1], u[k] * x[k], u[k + 1] * x[k + 1]);
                Pack<float, VEC> v;
                v.set(sig);
                v.store(ss + t * CPB + c);
                v.set(g);
                v.store(reinterpret_cast<float *>(sg + t * PAIRS + c / 2));
            } else {
                float *to = reinterpret_cast<float *>(su + t * pair_row(PAIRS) + pair_at(c / 2, PAIRS)) + (c & 1);
                to[0] = u[0];
                to[2] = u[0] * x[0];
                reinterpret_cast<float *>(sg + t * PAIRS + c / 2)[c & 1] = g[0];
                ss[t * CPB + c] = sig[0];
            }
        }
        St::get_groups(raw, buf, a, cb, b, t0, n, true, [&](int which, int t, int k, const float (&f)[VEC]) {
            float *to = (which ? sC : sB) + t * NP + k;
#pragma unroll
            for (int o = 0; o < 4; ++o) {
                if constexpr (VEC == 4) {
                    *reinterpret_cast<float4 *>(to + o * order_size(NP)) = make_float4(f[o], f[1 ^ o], f[2 ^ o], f[3 ^ o]);
                } else {
#pragma unroll
                    for (int j = 0; j < VEC; ++j) to[o * order_size(NP) - k % 4 + ((k % 4 + j) ^ o)] = f[j];
                }
            }
        });
        const float4 *mine = su + pair_at(pr, PAIRS);
        const float *gB = sB + m * order_size(NP) + ln * 4, *gC = sC + m * order_size(NP) + ln * 4;
        __syncthreads();

        f32x2 h0[2][2], hh[kChunk][2][2], dAt[2][2] = {};              // dAt: the chunk's share; short sums lose less
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const bool on = c0 + c < cb.count;
            order(on ? ck_h[c] : make_float4(0.f, 0.f, 0.f, 0.f), h0[c]);
            if (seg > 0) {
                const float U = on ? ck_u[c] : 0.f;
#pragma unroll
                for (int p = 0; p < 2; ++p)
                    h0[c][p] = up ? carry2<true>(pk(U, U), A2[c][p], hin[c][p], h0[c][p])
                                  : carry2<false>(pk(U, U), A2[c][p], hin[c][p], h0[c][p]);
            }
        }
        if (chunk > 0) checkpoint();
#pragma unroll
        for (int k = 0; k < kChunk; ++k) {
            const float4 q = mine[k * pair_row(PAIRS)];
            const ulonglong2 Bv = *reinterpret_cast<const ulonglong2 *>(gB + k * NP);
            const f32x2 Bp[2] = {Bv.x, Bv.y}, uu[2] = {pk(q.x, q.x), pk(q.y, q.y)}, ux[2] = {pk(q.z, q.z), pk(q.w, q.w)};
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int p = 0; p < 2; ++p)
                    hh[k][c][p] = fma2(decay2(uu[c], A2[c][p]), k ? hh[k ? k - 1 : 0][c][p] : h0[c][p], mul2(ux[c], Bp[p]));
        }
        // a token's operands are loaded before the last one's sums are stored: the loads behind a store to
        // shared memory would wait for it
        struct Operands {
            float4 q;
            float2 g;
            ulonglong2 B, C;
        };
        auto operands = [&](int t) {
            return Operands{mine[t * pair_row(PAIRS)], sg[t * PAIRS + pr], *reinterpret_cast<const ulonglong2 *>(gB + t * NP),
                            *reinterpret_cast<const ulonglong2 *>(gC + t * NP)};
        };
        Operands next = operands(kChunk - 1);
#pragma unroll
        for (int t = kChunk - 1; t >= 0; --t) {
            const Operands at_t = next;
            if (t > 0) next = operands(t - 1);
            const float4 q = at_t.q;
            const float2 gv = at_t.g;
            const f32x2 Bp[2] = {at_t.B.x, at_t.B.y}, Cp[2] = {at_t.C.x, at_t.C.y};
            const f32x2 uu[2] = {pk(q.x, q.x), pk(q.y, q.y)}, ux[2] = {pk(q.z, q.z), pk(q.w, q.w)};
            const f32x2 gg[2] = {pk(gv.x, gv.x), pk(gv.y, gv.y)};
            f32x2 vB[2], vC[2];
            float v[4];                                                // sums over n: dh B of both channels, A r of both
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                f32x2 a1, a2;
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    const f32x2 av = decay2(uu[c], A2[c][p]);
                    dh[c][p] = fma2(Cp[p], gg[c], dh[c][p]);
                    vB[p] = c ? fma2(dh[c][p], ux[c], vB[p]) : mul2(dh[c][p], ux[c]);
                    vC[p] = c ? fma2(gg[c], hh[t][c][p], vC[p]) : mul2(gg[c], hh[t][c][p]);
                    a1 = p ? fma2(dh[c][p], Bp[p], a1) : mul2(dh[c][p], Bp[p]);
                    dh[c][p] = mul2(dh[c][p], av);             // a dh: what reaches h_{t-1}
                    const f32x2 r = mul2(dh[c][p], t ? hh[t ? t - 1 : 0][c][p] : h0[c][p]);
                    a2 = p ? fma2(A2[c][p], r, a2) : mul2(A2[c][p], r);
                    dAt[c][p] = fma2(uu[c], r, dAt[c][p]);
                }
                v[c] = sum2(a1);
                v[2 + c] = sum2(a2);
            }
            // dB, dC over the warp's channels: states 0, 1 of the lane's order are kept, then
            // state 0, then one of dB and dC
            if constexpr (CL >= 2) {
                vB[0] = add2(vB[0], __shfl_xor_sync(0xffffffffu, vB[1], LN));
                vC[0] = add2(vC[0], __shfl_xor_sync(0xffffffffu, vC[1], LN));
            }
            float *to = sr + (warp * kChunk + t) * 2 * NP + ln * 4;
            float bl, bh, cl0, ch;
            unpk(vB[0], bl, bh);
            unpk(vC[0], cl0, ch);
            if constexpr (CL >= 4) {
                bl += __shfl_xor_sync(0xffffffffu, bh, 2 * LN);
                cl0 += __shfl_xor_sync(0xffffffffu, ch, 2 * LN);
            }
            if constexpr (CL >= 8) {
                const bool wc = cl & 4;
                float r = (wc ? cl0 : bl) + __shfl_xor_sync(0xffffffffu, wc ? bl : cl0, 4 * LN);
                if constexpr (CL >= 16) r += __shfl_xor_sync(0xffffffffu, r, 8 * LN);
                if (CL < 16 || !(cl & 8)) to[(wc ? NP : 0) + m] = r;
            } else if constexpr (CL == 4) {
                to[m] = bl;
                to[NP + m] = cl0;
            } else if constexpr (CL == 2) {
                *reinterpret_cast<float2 *>(to + m) = make_float2(bl, bh);
                *reinterpret_cast<float2 *>(to + NP + m) = make_float2(cl0, ch);
            } else {
                *reinterpret_cast<ulonglong2 *>(to) = make_ulonglong2(vB[0], vB[1]);
                *reinterpret_cast<ulonglong2 *>(to + NP) = make_ulonglong2(vC[0], vC[1]);
            }
            lane_reduce<4, NL, PARTS>(v, lane);
            float *part = reinterpret_cast<float *>(sp + (t * PARTS + ln % PARTS) * PR + pair_at(pr, PAIRS));
            if constexpr (NL == 1) *reinterpret_cast<float4 *>(part) = make_float4(v[0], v[1], v[2], v[3]);
            else if constexpr (NL == 2) *reinterpret_cast<float2 *>(part + reduced_first<4, NL, PARTS>(lane)) = make_float2(v[0], v[1]);
            else if (reduced_owner<4, NL, PARTS>(lane)) part[reduced_first<4, NL, PARTS>(lane)] = v[0];
        }
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int p = 0; p < 2; ++p) dA[c][p] = add2(dA[c][p], dAt[c][p]);
        __syncthreads();
        // rows of dx and ddelta, and the CTA's share of dB and dC
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int t = St::tok(i), c = St::chan();
            if (!full && (t0 + t >= t_stop || c >= cb.count)) continue;
            if (!St::EVEN && t >= kChunk) continue;
            float x[VEC], g[VEC], u[VEC], sig[VEC], s1[VEC], s2[VEC];
            St::get(raw, buf, 0, i, a, cb, b, t0, n, a.x, x);
            St::get(raw, buf, 2, i, a, cb, b, t0, n, a.dy, g);
            Pack<float, VEC> sv;
            sv.load(ss + t * CPB + c);
            sv.get(sig);
            const float4 *up = su + t * pair_row(PAIRS) + pair_at(c / 2, PAIRS), *part = sp + t * PARTS * PR + pair_at(c / 2, PAIRS);
            if constexpr (VEC == 4) {
                const float4 u0 = up[0], u1 = up[PAIRS / 2 + 4];       // an even pair and the odd one after it
                u[0] = u0.x; u[1] = u0.y; u[2] = u1.x; u[3] = u1.y;
                ulonglong2 p0 = {}, p1 = {};
#pragma unroll
                for (int q = 0; q < PARTS; ++q) {
                    const ulonglong2 q0 = *reinterpret_cast<const ulonglong2 *>(part + q * PR);
                    const ulonglong2 q1 = *reinterpret_cast<const ulonglong2 *>(part + q * PR + PAIRS / 2 + 4);
                    p0 = q ? make_ulonglong2(add2(p0.x, q0.x), add2(p0.y, q0.y)) : q0;
                    p1 = q ? make_ulonglong2(add2(p1.x, q1.x), add2(p1.y, q1.y)) : q1;
                }
                unpk(p0.x, s1[0], s1[1]);
                unpk(p0.y, s2[0], s2[1]);
                unpk(p1.x, s1[2], s1[3]);
                unpk(p1.y, s2[2], s2[3]);
            } else {
#pragma unroll
                for (int k = 0; k < VEC; ++k) {
                    u[k] = reinterpret_cast<const float *>(up)[(c + k) & 1];
                    s1[k] = s2[k] = 0.f;
#pragma unroll
                    for (int q = 0; q < PARTS; ++q) {
                        s1[k] += reinterpret_cast<const float *>(part + q * PR)[(c + k) & 1];
                        s2[k] += reinterpret_cast<const float *>(part + q * PR)[2 + ((c + k) & 1)];
                    }
                }
            }
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                const float f = s1[k];
                s1[k] = fmaf(u[k], f, skip[k] * g[k]);                 // dx
                s2[k] = fmaf(s2[k], kLn2, x[k] * f) * sig[k];          // ddelta
            }
            if (!full && t0 + t >= n) {
#pragma unroll
                for (int k = 0; k < VEC; ++k) s1[k] = s2[k] = 0.f;
            }
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                dbs[k] += s2[k];
                dDs[k] = fmaf(g[k], x[k], dDs[k]);                     // padding has arrived as 0
            }
            const size_t to = out + i * at.rows;
            typename St::Vec v;
            v.set(s1);
            v.store((T *)a.dx + to);
            v.set(s2);
            v.store((T *)a.ddelta + to);
        }
        out -= (size_t)kChunk * D;
        for (int e = tid; e < kChunk * 2 * NP / 4; e += kGradThreads) {
            const int t = e / (NP / 2), k = e % (NP / 2) * 4;
            if (!full && (t0 + t >= n || t0 + t >= t_stop)) continue;
            const float *p = sr + t * 2 * NP + k;
            ulonglong2 f = *reinterpret_cast<const ulonglong2 *>(p);
#pragma unroll
            for (int q = 1; q < kGradWarps; ++q) {
                const ulonglong2 g = *reinterpret_cast<const ulonglong2 *>(p + q * kChunk * 2 * NP);
                f = make_ulonglong2(add2(f.x, g.x), add2(f.y, g.y));
            }
            *reinterpret_cast<ulonglong2 *>(dbc + t * dbc_row + k) = f;
        }
        dbc -= kChunk * dbc_row;
    }
    // whole chunks of padding
    const int done = t_begin + chunks * kChunk;
    for (int64_t e = tid; e < (int64_t)max(t_stop - done, 0) * cb.count; e += kGradThreads) {
        const size_t at = ((size_t)b * a.T + done + e / cb.count) * D + cb.first + e % cb.count;
        ((T *)a.dx)[at] = from_f<T>(0.f);
        ((T *)a.ddelta)[at] = from_f<T>(0.f);
    }
    // one row of partials per (sequence, segment): dA [D][N], dD [D], dbias [D]
    float *row = ws + w.par + ((size_t)b * S + seg) * D * (N + 2);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        scatter(row, cb.first + c0 + c, c, dA[c]);
        if (seg == 0 && a.dS0) scatter(a.dS0, bd + c, c, dh[c]);
    }
    float *sums = reinterpret_cast<float *>(sp);                       // [threads][2 VEC]
    __syncthreads();                                                   // the last rows have been written
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
        sums[tid * 2 * VEC + k] = dDs[k];
        sums[tid * 2 * VEC + VEC + k] = dbs[k];
    }
    __syncthreads();
    for (int e = tid; e < 2 * CPB; e += kGradThreads) {
        const int which = e / CPB, c = e % CPB;
        float f = 0.f;
        for (int q = 0; q < kGradThreads / St::ROW; ++q) f += sums[(q * St::ROW + c / VEC) * 2 * VEC + which * VEC + c % VEC];
        if (c < cb.count) row[(size_t)D * N + which * D + cb.first + c] = f;
    }
}

// Launch 3: four neighbouring values of dB or dC of one (token, group): the sum over the group's
// channel blocks.
template <typename T> __global__ void __launch_bounds__(kSumThreads) groups_kernel(SsmArgs a, BwdWs w, const float *ws, int NP) {
    const int quads = NP / 2;                                          // of a row: dB [NP], dC [NP]
    const int64_t i = (int64_t)blockIdx.x * kSumThreads + threadIdx.x, rows = (int64_t)a.B * a.T * a.G;
    const int64_t row = i >> (31 - __clz(quads));                      // quads is a power of two
    const int k = (int)(i & (quads - 1)) * 4, which = k >= NP, nn = k - which * NP;
    if (row >= rows || nn >= a.N) return;
    bool real = true;
    if (a.lens) {
        const int64_t bt = row / a.G;
        const int b = (int)(bt / a.T);
        real = bt - (int64_t)b * a.T < seq_len(a.lens, b, a.T);
    }
    float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
    if (real) {
        const float *p = ws + w.dbc + (size_t)row * w.nb * 2 * NP + k;
#pragma unroll 8
        for (int q = 0; q < w.nb; ++q) {
            const float4 g = *reinterpret_cast<const float4 *>(p + (size_t)q * 2 * NP);
            f.x += g.x; f.y += g.y; f.z += g.z; f.w += g.w;
        }
    }
    T *to = (T *)(which ? a.dC : a.dB) + row * a.N + nn;
    const float e[4] = {f.x, f.y, f.z, f.w};
    if (a.N % 4 == 0) {
        Pack<T, 4> v;
        v.set(e);
        v.store(to);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (nn + j < a.N) to[j] = from_f<T>(e[j]);
    }
}

template <typename T, int LN, int VEC> cudaError_t run_grads(const SsmArgs &a, const BwdWs &w, cudaStream_t s) {
    constexpr int PAIRS = kGradThreads / LN, CPB = 2 * PAIRS, NP = 4 * LN;
    const size_t smem = Staging<T, kGradThreads, kChunk, CPB, NP, 3, VEC, kStages>::BYTES +
                        kChunk * (4 * pair_row(PAIRS) + 4 * sum_parts(LN) * part_row(LN) + 2 * PAIRS + CPB + kGradWarps * 2 * NP) * sizeof(float) +
                        8 * order_size(NP) * sizeof(float);
    const cudaError_t e = allow_smem(grads_kernel<T, LN, VEC>, smem);
    if (e != cudaSuccess) return e;
    const unsigned nblk = (unsigned)(a.B * channel_blocks(a.D, a.G, CPB));
    grads_kernel<T, LN, VEC><<<dim3(nblk, w.sp.S), kGradThreads, smem, s>>>(a, w, (float *)a.ws);
    return cudaGetLastError();
}
template <typename T, int LN> cudaError_t run_grads(const SsmArgs &a, const BwdWs &w, cudaStream_t s) {
    const int v = access_size<T>(a);
    if (v == 4) return run_grads<T, LN, 4>(a, w, s);
    if constexpr (sizeof(T) == 2)
        if (v == 2) return run_grads<T, LN, 2>(a, w, s);
    return run_grads<T, LN, 1>(a, w, s);
}

template <typename T> cudaError_t run_bwd(const SsmArgs &a, cudaStream_t s, int *nlaunch) {
    const BwdWs w = bwd_ws(a.B, a.T, a.D, a.G, a.N);
    float *ws = (float *)a.ws;
    cudaError_t e = cudaSuccess;
    if (a.T > 0 && a.B > 0) {
        const ScanWs sw{nullptr, ws + w.E, ws + w.U, ws + w.R, ws + w.chk, ws + w.ucum};
        e = w.sp.S > 1 ? run_scan<T, kSegCheckpoints>(a, w.sp, sw, s, nlaunch) : run_scan<T, kCheckpoints>(a, w.sp, sw, s, nlaunch);
        if (e != cudaSuccess) return e;
    }
    if (a.B > 0) {
        switch (grad_lanes(a.N)) {
            case 2: e = run_grads<T, 2>(a, w, s); break;
            case 4: e = run_grads<T, 4>(a, w, s); break;
            case 8: e = run_grads<T, 8>(a, w, s); break;
            case 16: e = run_grads<T, 16>(a, w, s); break;
            default: e = run_grads<T, 32>(a, w, s); break;
        }
        if (e != cudaSuccess) return e;
        *nlaunch += 1;
    }
    if (a.T > 0 && a.B > 0) {
        const int NP = padded_states(a.N);
        const int64_t items = (int64_t)a.B * a.T * a.G * (NP / 2);
        groups_kernel<T><<<(unsigned)((items + kSumThreads - 1) / kSumThreads), kSumThreads, 0, s>>>(a, w, ws, NP);
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        *nlaunch += 1;
    }
    return launch_sum_rows(ws + w.par, w.rows, (int64_t)a.D * (a.N + 2), a.dA, (int64_t)a.D * a.N, a.dD, a.D, a.ddelta_bias, s,
                           nlaunch);
}

}  // namespace

size_t ssm_bwd_workspace(int B, int T, int D, int G, int N) { return bwd_ws(B, T, D, G, N).total * sizeof(float); }

cudaError_t launch_ssm_bwd(const SsmArgs &a, int dtype, cudaStream_t s, int *nlaunch) {
    return dtype == kBF16 ? run_bwd<__nv_bfloat16>(a, s, nlaunch) : run_bwd<float>(a, s, nlaunch);
}

}  // namespace qd
