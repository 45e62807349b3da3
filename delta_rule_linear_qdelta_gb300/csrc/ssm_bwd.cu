// Backward of the selective state space scan (ssm_fwd.cu has the forward's formulas).  With
// g = dy and the gradient dh_t of L with respect to h_t,
//
//   dh_t = C_t g_t + a_{t+1} dh_{t+1}   (+ dS_final at the last token),   r_t = dh_t a_t h_{t-1}
//   dx = u sum_n dh B + D g,  du = sum_n A r + x sum_n dh B,  ddelta = du softplus'
//   dA = sum_{b,t} u r,  dB = sum_d dh u x,  dC = sum_d g h,  dD = sum g x,  dS0 = a_1 dh_1
//
// Launches:
//  1. states: the forward recurrence again, which leaves the state entering every chunk of 16
//     tokens in the workspace (4 bytes per token and channel at N = 16).  Few channels over
//     many tokens: the tokens are cut into segments as in the forward; each starts from zero
//     and also leaves its end E, its sum of u and R, the gradient that its own tokens send to
//     the state entering it, R = sum_t (prod_{s<=t} a_s) C_t g_t.
//  2. gradients: a CTA walks its segment's chunks backwards.  Per chunk it recomputes the 16
//     states into registers from the checkpoint, then runs dh down the tokens.  Sums over n
//     join over the LN lanes of a channel; sums over channels (dB, dC) over the channels of a
//     warp by shuffles, over the CTA's warps through shared memory.
//  3. the sums over CTAs: dB, dC over the channel blocks, and dA, dD, d bias over sequences
//     and segments; in a fixed order, so results do not change from run to run.
// Bound by instruction issue: two exponentials and about 20 operations per (token, channel,
// state) in launch 2, one and 4 in launch 1.
#include "layer_common.cuh"
#include "ssm_tile.cuh"

namespace qd {
namespace {

using namespace ssm;

constexpr int kChunk = 16;            // tokens between checkpoints

// Everything in the workspace, in floats from its start.
struct BwdWs {
    Split sp;
    int nck, nb;                      // checkpoints a sequence; channel blocks a group
    int rows;                         // rows of dA/dD/dbias partials
    size_t chk, ucum, E, U, R, dbc, par, total;
};

__host__ __device__ constexpr int bwd_lanes(int N) { return padded_states(N) / 4; }

BwdWs bwd_ws(int B, int T, int D, int G, int N) {
    BwdWs w;
    const size_t NP = padded_states(N), bd = (size_t)B * D;
    const int CPB = kThreads / bwd_lanes(N);
    w.nb = channel_blocks(D, G, CPB) / G;
    w.sp = split_tokens((int64_t)B * G * w.nb, T, kSMs, 2 * kSMs, 2 * kTile);
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

__device__ __forceinline__ void put4(float *p, const float *v) { *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]); }
__device__ __forceinline__ void get4(const float *p, float *v) {
    const float4 f = *reinterpret_cast<const float4 *>(p);
    v[0] = f.x; v[1] = f.y; v[2] = f.z; v[3] = f.w;
}

// Launch 1.  Geometry as in the forward.
template <typename T, int LN, int SPL, bool WIDE, bool MULTI>
__global__ void __launch_bounds__(kThreads) states_kernel(SsmArgs a, BwdWs w, float *ws) {
    using G = Geo<T, LN, SPL, WIDE>;
    constexpr int CPB = G::CPB, NP = G::NP;
    extern __shared__ float smem[];
    float2 *su = reinterpret_cast<float2 *>(smem);                     // [kTile][CPB] (u, u x)
    float *sB = smem + 2 * kTile * CPB;                                // [kTile][NP]
    float *sC = sB + kTile * NP;                                       // [kTile][NP], MULTI
    float *sg = sC + kTile * NP;                                       // [kTile][CPB] dy, MULTI

    const int tid = threadIdx.x, ln = tid % LN, ch = tid / LN, seg = blockIdx.y;
    const int nblk = channel_blocks(a.D, a.G, CPB), b = blockIdx.x / nblk;
    const ChannelBlock cb(a, blockIdx.x % nblk, CPB);
    const int D = a.D, N = a.N, d = cb.first + ch;
    const bool live = ch < cb.count;
    const int n = seq_len(a.lens, b, a.T);
    const int t_begin = seg * w.sp.len, t_end = min(min(t_begin + w.sp.len, a.T), n);
    const size_t bd = (size_t)b * D + d, all = (size_t)a.B * D;

    float A2[SPL], h[SPL], P[SPL], R[SPL], U = 0.f;
#pragma unroll
    for (int i = 0; i < SPL; ++i) {
        const bool on = live && ln * SPL + i < N;
        A2[i] = on ? a.A[(size_t)d * N + ln * SPL + i] * kLog2e : 0.f;
        h[i] = on && seg == 0 && a.S0 ? a.S0[bd * N + ln * SPL + i] : 0.f;
        P[i] = 1.f;
        R[i] = 0.f;
    }
    typename G::Stage st;
    if (t_begin < t_end) st.load(a, cb, b, t_begin, n, MULTI);
    for (int t0 = t_begin; t0 < t_end; t0 += kTile) {
        st.store_tokens(a, cb, t0, n, su);
        st.store_groups(a, cb, b, t0, n, sB, sC, MULTI);
        if (MULTI) {
            for (int e = tid; e < kTile * G::ROW; e += kThreads) {
                const int t = e / G::ROW, c = e % G::ROW * G::VEC;
                typename G::Vec v;
                v.zero();
                if (t0 + t < n && c < cb.count) v.load((const T *)a.dy + ((size_t)b * a.T + t0 + t) * D + cb.first + c);
                float f[G::VEC];
                v.get(f);
#pragma unroll
                for (int k = 0; k < G::VEC; ++k) sg[t * CPB + c + k] = f[k];
            }
        }
        __syncthreads();
        if (t0 + kTile < t_end) st.load(a, cb, b, t0 + kTile, n, MULTI);
#pragma unroll 1
        for (int c0 = 0; c0 < kTile && t0 + c0 < t_end; c0 += kChunk) {
            const size_t ck = (size_t)((t0 + c0) / kChunk) * all + bd;
            if (live) {
#pragma unroll
                for (int i = 0; i < SPL; i += 4) put4(ws + w.chk + ck * NP + ln * SPL + i, h + i);
                if (MULTI && ln == 0) ws[w.ucum + ck] = U;
            }
#pragma unroll 4
            for (int t = c0; t < c0 + kChunk; ++t) {
                const float2 uu = su[t * CPB + ch];
                const float g = MULTI ? sg[t * CPB + ch] : 0.f;
                if (MULTI) U += uu.x;
#pragma unroll
                for (int i = 0; i < SPL; i += 4) {
                    float Bf[4], Cf[4];
                    get4(sB + t * NP + ln * SPL + i, Bf);
                    if (MULTI) get4(sC + t * NP + ln * SPL + i, Cf);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float av = exp2_fast(uu.x * A2[i + k]);
                        h[i + k] = fmaf(av, h[i + k], uu.y * Bf[k]);
                        if (MULTI) {
                            P[i + k] *= av;
                            R[i + k] = fmaf(P[i + k], g * Cf[k], R[i + k]);
                        }
                    }
                }
            }
        }
        __syncthreads();
    }
    if (MULTI && live) {
        const size_t at = seg * all + bd;
#pragma unroll
        for (int i = 0; i < SPL; i += 4) {
            put4(ws + w.E + at * NP + ln * SPL + i, h + i);
            put4(ws + w.R + at * NP + ln * SPL + i, R + i);
        }
        if (ln == 0) ws[w.U + at] = U;
    }
}

// Launch 2.  LN lanes by four states per channel.
template <typename T, int LN, bool WIDE>
__global__ void __launch_bounds__(kThreads) grads_kernel(SsmArgs a, BwdWs w, float *ws) {
    constexpr int CPB = kThreads / LN, NP = 4 * LN, CL = 32 / LN;      // CL channels a warp
    constexpr int VEC = WIDE ? 4 : 1, ROW = CPB / VEC, PER = (kChunk * ROW + kThreads - 1) / kThreads;
    constexpr int TB = LN < 4 ? LN : 4;                                // tokens whose sums over n join at once
    constexpr int OS = CPB + CL;                                       // row of the outputs, padded
    using Vec = Pack<T, VEC>;
    extern __shared__ float smem[];
    float4 *sp = reinterpret_cast<float4 *>(smem);                     // [kChunk][CPB] (u, x, g, softplus')
    float2 *so = reinterpret_cast<float2 *>(smem + 4 * kChunk * CPB);  // [kChunk][OS] (dx, ddelta)
    float *sB = smem + 4 * kChunk * CPB + 2 * kChunk * OS;             // [kChunk][NP]
    float *sC = sB + kChunk * NP;
    float *sr = sC + kChunk * NP;                                      // [8 warps][kChunk][2 NP] (dB, dC)

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, ln = tid % LN, ch = tid / LN, seg = blockIdx.y;
    const int nblk = channel_blocks(a.D, a.G, CPB), b = blockIdx.x / nblk, blk = blockIdx.x % nblk;
    const ChannelBlock cb(a, blk, CPB);
    const int D = a.D, N = a.N, d = cb.first + ch, S = w.sp.S;
    const bool live = ch < cb.count;
    const int n = seq_len(a.lens, b, a.T);
    const int t_begin = seg * w.sp.len, t_stop = min(t_begin + w.sp.len, a.T), t_end = min(t_stop, n);
    const size_t bd = (size_t)b * D + d, all = (size_t)a.B * D;
    const float Dsk = live && a.Dskip ? a.Dskip[d] : 0.f;

    float A2[4], dh[4], dA[4], hin[4];                                 // dh: what reaches the state from the right
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bool on = live && ln * 4 + i < N;
        A2[i] = on ? a.A[(size_t)d * N + ln * 4 + i] * kLog2e : 0.f;
        dh[i] = on && a.dS_final ? a.dS_final[bd * N + ln * 4 + i] : 0.f;
        dA[i] = hin[i] = 0.f;
    }
    float dDs = 0.f, dbs = 0.f;
    if (S > 1 && live) {
        for (int s = S - 1; s > seg; --s) {
            const float U = ws[w.U + s * all + bd];
            float r[4];
            get4(ws + w.R + (s * all + bd) * NP + ln * 4, r);
#pragma unroll
            for (int i = 0; i < 4; ++i) dh[i] = fmaf(exp2_fast(U * A2[i]), dh[i], r[i]);
        }
        for (int s = 0; s < seg; ++s) {
            const float U = ws[w.U + s * all + bd];
            float e[4];
            get4(ws + w.E + (s * all + bd) * NP + ln * 4, e);
#pragma unroll
            for (int i = 0; i < 4; ++i) hin[i] = fmaf(exp2_fast(U * A2[i]), hin[i], e[i]);
        }
    }

    Vec xr[PER], dr[PER], gr[PER];
    auto load = [&](int t0) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = tid + i * kThreads, t = e / ROW, c = e % ROW * VEC;
            xr[i].zero();
            dr[i].zero();
            gr[i].zero();
            if (t < kChunk && t0 + t < n && c < cb.count) {
                const size_t at = ((size_t)b * a.T + t0 + t) * D + cb.first + c;
                xr[i].load((const T *)a.x + at);
                dr[i].load((const T *)a.delta + at);
                gr[i].load((const T *)a.dy + at);
            }
        }
    };
    const int chunks = t_begin < t_end ? (t_end - t_begin + kChunk - 1) / kChunk : 0;
    if (chunks) load(t_begin + (chunks - 1) * kChunk);
    for (int c = chunks - 1; c >= 0; --c) {
        const int t0 = t_begin + c * kChunk;
        // stage the chunk
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = tid + i * kThreads, t = e / ROW, cc = e % ROW * VEC;
            if (t >= kChunk) break;
            float xf[VEC], df[VEC], gf[VEC];
            xr[i].get(xf);
            dr[i].get(df);
            gr[i].get(gf);
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                float u = 0.f, sig = 0.f;
                if (t0 + t < n && cc + k < cb.count) {
                    u = df[k] + (a.delta_bias ? a.delta_bias[cb.first + cc + k] : 0.f);
                    sig = 1.f;
                    if (a.softplus) u = softplus_grad_f(u, sig);
                }
                sp[t * CPB + cc + k] = make_float4(u, xf[k], gf[k], sig);
            }
        }
        for (int e = tid; e < 2 * kChunk * NP; e += kThreads) {
            const int which = e / (kChunk * NP), r = e % (kChunk * NP), t = r / NP, k = r % NP;
            float f = 0.f;
            if (t0 + t < n && k < N)
                f = to_f(((const T *)(which ? a.Cm : a.Bm))[(((size_t)b * a.T + t0 + t) * a.G + cb.group) * N + k]);
            sB[e] = f;
        }
        float h0[4] = {0.f, 0.f, 0.f, 0.f};
        if (live) {
            const size_t ck = (size_t)(t0 / kChunk) * all + bd;
            get4(ws + w.chk + ck * NP + ln * 4, h0);
            if (seg > 0) {
                const float U = ws[w.ucum + ck];
#pragma unroll
                for (int i = 0; i < 4; ++i) h0[i] = fmaf(exp2_fast(U * A2[i]), hin[i], h0[i]);
            }
        }
        __syncthreads();
        if (c > 0) load(t0 - kChunk);

        float hh[kChunk][4];
#pragma unroll
        for (int t = 0; t < kChunk; ++t) {
            const float4 q = sp[t * CPB + ch];
            float Bf[4];
            get4(sB + t * NP + ln * 4, Bf);
            const float ux = q.x * q.y;
#pragma unroll
            for (int i = 0; i < 4; ++i) hh[t][i] = fmaf(exp2_fast(q.x * A2[i]), t ? hh[t - 1][i] : h0[i], ux * Bf[i]);
        }
#pragma unroll
        for (int tb = kChunk - TB; tb >= 0; tb -= TB) {
            float s1[TB], s2[TB];
#pragma unroll
            for (int k = TB - 1; k >= 0; --k) {
                const int t = tb + k;
                const float4 q = sp[t * CPB + ch];
                float Bf[4], Cf[4], v[8];
                get4(sB + t * NP + ln * 4, Bf);
                get4(sC + t * NP + ln * 4, Cf);
                const float ux = q.x * q.y;
                s1[k] = s2[k] = 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float av = exp2_fast(q.x * A2[i]);
                    dh[i] = fmaf(Cf[i], q.z, dh[i]);
                    v[i] = dh[i] * ux;
                    v[4 + i] = q.z * hh[t][i];
                    s1[k] = fmaf(dh[i], Bf[i], s1[k]);
                    dh[i] *= av;                                       // a dh: what reaches h_{t-1}
                    const float r = dh[i] * (t ? hh[t > 0 ? t - 1 : 0][i] : h0[i]);
                    s2[k] = fmaf(A2[i], r, s2[k]);
                    dA[i] = fmaf(q.x, r, dA[i]);
                }
                lane_reduce<8, CL, LN>(v, lane);
                if (reduced_owner<8, CL, LN>(lane)) {
                    constexpr int KEPT = 8 / CL > 1 ? 8 / CL : 1;
                    const int first = reduced_first<8, CL, LN>(lane);
#pragma unroll
                    for (int j = 0; j < KEPT; ++j) {
                        const int idx = first + j;
                        sr[(warp * kChunk + t) * 2 * NP + (idx >> 2) * NP + ln * 4 + (idx & 3)] = v[j];
                    }
                }
            }
            lane_reduce<TB, LN, 1>(s1, lane);
            lane_reduce<TB, LN, 1>(s2, lane);
            if (reduced_owner<TB, LN, 1>(lane)) {
                const int t = tb + reduced_first<TB, LN, 1>(lane);
                const float4 q = sp[t * CPB + ch];
                const float dd = fmaf(s2[0], kLn2, q.y * s1[0]) * q.w;
                so[t * OS + ch] = make_float2(fmaf(q.x, s1[0], Dsk * q.z), dd);
                dbs += dd;
                dDs = fmaf(q.z, q.y, dDs);
            }
        }
        __syncthreads();
        // rows of dx and ddelta, and the CTA's share of dB and dC
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = tid + i * kThreads, t = e / ROW, cc = e % ROW * VEC;
            if (t >= kChunk || t0 + t >= t_stop || cc >= cb.count) continue;
            float fx[VEC], fd[VEC];
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                const float2 o = so[t * OS + cc + k];
                fx[k] = t0 + t < n ? o.x : 0.f;
                fd[k] = t0 + t < n ? o.y : 0.f;
            }
            const size_t at = ((size_t)b * a.T + t0 + t) * D + cb.first + cc;
            Vec v;
            v.set(fx);
            v.store((T *)a.dx + at);
            v.set(fd);
            v.store((T *)a.ddelta + at);
        }
        for (int e = tid; e < kChunk * 2 * NP; e += kThreads) {
            const int t = e / (2 * NP), k = e % (2 * NP);
            if (t0 + t >= n) continue;
            float f = 0.f;
#pragma unroll
            for (int q = 0; q < kThreads / 32; ++q) f += sr[(q * kChunk + t) * 2 * NP + k];
            ws[w.dbc + ((((size_t)b * a.T + t0 + t) * a.G + cb.group) * w.nb + blk % w.nb) * 2 * NP + k] = f;
        }
    }
    // padding after the sequence's end
    for (int t0 = t_begin + chunks * kChunk; t0 < t_stop; ++t0) {
        for (int c = tid; c < cb.count; c += kThreads) {
            const size_t at = ((size_t)b * a.T + t0) * D + cb.first + c;
            ((T *)a.dx)[at] = from_f<T>(0.f);
            ((T *)a.ddelta)[at] = from_f<T>(0.f);
        }
    }
    // one row of partials per (sequence, segment): dA [D][N], dD [D], dbias [D]
    float one[2] = {dDs, dbs};
    lane_reduce<1, LN, 1>(one, lane);
    lane_reduce<1, LN, 1>(one + 1, lane);
    if (live) {
        float *row = ws + w.par + ((size_t)b * S + seg) * D * (N + 2);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (ln * 4 + i < N) {
                row[(size_t)d * N + ln * 4 + i] = dA[i];
                if (seg == 0 && a.dS0) a.dS0[bd * N + ln * 4 + i] = dh[i];
            }
        }
        if (ln == 0) {
            row[(size_t)D * N + d] = one[0];
            row[(size_t)D * N + D + d] = one[1];
        }
    }
}

// Launch 3: dB, dC of one (token, group, which, n): the sum over the group's channel blocks.
template <typename T> __global__ void __launch_bounds__(kThreads) groups_kernel(SsmArgs a, BwdWs w, const float *ws, int NP) {
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x, rows = (int64_t)a.B * a.T * a.G;
    const int64_t row = i / (2 * NP);
    const int k = (int)(i % (2 * NP)), which = k / NP, nn = k % NP;
    if (row >= rows || nn >= a.N) return;
    const int64_t bt = row / a.G;
    const int b = (int)(bt / a.T), t = (int)(bt % a.T);
    float f = 0.f;
    if (t < seq_len(a.lens, b, a.T)) {
        const float *p = ws + w.dbc + (size_t)row * w.nb * 2 * NP + k;
#pragma unroll 4
        for (int q = 0; q < w.nb; ++q) f += p[(size_t)q * 2 * NP];
    }
    ((T *)(which ? a.dC : a.dB))[row * a.N + nn] = from_f<T>(f);
}

template <typename K> cudaError_t allow_smem(K kernel, size_t bytes) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

template <typename T, int LN, int SPL, bool WIDE> cudaError_t run_states(const SsmArgs &a, const BwdWs &w, cudaStream_t s) {
    using G = Geo<T, LN, SPL, WIDE>;
    const unsigned nblk = (unsigned)(a.B * channel_blocks(a.D, a.G, G::CPB));
    const size_t base = (2 * kTile * G::CPB + kTile * G::NP) * sizeof(float);
    const size_t more = (kTile * G::NP + kTile * G::CPB) * sizeof(float);
    if (w.sp.S > 1) {
        cudaError_t e = allow_smem(states_kernel<T, LN, SPL, WIDE, true>, base + more);
        if (e != cudaSuccess) return e;
        states_kernel<T, LN, SPL, WIDE, true><<<dim3(nblk, w.sp.S), kThreads, base + more, s>>>(a, w, (float *)a.ws);
    } else {
        cudaError_t e = allow_smem(states_kernel<T, LN, SPL, WIDE, false>, base);
        if (e != cudaSuccess) return e;
        states_kernel<T, LN, SPL, WIDE, false><<<dim3(nblk, 1), kThreads, base, s>>>(a, w, (float *)a.ws);
    }
    return cudaGetLastError();
}

template <typename T, int LN, bool WIDE> cudaError_t run_grads(const SsmArgs &a, const BwdWs &w, cudaStream_t s) {
    constexpr int CPB = kThreads / LN, NP = 4 * LN;
    const size_t smem = (4 * kChunk * CPB + 2 * kChunk * (CPB + 32 / LN) + 2 * kChunk * NP + 8 * kChunk * 2 * NP) * sizeof(float);
    const cudaError_t e = allow_smem(grads_kernel<T, LN, WIDE>, smem);
    if (e != cudaSuccess) return e;
    const unsigned nblk = (unsigned)(a.B * channel_blocks(a.D, a.G, CPB));
    grads_kernel<T, LN, WIDE><<<dim3(nblk, w.sp.S), kThreads, smem, s>>>(a, w, (float *)a.ws);
    return cudaGetLastError();
}

template <typename T, int LN, int SPL, int LNB> cudaError_t run_bwd(const SsmArgs &a, cudaStream_t s, int *nlaunch) {
    const BwdWs w = bwd_ws(a.B, a.T, a.D, a.G, a.N);
    constexpr int V = 16 / (int)sizeof(T);
    const int per = a.D / a.G;
    cudaError_t e = cudaSuccess;
    if (a.T > 0 && a.B > 0) {
        e = per % V == 0 && a.N % V == 0 ? run_states<T, LN, SPL, true>(a, w, s) : run_states<T, LN, SPL, false>(a, w, s);
        if (e != cudaSuccess) return e;
        *nlaunch += 1;
    }
    if (a.B > 0) {
        e = per % 4 == 0 ? run_grads<T, LNB, true>(a, w, s) : run_grads<T, LNB, false>(a, w, s);
        if (e != cudaSuccess) return e;
        *nlaunch += 1;
    }
    if (a.T > 0 && a.B > 0) {
        const int NP = padded_states(a.N);
        const int64_t items = (int64_t)a.B * a.T * a.G * 2 * NP;
        groups_kernel<T><<<(unsigned)((items + kThreads - 1) / kThreads), kThreads, 0, s>>>(a, w, (const float *)a.ws, NP);
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        *nlaunch += 1;
    }
    return launch_sum_rows((const float *)a.ws + w.par, w.rows, (int64_t)a.D * (a.N + 2), a.dA, (int64_t)a.D * a.N, a.dD, a.D,
                           a.ddelta_bias, s, nlaunch);
}

}  // namespace

size_t ssm_bwd_workspace(int B, int T, int D, int G, int N) { return bwd_ws(B, T, D, G, N).total * sizeof(float); }

cudaError_t launch_ssm_bwd(const SsmArgs &a, int dtype, cudaStream_t s, int *nlaunch) {
    if (a.N <= 8) return dtype == kBF16 ? run_bwd<__nv_bfloat16, 2, 4, 2>(a, s, nlaunch) : run_bwd<float, 2, 4, 2>(a, s, nlaunch);
    if (a.N <= 16) return dtype == kBF16 ? run_bwd<__nv_bfloat16, 4, 4, 4>(a, s, nlaunch) : run_bwd<float, 4, 4, 4>(a, s, nlaunch);
    if (a.N <= 32) return dtype == kBF16 ? run_bwd<__nv_bfloat16, 4, 8, 8>(a, s, nlaunch) : run_bwd<float, 4, 8, 8>(a, s, nlaunch);
    if (a.N <= 64) return dtype == kBF16 ? run_bwd<__nv_bfloat16, 8, 8, 16>(a, s, nlaunch) : run_bwd<float, 8, 8, 16>(a, s, nlaunch);
    return dtype == kBF16 ? run_bwd<__nv_bfloat16, 8, 16, 32>(a, s, nlaunch) : run_bwd<float, 8, 16, 32>(a, s, nlaunch);
}

}  // namespace qd
