// Selective state space scan, forward over a sequence and one token in place.  Per channel
// d with its group's B, C and n = 0 .. N-1:
//
//   u_t = softplus(delta_t + bias) (or the sum itself),  a = exp(u_t A[d][n])
//   h_t[n] = a h_{t-1}[n] + u_t x_t B_t[n],   y_t = sum_n C_t[n] h_t[n] + D x_t
//
// Each (token, channel, state) costs one exponential and six operations and no state ever
// leaves the chip, so a sequence is bound by instruction issue, not by memory.
//
// Layout: LN lanes share a channel and hold SPL = NP / LN of its states each in registers
// (NP: N rounded up to 8, 16, 32, 64 or 128); a CTA of 256 threads is CPB = 256 / LN channels
// of one sequence and walks the tokens in tiles of 32.  A tile's u, u x, B and C are staged
// in shared memory as fp32 (softplus is thus taken once per token and channel), the next
// tile's loads are in flight meanwhile, and y goes back through shared memory so that rows
// are written as they are read.  The sum over n is split over the LN lanes and joined for LN
// tokens at a time, LN - 1 shuffles in all.
//
// Few channels over many tokens: the tokens are cut into S segments.  A first launch takes
// every segment but the last from a zero state (segment 0 from S0) to its end state and its
// sum of u; in the second launch a segment folds the ends before it, h <- exp(A U_s) h + E_s,
// and then runs as usual.
#include "layer_common.cuh"
#include "ssm_tile.cuh"

namespace qd {
namespace {

using namespace ssm;

// Workspace of the segmented scan: E [S][B][D][NP] (slot 0: S0; slot s + 1: the end of
// segment s), then U [S][B][D].
template <typename T, int LN, int SPL, bool WIDE, bool STATES>
__global__ void __launch_bounds__(kThreads) scan_kernel(SsmArgs a, Split sp, float *wsE, float *wsU) {
    using G = Geo<T, LN, SPL, WIDE>;
    constexpr int CPB = G::CPB, NP = G::NP;
    extern __shared__ float smem[];
    float2 *su = reinterpret_cast<float2 *>(smem);                     // [TT][CPB] (u, u x)
    float *sB = smem + 2 * kTile * CPB;                                // [TT][NP]
    float *sC = sB + kTile * NP;                                       // [TT][NP]
    float *sy = sC + (STATES ? 0 : kTile * NP);                        // [TT][CPB + 32 / LN]
    constexpr int YS = CPB + 32 / LN;

    const int tid = threadIdx.x, lane = tid & 31, ln = tid % LN, ch = tid / LN;
    const int nblk = channel_blocks(a.D, a.G, CPB), b = blockIdx.x / nblk, seg = blockIdx.y;
    const ChannelBlock cb(a, blockIdx.x % nblk, CPB);
    const int D = a.D, N = a.N;
    const int d = cb.first + ch;
    const bool live = ch < cb.count;
    const int n = seq_len(a.lens, b, a.T);
    const int t_begin = seg * sp.len, t_end = min(t_begin + sp.len, a.T);
    const size_t state = ((size_t)b * D + d) * N + ln * SPL;

    float A2[SPL], h[SPL];                                             // A log2(e)
#pragma unroll
    for (int i = 0; i < SPL; ++i) {
        const bool on = live && ln * SPL + i < N;
        A2[i] = on ? a.A[(size_t)d * N + ln * SPL + i] * kLog2e : 0.f;
        h[i] = on && seg == 0 && a.S0 && (STATES || sp.S == 1) ? a.S0[state + i] : 0.f;
    }
    const size_t slot = ((size_t)b * D + d) * NP + ln * SPL, slots = (size_t)a.B * D * NP;
    if (STATES && seg == 0 && live) {
#pragma unroll
        for (int i = 0; i < SPL; i += 4) *reinterpret_cast<float4 *>(wsE + slot + i) = make_float4(h[i], h[i + 1], h[i + 2], h[i + 3]);
    }
    if (!STATES && sp.S > 1 && live) {
        const int from = seg == 0 ? 0 : 1;
#pragma unroll
        for (int i = 0; i < SPL; i += 4) {
            const float4 e = *reinterpret_cast<const float4 *>(wsE + from * slots + slot + i);
            h[i] = e.x; h[i + 1] = e.y; h[i + 2] = e.z; h[i + 3] = e.w;
        }
        for (int s = 1; s < seg; ++s) {
            const float U = wsU[((size_t)s * a.B + b) * D + d];
#pragma unroll
            for (int i = 0; i < SPL; i += 4) {
                const float4 e = *reinterpret_cast<const float4 *>(wsE + (s + 1) * slots + slot + i);
                h[i] = fmaf(exp2_fast(U * A2[i]), h[i], e.x);
                h[i + 1] = fmaf(exp2_fast(U * A2[i + 1]), h[i + 1], e.y);
                h[i + 2] = fmaf(exp2_fast(U * A2[i + 2]), h[i + 2], e.z);
                h[i + 3] = fmaf(exp2_fast(U * A2[i + 3]), h[i + 3], e.w);
            }
        }
    }

    float U = 0.f;
    typename G::Stage st;
    if (t_begin < min(t_end, n)) st.load(a, cb, b, t_begin, n, !STATES);
    for (int t0 = t_begin; t0 < t_end; t0 += kTile) {
        const bool any = t0 < n;                                       // uniform over the CTA
        if (!any && STATES) break;
        typename G::Vec xk[G::PER];
        if (any) {
            st.store_tokens(a, cb, t0, n, su);
            st.store_groups(a, cb, b, t0, n, sB, sC, !STATES);
#pragma unroll
            for (int i = 0; i < G::PER; ++i) xk[i] = st.x[i];
            __syncthreads();
            if (t0 + kTile < min(t_end, n)) st.load(a, cb, b, t0 + kTile, n, !STATES);
#pragma unroll 2
            for (int t = 0; t < kTile; t += LN) {
                float yv[LN];
#pragma unroll
                for (int k = 0; k < LN; ++k) {
                    const float2 uu = su[(t + k) * CPB + ch];
                    const float *Bt = sB + (t + k) * NP + ln * SPL, *Ct = sC + (t + k) * NP + ln * SPL;
                    float acc = 0.f;
                    if (STATES) U += uu.x;
#pragma unroll
                    for (int i = 0; i < SPL; i += 4) {
                        const float4 Bv = *reinterpret_cast<const float4 *>(Bt + i);
                        h[i] = fmaf(exp2_fast(uu.x * A2[i]), h[i], uu.y * Bv.x);
                        h[i + 1] = fmaf(exp2_fast(uu.x * A2[i + 1]), h[i + 1], uu.y * Bv.y);
                        h[i + 2] = fmaf(exp2_fast(uu.x * A2[i + 2]), h[i + 2], uu.y * Bv.z);
                        h[i + 3] = fmaf(exp2_fast(uu.x * A2[i + 3]), h[i + 3], uu.y * Bv.w);
                        if (!STATES) {
                            const float4 Cv = *reinterpret_cast<const float4 *>(Ct + i);
                            acc = fmaf(Cv.x, h[i], acc);
                            acc = fmaf(Cv.y, h[i + 1], acc);
                            acc = fmaf(Cv.z, h[i + 2], acc);
                            acc = fmaf(Cv.w, h[i + 3], acc);
                        }
                    }
                    yv[k] = acc;
                }
                if (!STATES) {
                    lane_reduce<LN, LN, 1>(yv, lane);
                    sy[(t + reduced_first<LN, LN, 1>(lane)) * YS + ch] = yv[0];
                }
            }
            __syncthreads();
        }
        if (!STATES) G::write_y(a, cb, b, t0, t_end, n, any, xk, sy, YS);
    }
    if (live) {
        if (STATES) {
#pragma unroll
            for (int i = 0; i < SPL; i += 4)
                *reinterpret_cast<float4 *>(wsE + (seg + 1) * slots + slot + i) = make_float4(h[i], h[i + 1], h[i + 2], h[i + 3]);
            if (ln == 0) wsU[((size_t)seg * a.B + b) * D + d] = U;
        } else if (a.S_final && seg == sp.S - 1) {
#pragma unroll
            for (int i = 0; i < SPL; ++i)
                if (ln * SPL + i < N) a.S_final[state + i] = h[i];
        }
    }
}

// One token: the state is read once and written once, everything else is small.  A thread
// takes four states of a channel (one at a time when N is no multiple of four).
template <typename T, int LN, int SPL>
__global__ void __launch_bounds__(kThreads) step_kernel(SsmArgs a, int per_group) {
    constexpr int CPB = kThreads / LN;
    const int64_t nblk = (a.D + CPB - 1) / CPB;
    const size_t b = blockIdx.x / nblk;
    const int ln = threadIdx.x % LN, ch = threadIdx.x / LN, lane = threadIdx.x & 31;
    const int d = (int)(blockIdx.x % nblk) * CPB + ch, N = a.N;
    const bool live = d < a.D;
    float acc = 0.f, x = 0.f;
    if (live) {
        const size_t bd = b * a.D + d;
        x = to_f(((const T *)a.x)[bd]);
        float u = to_f(((const T *)a.delta)[bd]) + (a.delta_bias ? a.delta_bias[d] : 0.f);
        if (a.softplus) u = softplus_f(u);
        const float ux = u * x;
        const size_t grp = (b * a.G + d / per_group) * N;
        const T *Bp = (const T *)a.Bm + grp, *Cp = (const T *)a.Cm + grp;
        float *S = a.S_final + bd * N;
        const float *A = a.A + (size_t)d * N;
        if (N % 4 == 0) {
            float4 s[SPL / 4];
#pragma unroll
            for (int i = 0; i < SPL / 4; ++i) {
                const int k = (i * LN + ln) * 4;
                if (k < N) s[i] = *reinterpret_cast<const float4 *>(S + k);
            }
#pragma unroll
            for (int i = 0; i < SPL / 4; ++i) {
                const int k = (i * LN + ln) * 4;
                if (k < N) {
                    const float4 Av = *reinterpret_cast<const float4 *>(A + k);
                    Pack<T, 4> Bv, Cv;
                    float Bf[4], Cf[4];
                    Bv.load(Bp + k);
                    Cv.load(Cp + k);
                    Bv.get(Bf);
                    Cv.get(Cf);
                    s[i].x = fmaf(exp2_fast(u * (Av.x * kLog2e)), s[i].x, ux * Bf[0]);
                    s[i].y = fmaf(exp2_fast(u * (Av.y * kLog2e)), s[i].y, ux * Bf[1]);
                    s[i].z = fmaf(exp2_fast(u * (Av.z * kLog2e)), s[i].z, ux * Bf[2]);
                    s[i].w = fmaf(exp2_fast(u * (Av.w * kLog2e)), s[i].w, ux * Bf[3]);
                    acc += s[i].x * Cf[0] + s[i].y * Cf[1] + s[i].z * Cf[2] + s[i].w * Cf[3];
                    *reinterpret_cast<float4 *>(S + k) = s[i];
                }
            }
        } else {
            for (int k = ln; k < N; k += LN) {
                const float s = fmaf(exp2_fast(u * (A[k] * kLog2e)), S[k], ux * to_f(Bp[k]));
                acc = fmaf(s, to_f(Cp[k]), acc);
                S[k] = s;
            }
        }
    }
    lane_reduce<1, LN, 1>(&acc, lane);
    if (live && ln == 0) ((T *)a.y)[b * a.D + d] = from_f<T>(acc + (a.Dskip ? a.Dskip[d] * x : 0.f));
}

// Segments: none while every SM has a CTA; otherwise enough for about four CTAs per SM, of
// at least four tiles each.
Split fwd_split(int B, int T, int D, int G, int N) {
    const int64_t ctas = (int64_t)B * channel_blocks(D, G, kThreads / lanes_for(N));
    return split_tokens(ctas, T, kSMs, 4 * kSMs, 4 * kTile);
}

template <typename T, int LN, int SPL, bool WIDE> cudaError_t run_scan(const SsmArgs &a, cudaStream_t s, int *nlaunch) {
    using G = Geo<T, LN, SPL, WIDE>;
    const Split sp = fwd_split(a.B, a.T, a.D, a.G, a.N);
    const unsigned nblk = (unsigned)(a.B * channel_blocks(a.D, a.G, G::CPB));
    float *wsE = (float *)a.ws, *wsU = wsE + (size_t)sp.S * a.B * a.D * G::NP;
    if (sp.S > 1) {
        const size_t smem = (2 * kTile * G::CPB + kTile * G::NP) * sizeof(float);
        scan_kernel<T, LN, SPL, WIDE, true><<<dim3(nblk, sp.S - 1), kThreads, smem, s>>>(a, sp, wsE, wsU);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        *nlaunch += 1;
    }
    const size_t smem = (2 * kTile * G::CPB + 2 * kTile * G::NP + kTile * (G::CPB + 32 / LN)) * sizeof(float);
    cudaError_t e = cudaFuncSetAttribute(scan_kernel<T, LN, SPL, WIDE, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    scan_kernel<T, LN, SPL, WIDE, false><<<dim3(nblk, sp.S), kThreads, smem, s>>>(a, sp, wsE, wsU);
    e = cudaGetLastError();
    if (e == cudaSuccess) *nlaunch += 1;
    return e;
}

template <typename T, int LN, int SPL> cudaError_t run_scan(const SsmArgs &a, cudaStream_t s, int *nlaunch) {
    // whole 16-byte accesses along the channels of a group and along the states
    constexpr int V = 16 / (int)sizeof(T);
    const bool wide = (a.D / a.G) % V == 0 && a.N % V == 0;
    return wide ? run_scan<T, LN, SPL, true>(a, s, nlaunch) : run_scan<T, LN, SPL, false>(a, s, nlaunch);
}

template <typename T, int LN, int SPL> cudaError_t run_step(const SsmArgs &a, cudaStream_t s, int *nlaunch) {
    const int64_t blocks = (int64_t)a.B * ((a.D + kThreads / LN - 1) / (kThreads / LN));
    step_kernel<T, LN, SPL><<<(unsigned)blocks, kThreads, 0, s>>>(a, a.D / a.G);
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) *nlaunch += 1;
    return e;
}

}  // namespace

size_t ssm_fwd_workspace(int B, int T, int D, int G, int N) {
    const Split sp = fwd_split(B, T, D, G, N);
    return sp.S == 1 ? 0 : (size_t)sp.S * B * D * (padded_states(N) + 1) * sizeof(float);
}

#define QD_SSM_N(call)                                                         \
    if (a.N <= 8) return dtype == kBF16 ? call(__nv_bfloat16, 2, 4) : call(float, 2, 4);   \
    if (a.N <= 16) return dtype == kBF16 ? call(__nv_bfloat16, 4, 4) : call(float, 4, 4);  \
    if (a.N <= 32) return dtype == kBF16 ? call(__nv_bfloat16, 4, 8) : call(float, 4, 8);  \
    if (a.N <= 64) return dtype == kBF16 ? call(__nv_bfloat16, 8, 8) : call(float, 8, 8);  \
    return dtype == kBF16 ? call(__nv_bfloat16, 8, 16) : call(float, 8, 16);

cudaError_t launch_ssm_fwd(const SsmArgs &a, int dtype, cudaStream_t s, int *nlaunch) {
#define QD_SSM_CALL(T, LN, SPL) run_scan<T, LN, SPL>(a, s, nlaunch)
    QD_SSM_N(QD_SSM_CALL)
#undef QD_SSM_CALL
}

cudaError_t launch_ssm_step(const SsmArgs &a, int dtype, cudaStream_t s, int *nlaunch) {
#define QD_SSM_CALL(T, LN, SPL) run_step<T, LN, SPL>(a, s, nlaunch)
    QD_SSM_N(QD_SSM_CALL)
#undef QD_SSM_CALL
}

}  // namespace qd
