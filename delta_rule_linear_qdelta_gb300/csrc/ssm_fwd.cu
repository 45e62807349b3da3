// Selective state space scan, forward over a sequence and one token in place.  The recurrence
// is in ssm_scan.cuh; this file cuts sequences into segments and has the one-token kernel.
//
// Few channels over many tokens leave SMs idle, so the tokens are then cut into S segments.  A
// first launch takes every segment but the last from a zero state (segment 0 from S0) to its
// end E_s and its sum of u, U_s; in the second, a segment folds the ends before it,
// h <- exp(A U_s) h + E_s, and runs as usual.  The first launch costs about 0.6 of the second.
#include "layer_common.cuh"
#include "ssm_scan.cuh"

namespace qd {
namespace {

using namespace ssm;

constexpr int kStepThreads = 256;

// One token: the state is read once and written once, everything else is small.  A thread
// takes four states of a channel (one at a time when N is no multiple of four).
template <typename T, int LN, int SPL>
__global__ void __launch_bounds__(kStepThreads) step_kernel(SsmArgs a, int per_group) {
    constexpr int CPB = kStepThreads / LN;
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
        if (a.softplus) {
            float none = 0.f, e0, e1;
            softplus2(u, none, e0, e1);
        }
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

// Segments: none while every SM has a CTA (256 CTAs of 8 x 2048 tokens x 2048 channels: 275 us
// whole, 293 and 316 us in four and two segments, bf16); otherwise enough for four CTAs per SM
// (32 CTAs of 1 x 32768 x 2048: 578 us, 633 us at three).
Split fwd_split(int B, int T, int D, int G, int N) {
    return split_tokens(scan_ctas(B, D, G, N), T, kSMs, 4 * kSMs, 4 * kTile);
}

template <typename T> cudaError_t run_fwd(const SsmArgs &a, cudaStream_t s, int *nlaunch) {
    const Split sp = fwd_split(a.B, a.T, a.D, a.G, a.N);
    const size_t all = (size_t)a.B * a.D, states = all * padded_states(a.N);
    ScanWs w{};
    if (sp.S > 1) {
        w.start = (float *)a.ws;
        w.E = w.start + states;
        w.U = w.E + (sp.S - 1) * states;
        const cudaError_t e = run_scan<T, kEnds>(a, sp, w, s, nlaunch);
        if (e != cudaSuccess) return e;
    }
    return run_scan<T, kOutputs>(a, sp, w, s, nlaunch);
}

template <typename T, int LN, int SPL> cudaError_t run_step(const SsmArgs &a, cudaStream_t s, int *nlaunch) {
    const int64_t blocks = (int64_t)a.B * ((a.D + kStepThreads / LN - 1) / (kStepThreads / LN));
    step_kernel<T, LN, SPL><<<(unsigned)blocks, kStepThreads, 0, s>>>(a, a.D / a.G);
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) *nlaunch += 1;
    return e;
}
template <typename T> cudaError_t run_step(const SsmArgs &a, cudaStream_t s, int *nlaunch) {
    if (a.N <= 8) return run_step<T, 2, 4>(a, s, nlaunch);
    if (a.N <= 16) return run_step<T, 4, 4>(a, s, nlaunch);
    if (a.N <= 32) return run_step<T, 4, 8>(a, s, nlaunch);
    if (a.N <= 64) return run_step<T, 8, 8>(a, s, nlaunch);
    return run_step<T, 8, 16>(a, s, nlaunch);
}

}  // namespace

size_t ssm_fwd_workspace(int B, int T, int D, int G, int N) {
    const Split sp = fwd_split(B, T, D, G, N);
    const size_t all = (size_t)B * D;
    return sp.S == 1 ? 0 : (sp.S * all * padded_states(N) + (sp.S - 1) * all) * sizeof(float);
}

cudaError_t launch_ssm_fwd(const SsmArgs &a, int dtype, cudaStream_t s, int *nlaunch) {
    return dtype == kBF16 ? run_fwd<__nv_bfloat16>(a, s, nlaunch) : run_fwd<float>(a, s, nlaunch);
}

cudaError_t launch_ssm_step(const SsmArgs &a, int dtype, cudaStream_t s, int *nlaunch) {
    return dtype == kBF16 ? run_step<__nv_bfloat16>(a, s, nlaunch) : run_step<float>(a, s, nlaunch);
}

}  // namespace qd
