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
// takes states 4 i + 0..3, i = ln, ln + LN, .. of one channel (SPL of them; N no multiple of four: one by
// one) for kSeqs sequences, so A is read once for all of them and their states are in
// flight together.
constexpr int kSeqs = 4;

template <typename T, int LN, int SPL, bool WIDE>
__global__ void __launch_bounds__(kStepThreads) step_kernel(SsmArgs a, int per_group) {
    constexpr int CPB = kStepThreads / LN, Q = SPL / 4;
    const int64_t nblk = (a.D + CPB - 1) / CPB;
    const int64_t b0 = blockIdx.x / nblk * kSeqs;
    const int ln = threadIdx.x % LN, ch = threadIdx.x / LN, lane = threadIdx.x & 31;
    const int d = (int)(blockIdx.x % nblk) * CPB + ch, N = a.N;
    const bool live = d < a.D;
    const int seqs = live ? (int)min((int64_t)kSeqs, a.B - b0) : 0;
    const int grp = live ? d / per_group : 0;
    const float bias = live && a.delta_bias ? a.delta_bias[d] : 0.f, skip = live && a.Dskip ? a.Dskip[d] : 0.f;
    float u[kSeqs], x[kSeqs], acc[kSeqs];
    float4 s[WIDE ? kSeqs : 1][Q];
    if constexpr (WIDE) {
#pragma unroll
        for (int j = 0; j < kSeqs; ++j)
#pragma unroll
            for (int i = 0; i < Q; ++i) {
                const int k = (i * LN + ln) * 4;
                if (j < seqs && k < N) s[j][i] = *reinterpret_cast<const float4 *>(a.S_final + ((b0 + j) * a.D + d) * N + k);
            }
    }
#pragma unroll
    for (int j = 0; j < kSeqs; ++j) {
        const size_t bd = (b0 + (j < seqs ? j : 0)) * a.D + (live ? d : 0);
        x[j] = to_f(((const T *)a.x)[bd]);
        u[j] = to_f(((const T *)a.delta)[bd]) + bias;
        acc[j] = 0.f;
    }
    if (a.softplus) {
        float e0, e1;
#pragma unroll
        for (int j = 0; j < kSeqs; j += 2) softplus2(u[j], u[j + 1], e0, e1);
    }
    if constexpr (WIDE) {
#pragma unroll
        for (int i = 0; i < Q; ++i) {
            const int k = (i * LN + ln) * 4;
            if (k >= N || !live) continue;
            float4 A = *reinterpret_cast<const float4 *>(a.A + (size_t)d * N + k);
            A.x *= kLog2e; A.y *= kLog2e; A.z *= kLog2e; A.w *= kLog2e;
#pragma unroll
            for (int j = 0; j < kSeqs; ++j) {
                if (j >= seqs) continue;
                const size_t at = ((b0 + j) * a.G + grp) * N + k;
                Pack<T, 4> Bv, Cv;
                float B[4], C[4];
                Bv.load((const T *)a.Bm + at);
                Cv.load((const T *)a.Cm + at);
                Bv.get(B);
                Cv.get(C);
                const float ux = u[j] * x[j];
                float4 &h = s[j][i];
                h.x = fmaf(exp2_fast(u[j] * A.x), h.x, ux * B[0]);
                h.y = fmaf(exp2_fast(u[j] * A.y), h.y, ux * B[1]);
                h.z = fmaf(exp2_fast(u[j] * A.z), h.z, ux * B[2]);
                h.w = fmaf(exp2_fast(u[j] * A.w), h.w, ux * B[3]);
                acc[j] += h.x * C[0] + h.y * C[1] + h.z * C[2] + h.w * C[3];
                *reinterpret_cast<float4 *>(a.S_final + ((b0 + j) * a.D + d) * N + k) = h;
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < kSeqs; ++j) {
            if (j >= seqs) continue;
            const T *Bp = (const T *)a.Bm + ((b0 + j) * a.G + grp) * N, *Cp = (const T *)a.Cm + ((b0 + j) * a.G + grp) * N;
            float *S = a.S_final + ((b0 + j) * a.D + d) * N;
            for (int k = ln; k < N; k += LN) {
                const float h = fmaf(exp2_fast(u[j] * (a.A[(size_t)d * N + k] * kLog2e)), S[k], u[j] * x[j] * to_f(Bp[k]));
                acc[j] = fmaf(h, to_f(Cp[k]), acc[j]);
                S[k] = h;
            }
        }
    }
#pragma unroll
    for (int j = 0; j < kSeqs; ++j) {
        lane_reduce<1, LN, 1>(acc + j, lane);
        if (j < seqs && ln == 0) ((T *)a.y)[(b0 + j) * a.D + d] = from_f<T>(fmaf(skip, x[j], acc[j]));
    }
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
    const int64_t blocks = ((int64_t)a.B + kSeqs - 1) / kSeqs * ((a.D + kStepThreads / LN - 1) / (kStepThreads / LN));
    if (a.N % 4 == 0) step_kernel<T, LN, SPL, true><<<(unsigned)blocks, kStepThreads, 0, s>>>(a, a.D / a.G);
    else step_kernel<T, LN, SPL, false><<<(unsigned)blocks, kStepThreads, 0, s>>>(a, a.D / a.G);
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
