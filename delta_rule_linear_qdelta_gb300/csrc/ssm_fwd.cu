// Selective state space scan, forward over a sequence and one token in place.  The recurrence
// is in ssm_scan.cuh; this file cuts sequences into segments and has the one-token kernel.
//
// Few channels over many tokens leave SMs idle, so the tokens are then cut into S segments.  A
// first launch takes every segment but the last from a zero state (segment 0 from S0) to its
// end E_s and its sum of u, U_s; in the second, a segment folds the ends before it,
// h <- exp(A U_s) h + E_s, and runs as usual.  The first launch costs about 0.65 of the second.
#include "layer_common.cuh"
#include "ssm_scan.cuh"

namespace qd {
namespace {

using namespace ssm;

constexpr int kStepThreads = 256;

// One token: the state is read once and written once, everything else is small.  A thread
// takes states 4 i + 0..3, i = ln, ln + LN, .. of one channel (SPL of them; N no multiple of four: states
// ln, ln + LN, ..) for kSeqs sequences, so A is read once for all of them and their states are in
// flight together.  Bound by memory, read and write mixed: 512 x 2048 x 16, bf16, 31 us (4.5 TB/s).
// Single states are stored after the last load, which would otherwise wait for each store (fp32, 512 x 2048 x
// 15: 144 -> 52 us, with the loads in flight together); groups of four as they come (31 us; 33 at the end).
constexpr int kSeqs = 4;

template <typename T, int LN, int SPL, bool WIDE>
__global__ void __launch_bounds__(kStepThreads) step_kernel(SsmArgs a, int per_group) {
    constexpr int CPB = kStepThreads / LN, Q = SPL / 4;
    const unsigned nblk = (a.D + CPB - 1) / CPB;
    const int b0 = blockIdx.x / nblk * kSeqs;
    const int ln = threadIdx.x % LN, ch = threadIdx.x / LN, lane = threadIdx.x & 31;
    const int d = (int)(blockIdx.x % nblk) * CPB + ch, N = a.N;
    const bool live = d < a.D;
    const int seqs = live ? min(kSeqs, a.B - b0) : 0;
    // the channel's place in the first sequence, and from one sequence to the next
    const size_t to_tok = a.D, to_grp = (size_t)a.G * N, to_state = (size_t)a.D * N;
    const size_t tok = live ? b0 * to_tok + d : 0, grp = live ? b0 * to_grp + (size_t)(d / per_group) * N : 0;
    const T *xp = (const T *)a.x + tok, *dp = (const T *)a.delta + tok, *Bp = (const T *)a.Bm + grp, *Cp = (const T *)a.Cm + grp;
    float *S = a.S_final + tok * N;
    const float *A = a.A + (live ? (size_t)d * N : 0);
    const float bias = live && a.delta_bias ? a.delta_bias[d] : 0.f, skip = live && a.Dskip ? a.Dskip[d] : 0.f;

    ulonglong2 s[WIDE ? kSeqs : 1][Q];
    float sn[WIDE ? 1 : kSeqs][SPL];
    if constexpr (WIDE) {
#pragma unroll
        for (int j = 0; j < kSeqs; ++j)
#pragma unroll
            for (int i = 0; i < Q; ++i) {
                const int k = (i * LN + ln) * 4;
                if (j < seqs && k < N) s[j][i] = *reinterpret_cast<const ulonglong2 *>(S + j * to_state + k);
            }
    } else {
#pragma unroll
        for (int j = 0; j < kSeqs; ++j)
#pragma unroll
            for (int i = 0; i < SPL; ++i) {
                const int k = i * LN + ln;
                if (j < seqs && k < N) sn[j][i] = S[j * to_state + k];
            }
    }
    // a channel's lanes share out its sequences' inputs and hand them round
    constexpr int MINE = (kSeqs + LN - 1) / LN;
    float um[MINE + MINE % 2], xm[MINE], u[kSeqs], x[kSeqs], acc[kSeqs];
    um[MINE - 1 + MINE % 2] = 0.f;
#pragma unroll
    for (int i = 0; i < MINE; ++i) {
        const int j = i * LN + ln;
        xm[i] = j < seqs ? to_f(xp[j * to_tok]) : 0.f;
        um[i] = j < seqs ? to_f(dp[j * to_tok]) + bias : 0.f;
    }
    if (a.softplus) {
        float e0, e1;
#pragma unroll
        for (int i = 0; i < MINE; i += 2) softplus2(um[i], um[i + 1], e0, e1);
    }
#pragma unroll
    for (int j = 0; j < kSeqs; ++j) {
        x[j] = __shfl_sync(0xffffffffu, xm[j / LN], j % LN, LN);
        u[j] = __shfl_sync(0xffffffffu, um[j / LN], j % LN, LN);
        acc[j] = 0.f;
    }
    if constexpr (WIDE) {
#pragma unroll
        for (int i = 0; i < Q; ++i) {
            const int k = (i * LN + ln) * 4;
            if (k >= N || !live) continue;
            const ulonglong2 Av = *reinterpret_cast<const ulonglong2 *>(A + k);
            const f32x2 A2[2] = {mul2(Av.x, pk(kLog2e, kLog2e)), mul2(Av.y, pk(kLog2e, kLog2e))};
#pragma unroll
            for (int j = 0; j < kSeqs; ++j) {
                if (j >= seqs) continue;
                Pack<T, 4> Bv, Cv;
                f32x2 B[2], C[2];
                Bv.load(Bp + j * to_grp + k);
                Cv.load(Cp + j * to_grp + k);
                Bv.get2(B);
                Cv.get2(C);
                const f32x2 uu = pk(u[j], u[j]), ux = pk(u[j] * x[j], u[j] * x[j]);
                ulonglong2 &h = s[j][i];
                h.x = fma2(decay2(uu, A2[0]), h.x, mul2(ux, B[0]));
                h.y = fma2(decay2(uu, A2[1]), h.y, mul2(ux, B[1]));
                acc[j] += sum2(fma2(h.x, C[0], mul2(h.y, C[1])));
                *reinterpret_cast<ulonglong2 *>(S + j * to_state + k) = h;
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < SPL; ++i) {
            const int k = i * LN + ln;
            if (k >= N || !live) continue;
            const float A2 = A[k] * kLog2e;
#pragma unroll
            for (int j = 0; j < kSeqs; ++j) {
                if (j >= seqs) continue;
                float &h = sn[j][i];
                h = fmaf(decay(u[j], A2), h, u[j] * x[j] * to_f(Bp[j * to_grp + k]));
                acc[j] = fmaf(h, to_f(Cp[j * to_grp + k]), acc[j]);
            }
        }
#pragma unroll
        for (int j = 0; j < kSeqs; ++j)
#pragma unroll
            for (int i = 0; i < SPL; ++i) {
                const int k = i * LN + ln;
                if (j < seqs && k < N) S[j * to_state + k] = sn[j][i];
            }
    }
#pragma unroll
    for (int j = 0; j < kSeqs; ++j) acc[j] += ln == 0 ? skip * x[j] : 0.f;
    lane_reduce<kSeqs, LN, 1>(acc, lane);
    const int first = reduced_first<kSeqs, LN, 1>(lane);
    if (reduced_owner<kSeqs, LN, 1>(lane)) {
        T *y = (T *)a.y + tok;
#pragma unroll
        for (int i = 0; i < (kSeqs > LN ? kSeqs / LN : 1); ++i)
            if (first + i < seqs) y[(first + i) * to_tok] = from_f<T>(acc[i]);
    }
}

// Segments: none while every SM has a CTA (256 CTAs of 8 x 2048 tokens x 2048 channels, bf16: whole
// is 11 % faster than two or four segments); otherwise enough for four CTAs per SM (32 CTAs of
// 1 x 32768 x 2048: 490 us, 519 us at three).
Split fwd_split(int B, int T, int D, int G, int N) {
    return split_tokens(scan_ctas(B, D, G, N), T, kSMs, 4 * kSMs, 4 * kTile, kTile);
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
