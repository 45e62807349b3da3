// Shared by the operators around the token mixers (short convolution, selective scan,
// group norm): packed loads and stores, elementwise maps, lane reductions and the
// fixed-order sum of per-CTA partial results.
#pragma once

#include "qd_internal.cuh"

namespace qd {

constexpr int kSMs = 152;

// VEC consecutive elements as one access of VEC * sizeof(T) bytes (2 .. 16).
template <int BYTES> struct Bits;
template <> struct Bits<2> { using T = unsigned short; };
template <> struct Bits<4> { using T = unsigned; };
template <> struct Bits<8> { using T = uint2; };
template <> struct Bits<16> { using T = uint4; };

template <typename T, int VEC> struct Pack {
    typename Bits<sizeof(T) * VEC>::T bits;
    __device__ __forceinline__ void zero() { bits = {}; }
    __device__ __forceinline__ void load(const T *p) {
        bits = *reinterpret_cast<const typename Bits<sizeof(T) * VEC>::T *>(p);
    }
    __device__ __forceinline__ void store(T *p) const {
        *reinterpret_cast<typename Bits<sizeof(T) * VEC>::T *>(p) = bits;
    }
    __device__ __forceinline__ void get(float (&f)[VEC]) const {
        const T *e = reinterpret_cast<const T *>(&bits);
#pragma unroll
        for (int i = 0; i < VEC; ++i) f[i] = to_f(e[i]);
    }
    __device__ __forceinline__ void set(const float (&f)[VEC]) {
        T *e = reinterpret_cast<T *>(&bits);
#pragma unroll
        for (int i = 0; i < VEC; ++i) e[i] = from_f<T>(f[i]);
    }
};

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// sigmoid(x) = 1 / (1 + e^-x) with the approximate division (2 ulp), which returns 0 for a
// divisor above 2^126: x < -87, where the sigmoid is below the normal range of fp32.
__device__ __forceinline__ float sigmoid_f(float x) { return __fdividef(1.f, 1.f + exp2_fast(-x * kLog2e)); }

// d/dx SiLU(x), given s = sigmoid(x).
__device__ __forceinline__ float silu_grad(float x, float s) { return s * fmaf(x, 1.f - s, 1.f); }

// softplus(x) = max(x, 0) + log(1 + e), e = e^-|x| in (0, 1], and its derivative
// sigmoid(x) = (x >= 0 ? 1 : e) / (1 + e).  log(1 + e) = 2 atanh(s), s = e / (2 + e) <= 1/3,
// by atanh's own series 2 s (1 + s^2/3 + s^4/5 + ...): the first term left out is below
// 1.4e-8 of the sum, and nothing cancels, so small results keep their relative precision.
__device__ __forceinline__ float log1p_unit(float e) {
    const float s = __fdividef(e, 2.f + e), q = s * s;
    float p = 1.f / 13.f;
    p = fmaf(p, q, 1.f / 11.f);
    p = fmaf(p, q, 1.f / 9.f);
    p = fmaf(p, q, 1.f / 7.f);
    p = fmaf(p, q, 1.f / 5.f);
    p = fmaf(p, q, 1.f / 3.f);
    p = fmaf(p, q, 1.f);
    return 2.f * s * p;
}
__device__ __forceinline__ float softplus_f(float x) {
    const float e = exp2_fast(-fabsf(x) * kLog2e);
    return fmaxf(x, 0.f) + log1p_unit(e);
}
__device__ __forceinline__ float softplus_grad_f(float x, float &sig) {
    const float e = exp2_fast(-fabsf(x) * kLog2e);
    sig = __fdividef(x >= 0.f ? 1.f : e, 1.f + e);
    return fmaxf(x, 0.f) + log1p_unit(e);
}

// Sum each of CNT values (a power of two) over the NL lanes that differ in the lane bits
// STRIDE, 2 STRIDE, .., STRIDE NL / 2.  While a lane still holds several values it gives
// half of them away and keeps the sums of the other half, so CNT values over NL lanes cost
// CNT - 1 shuffles (CNT <= NL) in place of CNT log2(NL).  Afterwards v[0 .. max(1, CNT/NL))
// of a lane are the sums of the values from reduced_first<>(lane) on; reduced_owner<> picks
// one lane where several hold the same value.
template <int CNT, int NL, int STRIDE> __device__ __forceinline__ void lane_reduce(float *v, int lane) {
    if constexpr (NL > 1) {
        constexpr int BIT = STRIDE * NL / 2;
        if constexpr (CNT > 1) {
            const bool up = lane & BIT;
#pragma unroll
            for (int i = 0; i < CNT / 2; ++i) {
                const float keep = up ? v[i + CNT / 2] : v[i];
                const float give = up ? v[i] : v[i + CNT / 2];
                v[i] = keep + __shfl_xor_sync(0xffffffffu, give, BIT);
            }
            lane_reduce<CNT / 2, NL / 2, STRIDE>(v, lane);
        } else {
            v[0] += __shfl_xor_sync(0xffffffffu, v[0], BIT);
            lane_reduce<1, NL / 2, STRIDE>(v, lane);
        }
    }
}
template <int CNT, int NL, int STRIDE> __device__ __forceinline__ int reduced_first(int lane) {
    if constexpr (NL > 1 && CNT > 1)
        return ((lane & (STRIDE * NL / 2)) ? CNT / 2 : 0) + reduced_first<CNT / 2, NL / 2, STRIDE>(lane);
    else
        return 0;
}
template <int CNT, int NL, int STRIDE> __device__ __forceinline__ bool reduced_owner(int lane) {
    if constexpr (NL > 1 && CNT > 1) return reduced_owner<CNT / 2, NL / 2, STRIDE>(lane);
    else return (lane & (STRIDE * (NL - 1))) == 0;
}

// out[m] = sum over p < P of part[p][m], m < M, in a fixed order (the same inputs give the
// same bits).  Columns m < M1 go to out1, the next M2 to out2, the rest to out3; a NULL
// output drops its columns.
cudaError_t launch_sum_rows(const float *part, int P, int64_t M, float *out1, int64_t M1, float *out2, int64_t M2,
                            float *out3, cudaStream_t s, int *nlaunch);

}  // namespace qd
