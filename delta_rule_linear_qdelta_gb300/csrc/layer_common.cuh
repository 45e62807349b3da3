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
    // the elements as (VEC + 1) / 2 pairs; a single element's other half is 0
    __device__ __forceinline__ void get2(unsigned long long (&f)[(VEC + 1) / 2]) const {
        float e[VEC + 1];
        float(&g)[VEC] = *reinterpret_cast<float(*)[VEC]>(e);
        get(g);
        e[VEC] = 0.f;
#pragma unroll
        for (int i = 0; i < (VEC + 1) / 2; ++i)
            asm("mov.b64 %0, {%1, %2};" : "=l"(f[i]) : "f"(e[2 * i]), "f"(e[2 * i + 1]));
    }
    __device__ __forceinline__ void set2(const unsigned long long (&f)[(VEC + 1) / 2]) {
        float e[VEC + 1];
#pragma unroll
        for (int i = 0; i < (VEC + 1) / 2; ++i)
            asm("mov.b64 {%0, %1}, %2;" : "=f"(e[2 * i]), "=f"(e[2 * i + 1]) : "l"(f[i]));
        const float(&g)[VEC] = *reinterpret_cast<const float(*)[VEC]>(e);
        set(g);
    }
    __device__ __forceinline__ void set(const float (&f)[VEC]) {
        T *e = reinterpret_cast<T *>(&bits);
        if constexpr (sizeof(T) == 2 && VEC % 2 == 0) {   // two at once: one conversion instruction
#pragma unroll
            for (int i = 0; i < VEC; i += 2)
                reinterpret_cast<__nv_bfloat162 *>(e)[i / 2] = __floats2bfloat162_rn(f[i], f[i + 1]);
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i) e[i] = from_f<T>(f[i]);
        }
    }
};

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float rcp_fast(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two fp32 numbers in one 64-bit register and the packed instructions on them, which issue
// once for both.
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pk(float lo, float hi) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpk(f32x2 v, float &lo, float &hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 exp2_2(f32x2 x) {
    float a, b;
    unpk(x, a, b);
    return pk(exp2_fast(a), exp2_fast(b));
}
// The decay exp(u A) of two states, A2 = A log2(e).  Over -3e-3 .. 0, where a state remembers
// hundreds of tokens and errors of one sign add up, the hardware's exponential is low by 6e-9
// on average (measured; its spread is 3e-8); the shift of the argument, free in the fused
// multiply-add, brings that to 1e-9.  At u = 0 the decay is exactly 1.
constexpr float kDecayShift = 1e-8f;
__device__ __forceinline__ f32x2 decay2(f32x2 u, f32x2 A2) { return exp2_2(fma2(u, A2, pk(kDecayShift, kDecayShift))); }
__device__ __forceinline__ float decay(float u, float A2) { return exp2_fast(fmaf(u, A2, kDecayShift)); }
// exp(U A) v + e of two states, U a sum of step sizes.  CAREFUL: U A may be large and positive; exp(U A) can
// then overflow where the product does not, v being small or exactly 0, so it is taken in two halves,
// kept finite, one before v and one after.
template <bool CAREFUL> __device__ __forceinline__ f32x2 carry2(f32x2 U, f32x2 A2, f32x2 v, f32x2 e) {
    if constexpr (!CAREFUL) return fma2(decay2(U, A2), v, e);
    float a, b;
    unpk(fma2(mul2(U, pk(0.5f, 0.5f)), A2, pk(kDecayShift, kDecayShift)), a, b);
    asm("min.NaN.f32 %0, %0, %1;" : "+f"(a) : "f"(127.f));             // 2^127 twice times the smallest normal number overflows
    asm("min.NaN.f32 %0, %0, %1;" : "+f"(b) : "f"(127.f));
    const f32x2 half = pk(exp2_fast(a), exp2_fast(b));
    return fma2(half, mul2(half, v), e);
}
__device__ __forceinline__ float sum2(f32x2 v) {
    float a, b;
    unpk(v, a, b);
    return a + b;
}

// sigmoid(x) = 1 / (1 + e^-x) of two numbers; 0 where e^-x overflows.
__device__ __forceinline__ f32x2 sigmoid2(f32x2 x) {
    const f32x2 d = add2(exp2_2(mul2(x, pk(-kLog2e, -kLog2e))), pk(1.f, 1.f));
    float a, b;
    unpk(d, a, b);
    return pk(rcp_fast(a), rcp_fast(b));
}
// d/dx SiLU(x) = s + x s (1 - s), given s = sigmoid(x).
__device__ __forceinline__ f32x2 silu_grad2(f32x2 x, f32x2 s) { return fma2(mul2(x, s), fma2(s, pk(-1.f, -1.f), pk(1.f, 1.f)), s); }

// softplus(x) = max(x, 0) + log(1 + e), e = e^-|x| in (0, 1], of two numbers.  log(1 + e) = e P(e)
// with P the ninth-degree polynomial of least relative error on [0, 1] (5e-9, from an
// iterated weighted least-squares fit); evaluated in fp32 it is within 1.4e-7, and a small
// result keeps its relative precision.  e is returned for the derivative.
__device__ __forceinline__ void softplus2(float &x, float &y, float &ex, float &ey) {
    ex = exp2_fast(-fabsf(x) * kLog2e);
    ey = exp2_fast(-fabsf(y) * kLog2e);
    const f32x2 e = pk(ex, ey);
    auto both = [](float c) { return pk(c, c); };
    f32x2 p = both(-0.0032440212f);
    p = fma2(p, e, both(0.019851444f));
    p = fma2(p, e, both(-0.0569595f));
    p = fma2(p, e, both(0.10603651f));
    p = fma2(p, e, both(-0.1530559f));
    p = fma2(p, e, both(0.19675939f));
    p = fma2(p, e, both(-0.24954134f));
    p = fma2(p, e, both(0.33329964f));
    p = fma2(p, e, both(-0.499999f));
    p = fma2(p, e, both(1.f));
    float a, b;
    unpk(mul2(p, e), a, b);
    x = fmaxf(x, 0.f) + a;
    y = fmaxf(y, 0.f) + b;
}
// sigmoid(x), the derivative of softplus, from e = e^-|x|: nothing cancels on either side.
__device__ __forceinline__ float softplus_grad(float x, float e) { return (x >= 0.f ? 1.f : e) * rcp_fast(1.f + e); }

// Asynchronous copy of BYTES to shared memory, or zeros where there is nothing to copy.
template <int BYTES> __device__ __forceinline__ void copy_async(void *dst, const void *src, bool on) {
    const unsigned to = (unsigned)__cvta_generic_to_shared(dst);
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(to), "l"(src), "n"(BYTES), "r"(on ? BYTES : 0) : "memory");
}
template <int BYTES> __device__ __forceinline__ void copy_async(void *dst, const void *src) {
    const unsigned to = (unsigned)__cvta_generic_to_shared(dst);
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to), "l"(src), "n"(BYTES) : "memory");
}
__device__ __forceinline__ void copies_issued() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT> __device__ __forceinline__ void copies_done() { asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory"); }

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
