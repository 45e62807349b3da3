// Group norm of each token's channels with an activation or a gate, and its backward.
// A token's row is H groups of d channels; per group
//   xh = (x - mean) rstd (center) or x rstd,  rstd = 1 / sqrt(mean of squares + eps)
//   n  = xh w + b,   y = act(n), or n act(z) with a gate z
// Backward, with dn the gradient of n and g = dn w:
//   dx = rstd (g - mean(g) [center] - xh mean(g xh)),  dw = sum dn xh,  db = sum dn
//
// Bound by memory.  A group stays in registers from its load to its store (VEC channels a
// lane in 16-byte accesses, K of them): the mean, then the mean of the squared differences
// from it, so no precision is lost where the mean is large.  A thread keeps its channels
// from token to token, so weights are read once per thread and dw, db add up in registers.
#include "layer_common.cuh"

namespace qd {
namespace {

constexpr int kNormThreads = 256;

// How a CTA's threads cover the groups: LPG threads to a group (a power of two up to 32, or
// the whole CTA), HB groups of one token side by side, MB tokens at once.
struct NormPlan {
    int lpg, HB, MB, nhb, gm;
};

__device__ __forceinline__ float group_total(float v, int lpg, float *sm) {
    if (lpg <= 32) {
        for (int o = lpg / 2; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        return v;
    }
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();                                   // the last total has been read by all
    if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
    __syncthreads();
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < kNormThreads / 32; ++i) t += sm[i];
    return t;
}

template <int VEC> __device__ __forceinline__ void load_param(const float *p, float (&f)[VEC]) {
    if constexpr (VEC >= 4) {
#pragma unroll
        for (int i = 0; i < VEC / 4; ++i) {
            const float4 v = reinterpret_cast<const float4 *>(p)[i];
            f[4 * i] = v.x; f[4 * i + 1] = v.y; f[4 * i + 2] = v.z; f[4 * i + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) f[i] = p[i];
    }
}

// xh of the thread's channels of one group, and the group's rstd.
template <int VEC, int K>
__device__ __forceinline__ float normalise(float (&v)[K][VEC], const bool (&on)[K], int d, int center, float eps, int lpg,
                                           float *sm) {
    const float inv_d = 1.f / (float)d;
    if (center) {
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int c = 0; c < VEC; ++c) s += v[k][c];
        const float mean = group_total(s, lpg, sm) * inv_d;
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int c = 0; c < VEC; ++c) v[k][c] = on[k] ? v[k][c] - mean : 0.f;
    }
    float q = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int c = 0; c < VEC; ++c) q = fmaf(v[k][c], v[k][c], q);
    const float rstd = 1.f / sqrtf(group_total(q, lpg, sm) * inv_d + eps);
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int c = 0; c < VEC; ++c) v[k][c] *= rstd;
    return rstd;
}

// The thread's place: group h (or none), first token, and its K channel offsets.
template <int VEC, int K> struct Place {
    int h, ml, hl;
    bool live, on[K];
    int c[K];
    __device__ __forceinline__ Place(const NormArgs &a, const NormPlan &p) {
        const int slot = threadIdx.x / p.lpg, l = threadIdx.x % p.lpg;
        hl = slot % p.HB;
        ml = slot / p.HB;
        h = (blockIdx.x % p.nhb) * p.HB + hl;
        live = ml < p.MB && h < a.H;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            c[k] = (l + k * p.lpg) * VEC;
            on[k] = live && c[k] < a.d;
        }
    }
};

template <typename T, int VEC, int K>
__global__ void __launch_bounds__(kNormThreads) norm_fwd_kernel(NormArgs a, NormPlan p) {
    __shared__ float sm[kNormThreads / 32];
    const Place<VEC, K> at(a, p);
    float w[K][VEC], b[K][VEC];
#pragma unroll
    for (int k = 0; k < K; ++k) {
#pragma unroll
        for (int c = 0; c < VEC; ++c) {
            w[k][c] = 1.f;
            b[k][c] = 0.f;
        }
        if (at.on[k]) {
            if (a.w) load_param<VEC>(a.w + (size_t)at.h * a.d + at.c[k], w[k]);
            if (a.b) load_param<VEC>(a.b + (size_t)at.h * a.d + at.c[k], b[k]);
        }
    }
    const int64_t first = (int64_t)(blockIdx.x / p.nhb) * p.MB, turn = (int64_t)p.gm * p.MB;
    Pack<T, VEC> x[K], z[K], xn[K], zn[K];
    auto fetch = [&](int64_t m) {
        const size_t row = ((size_t)m * a.H + at.h) * a.d;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            xn[k].zero();
            zn[k].zero();
            if (at.on[k] && m < a.M) {
                xn[k].load((const T *)a.x + row + at.c[k]);
                if (a.z) zn[k].load((const T *)a.z + row + at.c[k]);
            }
        }
    };
    fetch(first + at.ml);
    // every thread of the CTA makes the same number of turns: the group totals synchronise
    for (int64_t m0 = first; m0 < a.M; m0 += turn) {
        const int64_t m = m0 + at.ml;
        const size_t row = ((size_t)m * a.H + at.h) * a.d;
        float v[K][VEC];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            x[k] = xn[k];
            z[k] = zn[k];
            x[k].get(v[k]);
        }
        fetch(m + turn);                               // the next token's, while this one is computed
        normalise<VEC, K>(v, at.on, a.d, a.center, a.eps, p.lpg, sm);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float g[VEC];
            z[k].get(g);
#pragma unroll
            for (int c = 0; c < VEC; ++c) {
                const float n = fmaf(v[k][c], w[k][c], b[k][c]);
                const float t = a.z ? g[c] : n;
                const float act = a.silu ? t * sigmoid_f(t) : t;
                v[k][c] = a.z ? n * act : act;
            }
            if (at.on[k] && m < a.M) {
                x[k].set(v[k]);
                x[k].store((T *)a.y + row + at.c[k]);
            }
        }
    }
}

template <typename T, int VEC, int K>
__global__ void __launch_bounds__(kNormThreads) norm_bwd_kernel(NormArgs a, NormPlan p) {
    __shared__ float sm[kNormThreads / 32];
    extern __shared__ float sp[];
    const Place<VEC, K> at(a, p);
    float w[K][VEC], b[K][VEC], dw[K][VEC], db[K][VEC];
#pragma unroll
    for (int k = 0; k < K; ++k) {
#pragma unroll
        for (int c = 0; c < VEC; ++c) {
            w[k][c] = 1.f;
            b[k][c] = dw[k][c] = db[k][c] = 0.f;
        }
        if (at.on[k]) {
            if (a.w) load_param<VEC>(a.w + (size_t)at.h * a.d + at.c[k], w[k]);
            if (a.b) load_param<VEC>(a.b + (size_t)at.h * a.d + at.c[k], b[k]);
        }
    }
    const float inv_d = 1.f / (float)a.d;
    const int64_t begin = (int64_t)(blockIdx.x / p.nhb) * p.MB, turn = (int64_t)p.gm * p.MB;
    Pack<T, VEC> x[K], z[K], dy[K], xn[K], zn[K], dyn[K];
    auto fetch = [&](int64_t m) {
        const size_t row = ((size_t)m * a.H + at.h) * a.d;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            xn[k].zero();
            zn[k].zero();
            dyn[k].zero();
            if (at.on[k] && m < a.M) {
                xn[k].load((const T *)a.x + row + at.c[k]);
                dyn[k].load((const T *)a.dy + row + at.c[k]);
                if (a.z) zn[k].load((const T *)a.z + row + at.c[k]);
            }
        }
    };
    fetch(begin + at.ml);
    for (int64_t m0 = begin; m0 < a.M; m0 += turn) {
        const int64_t m = m0 + at.ml;
        const size_t row = ((size_t)m * a.H + at.h) * a.d;
        float v[K][VEC];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            x[k] = xn[k];
            z[k] = zn[k];
            dy[k] = dyn[k];
            x[k].get(v[k]);
        }
        fetch(m + turn);
        const float rstd = normalise<VEC, K>(v, at.on, a.d, a.center, a.eps, p.lpg, sm);
        float s1 = 0.f, s2 = 0.f, g[K][VEC];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float gate[VEC], dz[VEC];
            dy[k].get(g[k]);
            z[k].get(gate);
#pragma unroll
            for (int c = 0; c < VEC; ++c) {
                const float n = fmaf(v[k][c], w[k][c], b[k][c]);
                const float t = a.z ? gate[c] : n;
                const float s = a.silu ? sigmoid_f(t) : 1.f;
                const float slope = a.silu ? silu_grad(t, s) : 1.f;
                float dn;
                if (a.z) {
                    dz[c] = g[k][c] * n * slope;
                    dn = g[k][c] * (a.silu ? t * s : t);
                } else {
                    dn = g[k][c] * slope;
                }
                dw[k][c] = fmaf(dn, v[k][c], dw[k][c]);
                db[k][c] += dn;
                g[k][c] = dn * w[k][c];
                s1 += g[k][c];
                s2 = fmaf(g[k][c], v[k][c], s2);
            }
            if (a.z && at.on[k] && m < a.M) {
                z[k].set(dz);
                z[k].store((T *)a.dz + row + at.c[k]);
            }
        }
        s1 = a.center ? group_total(s1, p.lpg, sm) * inv_d : 0.f;
        s2 = group_total(s2, p.lpg, sm) * inv_d;
#pragma unroll
        for (int k = 0; k < K; ++k) {
#pragma unroll
            for (int c = 0; c < VEC; ++c) g[k][c] = rstd * (g[k][c] - s1 - v[k][c] * s2);
            if (at.on[k] && m < a.M) {
                x[k].set(g[k]);
                x[k].store((T *)a.dx + row + at.c[k]);
            }
        }
    }
    if (!a.part) return;
    // join the CTA's MB tokens and leave one row of partials: dw [H][d], db [H][d]
    const size_t HD = (size_t)a.H * a.d;
    float *part = a.part + (size_t)(blockIdx.x / p.nhb) * 2 * HD;
    const int width = p.HB * p.lpg * VEC * K;          // one token's channels in the CTA
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        float(&acc)[K][VEC] = which ? db : dw;
        if (p.MB > 1) {
            __syncthreads();
            if (at.live && at.ml > 0)
#pragma unroll
                for (int k = 0; k < K; ++k)
#pragma unroll
                    for (int c = 0; c < VEC; ++c)
                        sp[(size_t)(at.ml - 1) * width + (k * VEC + c) * p.HB * p.lpg + threadIdx.x % (p.HB * p.lpg)] = acc[k][c];
            __syncthreads();
            if (at.live && at.ml == 0)
#pragma unroll
                for (int k = 0; k < K; ++k)
#pragma unroll
                    for (int c = 0; c < VEC; ++c)
                        for (int q = 0; q + 1 < p.MB; ++q)
                            acc[k][c] += sp[(size_t)q * width + (k * VEC + c) * p.HB * p.lpg + threadIdx.x];
        }
        if (at.ml == 0) {
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (at.on[k])
#pragma unroll
                    for (int c = 0; c < VEC; ++c) part[which * HD + (size_t)at.h * a.d + at.c[k] + c] = acc[k][c];
        }
    }
}

struct NormShape {
    int vec, K;
    NormPlan p;
};
// The group's accesses are shared out over the fewest lanes of a warp that take it one
// access each (or four, on a whole warp), and over a whole CTA beyond that.  The grid holds
// about eight CTAs per SM, which then walk the tokens.
NormShape norm_shape(int M, int H, int d, int dtype, int ctas_per_sm) {
    NormShape s;
    const int wide = dtype == kBF16 ? 8 : 4;
    s.vec = d % wide == 0 ? wide : 1;
    const int nv = d / s.vec;
    if (nv <= 32) {
        s.p.lpg = 1;
        while (s.p.lpg < nv) s.p.lpg *= 2;
        s.K = 1;
    } else if (nv <= 128) {
        s.p.lpg = 32;
        s.K = nv <= 64 ? 2 : 4;
    } else {
        s.p.lpg = kNormThreads;
        s.K = nv <= kNormThreads ? 1 : nv <= 4 * kNormThreads ? 4 : nv <= 8 * kNormThreads ? 8 : 32;
    }
    const int slots = kNormThreads / s.p.lpg;
    s.p.HB = H < slots ? H : slots;
    s.p.MB = slots / s.p.HB;
    s.p.nhb = (H + s.p.HB - 1) / s.p.HB;
    const int64_t most = ((int64_t)M + s.p.MB - 1) / s.p.MB;
    int64_t gm = ((int64_t)ctas_per_sm * kSMs + s.p.nhb - 1) / s.p.nhb;
    if (gm > most) gm = most;
    s.p.gm = (int)gm;
    return s;
}

template <typename T, int VEC, int K> void run_fwd(const NormArgs &a, const NormPlan &p, cudaStream_t s) {
    norm_fwd_kernel<T, VEC, K><<<(unsigned)(p.gm * p.nhb), kNormThreads, 0, s>>>(a, p);
}
template <typename T, int VEC, int K> void run_bwd(const NormArgs &a, const NormPlan &p, cudaStream_t s) {
    const size_t smem = (size_t)(p.MB - 1) * p.HB * p.lpg * VEC * K * sizeof(float);
    norm_bwd_kernel<T, VEC, K><<<(unsigned)(p.gm * p.nhb), kNormThreads, smem, s>>>(a, p);
}
template <typename T, int VEC> void run(bool back, const NormArgs &a, const NormShape &s, cudaStream_t st) {
#define QD_NORM_K(k) back ? run_bwd<T, VEC, k>(a, s.p, st) : run_fwd<T, VEC, k>(a, s.p, st)
    if (s.K == 1) QD_NORM_K(1);
    else if (s.K == 2) QD_NORM_K(2);
    else if (s.K == 4) QD_NORM_K(4);
    else if constexpr (VEC <= 4) {
        if (s.K == 8) QD_NORM_K(8);
        else if constexpr (VEC == 1) QD_NORM_K(32);
    }
#undef QD_NORM_K
}

cudaError_t launch(bool back, const NormArgs &a, const NormShape &s, int dtype, cudaStream_t st, int *nlaunch) {
    if (dtype == kBF16) {
        if (s.vec == 8) run<__nv_bfloat16, 8>(back, a, s, st);
        else run<__nv_bfloat16, 1>(back, a, s, st);
    } else {
        if (s.vec == 4) run<float, 4>(back, a, s, st);
        else run<float, 1>(back, a, s, st);
    }
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) *nlaunch += 1;
    return e;
}

constexpr int kFwdCtas = 8, kBwdCtas = 3;

}  // namespace

cudaError_t launch_norm_fwd(const NormArgs &a, int dtype, cudaStream_t s, int *nlaunch) {
    return launch(false, a, norm_shape(a.M, a.H, a.d, dtype, kFwdCtas), dtype, s, nlaunch);
}

size_t norm_bwd_workspace(int M, int H, int d, int dtype) {
    return (size_t)norm_shape(M, H, d, dtype, kBwdCtas).p.gm * 2 * H * d * sizeof(float);
}

cudaError_t launch_norm_bwd(const NormArgs &a, int dtype, cudaStream_t s, int *nlaunch) {
    const NormShape sh = norm_shape(a.M, a.H, a.d, dtype, kBwdCtas);
    if (a.M > 0) {
        const cudaError_t e = launch(true, a, sh, dtype, s, nlaunch);
        if (e != cudaSuccess) return e;
    }
    if (!a.dw && !a.db) return cudaSuccess;
    const int64_t HD = (int64_t)a.H * a.d;
    return launch_sum_rows(a.part, sh.p.gm, 2 * HD, a.dw, HD, a.db, HD, nullptr, s, nlaunch);
}

}  // namespace qd
