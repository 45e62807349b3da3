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
// 16384 tokens x 16 groups of 128, gated, bf16: forward 37 us (5410 GB/s, 80 % of the copy
// bandwidth), backward 70 us with the sum of the partials (4790 GB/s; at its 80 registers, for three
// CTAs an SM, it spills 36 bytes).  The backward of single accesses (odd widths above 128) spills 430 bytes
// and more: half of each pair that it holds is empty.
#include "layer_common.cuh"

namespace qd {
namespace {

constexpr int kNormThreads = 256;
// Threads on an SM: the backward's registers leave room for these.
constexpr int kFwdThreads = 2048;
__host__ __device__ constexpr int bwd_threads(int K) { return K == 1 ? 768 : 512; }
// Threads of a CTA: one group's when it takes more than a warp.
__host__ __device__ constexpr int cta_threads(int LPG) { return LPG > 32 ? LPG : kNormThreads; }

// How a CTA's threads cover the groups: lpg threads to a group (a power of two up to 32, or a
// whole CTA of 128, 256 or 512), HB groups of one token side by side, MB tokens at once.
struct NormPlan {
    int lpg, HB, MB, nhb, gm;
};

// LPG: the threads of a group (16, 32, or a whole CTA's 128, 256 or 512), or 0 where only the plan
// knows (up to 32).  LPG = 16 is the instance of groups that fill their lanes (128 channels in
// bf16, 64 in fp32: the usual head): nothing has to be masked inside a group.
template <int LPG, int CNT> __device__ __forceinline__ void group_totals(float (&v)[CNT], int lpg, float *sm) {
    const int n = LPG ? LPG : lpg;
    auto join = [&](int o) {
#pragma unroll
        for (int i = 0; i < CNT; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    };
    if (n > 16) join(16);
    if (n > 8) join(8);
    if (n > 4) join(4);
    if (n > 2) join(2);
    if (n > 1) join(1);
    if (LPG > 32) {
        __syncthreads();                               // the last totals have been read by all
        if ((threadIdx.x & 31) == 0) {
#pragma unroll
            for (int i = 0; i < CNT; ++i) sm[(threadIdx.x >> 5) * CNT + i] = v[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < CNT; ++i) {
            v[i] = 0.f;
#pragma unroll
            for (int q = 0; q < cta_threads(LPG) / 32; ++q) v[i] += sm[q * CNT + i];
        }
    }
}

__device__ __forceinline__ f32x2 both(float c) { return pk(c, c); }

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
    // the group's parameter, or `none` where there is none
    __device__ __forceinline__ void param(const float *p, int d, float none, f32x2 (&f)[K][(VEC + 1) / 2]) const {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            constexpr int Q = VEC < 4 ? VEC : 4, H = (Q + 1) / 2;      // floats of an access, pairs of it
#pragma unroll
            for (int i = 0; i < (VEC + 1) / 2; ++i) f[k][i] = both(none);
            if (p && on[k]) {
#pragma unroll
                for (int i = 0; i < VEC / Q; ++i) {
                    Pack<float, Q> q;
                    f32x2 g[H];
                    q.load(p + (size_t)h * d + c[k] + Q * i);
                    q.get2(g);
#pragma unroll
                    for (int j = 0; j < H; ++j) f[k][H * i + j] = g[j];
                }
            }
        }
    }
};

// xh of the thread's channels of one group, and the group's rstd.
template <int VEC, int K, int LPG, int HV>
__device__ __forceinline__ float normalise(f32x2 (&v)[K][HV], const bool (&on)[K], const NormArgs &a, float inv_d, int lpg, float *sm) {
    if (a.center) {
        f32x2 s = 0;
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < HV; ++i) s = add2(s, v[k][i]);
        float tot[1] = {sum2(s)};
        group_totals<LPG>(tot, lpg, sm);
        const float m = -tot[0] * inv_d;
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < HV; ++i) v[k][i] = LPG == 16 || on[k] ? add2(v[k][i], pk(m, VEC == 1 ? 0.f : m)) : 0;
    }
    f32x2 q = 0;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < HV; ++i) q = fma2(v[k][i], v[k][i], q);
    float tot[1] = {sum2(q)};
    group_totals<LPG>(tot, lpg, sm);
    // the hardware's reciprocal root (2 ulp) and one Newton step; an infinite sum of squares leaves 0, of which
    // the step would make a NaN
    const float var = fmaf(tot[0], inv_d, a.eps), r0 = rsqrtf(var);
    const float rstd = r0 == 0.f ? 0.f : r0 * fmaf(-0.5f * var * r0, r0, 1.5f);
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < HV; ++i) v[k][i] = mul2(v[k][i], both(rstd));
    return rstd;
}

template <typename T, int VEC, int K, int LPG>
__global__ void __launch_bounds__(cta_threads(LPG)) norm_fwd_kernel(NormArgs a, NormPlan p) {
    constexpr int HV = (VEC + 1) / 2;
    __shared__ float sm[cta_threads(LPG) / 32];
    const Place<VEC, K> at(a, p);
    f32x2 w[K][HV], b[K][HV];
    at.param(a.w, a.d, 1.f, w);
    at.param(a.b, a.d, 0.f, b);
    const float inv_d = 1.f / (float)a.d;
    const int64_t first = (int64_t)(blockIdx.x / p.nhb) * p.MB, turn = (int64_t)p.gm * p.MB;
    const size_t step = (size_t)turn * a.H * a.d;
    size_t row = ((size_t)(first + at.ml) * a.H + at.h) * a.d;
    Pack<T, VEC> xn[K], zn[K];
    auto fetch = [&](int64_t m, size_t row) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (LPG != 16) {
                xn[k].zero();
                zn[k].zero();
            }
            // (a dead lane of a full group computes on what it has, and stores nothing)
            if (at.on[k] && m < a.M) {
                xn[k].load((const T *)a.x + row + at.c[k]);
                if (a.z) zn[k].load((const T *)a.z + row + at.c[k]);
            }
        }
    };
    if (LPG == 16) {
        xn[0].zero();
        zn[0].zero();
    }
    fetch(first + at.ml, row);
    // every thread of the CTA makes the same number of turns: the group totals synchronise
    for (int64_t m0 = first; m0 < a.M; m0 += turn, row += step) {
        const int64_t m = m0 + at.ml;
        f32x2 v[K][HV], t[K][HV];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            xn[k].get2(v[k]);
            zn[k].get2(t[k]);
        }
        fetch(m + turn, row + step);                   // the next token's, while this one is computed
        normalise<VEC, K, LPG, HV>(v, at.on, a, inv_d, p.lpg, sm);
#pragma unroll
        for (int k = 0; k < K; ++k) {
#pragma unroll
            for (int i = 0; i < HV; ++i) v[k][i] = fma2(v[k][i], w[k][i], b[k][i]);
            if (a.z) {
                if (a.silu) {
#pragma unroll
                    for (int i = 0; i < HV; ++i) t[k][i] = mul2(t[k][i], sigmoid2(t[k][i]));
                }
#pragma unroll
                for (int i = 0; i < HV; ++i) v[k][i] = mul2(v[k][i], t[k][i]);
            } else if (a.silu) {
#pragma unroll
                for (int i = 0; i < HV; ++i) v[k][i] = mul2(v[k][i], sigmoid2(v[k][i]));
            }
            if (at.on[k] && m < a.M) {
                Pack<T, VEC> y;
                y.set2(v[k]);
                y.store((T *)a.y + row + at.c[k]);
            }
        }
    }
}

template <typename T, int VEC, int K, int LPG>
__global__ void __launch_bounds__(cta_threads(LPG), K * VEC > 8 ? 1 : bwd_threads(K) / cta_threads(LPG)) norm_bwd_kernel(NormArgs a, NormPlan p) {
    constexpr int HV = (VEC + 1) / 2;
    __shared__ float sm[2 * cta_threads(LPG) / 32];
    extern __shared__ float sp[];
    const Place<VEC, K> at(a, p);
    f32x2 w[K][HV], b[K][HV], dw[K][HV] = {}, db[K][HV] = {};
    at.param(a.w, a.d, 1.f, w);
    at.param(a.b, a.d, 0.f, b);
    const float inv_d = 1.f / (float)a.d;
    const int64_t begin = (int64_t)(blockIdx.x / p.nhb) * p.MB, turn = (int64_t)p.gm * p.MB;
    const size_t step = (size_t)turn * a.H * a.d;
    size_t row = ((size_t)(begin + at.ml) * a.H + at.h) * a.d;
    Pack<T, VEC> xn[K], zn[K], dyn[K];
    auto fetch = [&](int64_t m, size_t row) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (LPG != 16) {
                xn[k].zero();
                zn[k].zero();
            }
            dyn[k].zero();                             // (no gradient comes from a dead lane)
            if (at.on[k] && m < a.M) {
                xn[k].load((const T *)a.x + row + at.c[k]);
                dyn[k].load((const T *)a.dy + row + at.c[k]);
                if (a.z) zn[k].load((const T *)a.z + row + at.c[k]);
            }
        }
    };
    if (LPG == 16) {
        xn[0].zero();
        zn[0].zero();
    }
    fetch(begin + at.ml, row);
    for (int64_t m0 = begin; m0 < a.M; m0 += turn, row += step) {
        const int64_t m = m0 + at.ml;
        f32x2 v[K][HV], g[K][HV], z[K][HV];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            xn[k].get2(v[k]);
            dyn[k].get2(g[k]);
            zn[k].get2(z[k]);
        }
        fetch(m + turn, row + step);
        const float rstd = normalise<VEC, K, LPG, HV>(v, at.on, a, inv_d, p.lpg, sm);
        f32x2 s1 = 0, s2 = 0;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (a.z) {
#pragma unroll
                for (int i = 0; i < HV; ++i) {
                    const f32x2 n = fma2(v[k][i], w[k][i], b[k][i]), gn = mul2(g[k][i], n);
                    if (a.silu) {
                        const f32x2 s = sigmoid2(z[k][i]);
                        g[k][i] = mul2(g[k][i], mul2(z[k][i], s));
                        z[k][i] = mul2(gn, silu_grad2(z[k][i], s));
                    } else {
                        g[k][i] = mul2(g[k][i], z[k][i]);
                        z[k][i] = gn;
                    }
                }
                if (at.on[k] && m < a.M) {
                    Pack<T, VEC> o;
                    o.set2(z[k]);
                    o.store((T *)a.dz + row + at.c[k]);
                }
            } else if (a.silu) {
#pragma unroll
                for (int i = 0; i < HV; ++i) {
                    const f32x2 n = fma2(v[k][i], w[k][i], b[k][i]);
                    g[k][i] = mul2(g[k][i], silu_grad2(n, sigmoid2(n)));
                }
            }
#pragma unroll
            for (int i = 0; i < HV; ++i) {
                dw[k][i] = fma2(g[k][i], v[k][i], dw[k][i]);
                db[k][i] = add2(db[k][i], g[k][i]);
                g[k][i] = mul2(g[k][i], w[k][i]);
                s1 = add2(s1, g[k][i]);
                s2 = fma2(g[k][i], v[k][i], s2);
            }
        }
        float tot[2] = {sum2(s1), sum2(s2)};
        group_totals<LPG>(tot, p.lpg, sm);
        const f32x2 m1 = both(a.center ? -tot[0] * inv_d : 0.f), m2 = both(-tot[1] * inv_d);
#pragma unroll
        for (int k = 0; k < K; ++k) {
#pragma unroll
            for (int i = 0; i < HV; ++i) g[k][i] = mul2(both(rstd), fma2(v[k][i], m2, add2(g[k][i], m1)));
            if (at.on[k] && m < a.M) {
                Pack<T, VEC> o;
                o.set2(g[k]);
                o.store((T *)a.dx + row + at.c[k]);
            }
        }
    }
    if (!a.part) return;
    // join the CTA's MB tokens and leave one row of partials: dw [H][d], db [H][d]
    const size_t HD = (size_t)a.H * a.d;
    float *part = a.part + (size_t)(blockIdx.x / p.nhb) * 2 * HD;
    const int side = p.HB * p.lpg, width = side * VEC * K;             // threads and channels of one token in the CTA
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        float acc[K][2 * HV];
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < HV; ++i) unpk(which ? db[k][i] : dw[k][i], acc[k][2 * i], acc[k][2 * i + 1]);
        if (p.MB > 1) {
            __syncthreads();
            if (at.live && at.ml > 0)
#pragma unroll
                for (int k = 0; k < K; ++k)
#pragma unroll
                    for (int c = 0; c < VEC; ++c)
                        sp[(size_t)(at.ml - 1) * width + (k * VEC + c) * side + threadIdx.x % side] = acc[k][c];
            __syncthreads();
            if (at.live && at.ml == 0)
#pragma unroll
                for (int k = 0; k < K; ++k)
#pragma unroll
                    for (int c = 0; c < VEC; ++c)
                        for (int q = 0; q + 1 < p.MB; ++q) acc[k][c] += sp[(size_t)q * width + (k * VEC + c) * side + threadIdx.x];
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
// A thread holds up to 8 channels (bf16: one 16-byte access, or the 4- or 2-byte ones that odd
// widths leave; fp32: two): fewer keep its lanes' shuffles busier than its loads, and with 32 a
// lane needs 250 registers (1000 channels, bf16: 42 us forward, 131 us backward at 20000 groups,
// 27 and 59 us at 8).  The group goes to the fewest lanes of a warp, or to the smallest CTA, that
// take it so; beyond 4096 channels a thread holds 16.  The grid fills the SMs once and
// walks the tokens.
NormShape norm_shape(int M, int H, int d, int dtype, bool back) {
    NormShape s;
    const int wide = dtype == kBF16 ? 8 : 4;
    s.vec = d % wide == 0 ? wide : d % 2 == 0 ? 2 : 1;
    const int nv = d / s.vec, most = 8 / s.vec;        // accesses of a group; of a thread
    s.K = 1;
    while (s.K < most && nv > 32 * s.K) s.K *= 2;
    s.p.lpg = s.K > 1 ? 32 : 1;
    while (s.p.lpg < 512 && s.p.lpg * s.K < nv) s.p.lpg *= 2;
    if (s.p.lpg == 64) s.p.lpg = 128;
    if (s.p.lpg * s.K < nv) s.K *= 2;
    const int nt = cta_threads(s.p.lpg), slots = nt / s.p.lpg, ctas_per_sm = s.K > most ? 1 : (back ? bwd_threads(s.K) : kFwdThreads) / nt;
    s.p.HB = H < slots ? H : slots;
    s.p.MB = slots / s.p.HB;
    s.p.nhb = (H + s.p.HB - 1) / s.p.HB;
    const int64_t turns = ((int64_t)M + s.p.MB - 1) / s.p.MB;
    int64_t gm = ((int64_t)ctas_per_sm * kSMs + s.p.nhb - 1) / s.p.nhb;
    if (gm > turns) gm = turns;
    s.p.gm = (int)gm;
    return s;
}

template <typename T, int VEC, int K, int LPG> void run_fwd(const NormArgs &a, const NormPlan &p, cudaStream_t s) {
    norm_fwd_kernel<T, VEC, K, LPG><<<(unsigned)(p.gm * p.nhb), cta_threads(LPG), 0, s>>>(a, p);
}
template <typename T, int VEC, int K, int LPG> void run_bwd(const NormArgs &a, const NormPlan &p, cudaStream_t s) {
    const size_t smem = (size_t)(p.MB - 1) * p.HB * p.lpg * VEC * K * sizeof(float);
    norm_bwd_kernel<T, VEC, K, LPG><<<(unsigned)(p.gm * p.nhb), cta_threads(LPG), smem, s>>>(a, p);
}
template <typename T, int VEC> void run(bool back, const NormArgs &a, const NormShape &s, cudaStream_t st) {
#define QD_NORM_K(k, l) back ? run_bwd<T, VEC, k, l>(a, s.p, st) : run_fwd<T, VEC, k, l>(a, s.p, st)
    constexpr int MOST = 8 / VEC;
    if (s.K > MOST) QD_NORM_K(2 * MOST, 512);
    else if (s.p.lpg == 512) QD_NORM_K(MOST, 512);
    else if (s.p.lpg == 256) QD_NORM_K(MOST, 256);
    else if (s.p.lpg == 128) QD_NORM_K(MOST, 128);
    else if (s.K == 1) {
        if constexpr (VEC > 2) {
            if (a.d == 16 * VEC) {
                QD_NORM_K(1, 16);
                return;
            }
        }
        QD_NORM_K(1, 0);
    }
    else if constexpr (MOST > 1) {
        if (s.K == MOST) QD_NORM_K(MOST, 32);
        else if constexpr (MOST > 2) {
            if (s.K == 2) QD_NORM_K(2, 32);
            else if constexpr (MOST > 4) QD_NORM_K(4, 32);
        }
    }
#undef QD_NORM_K
}

cudaError_t launch(bool back, const NormArgs &a, const NormShape &s, int dtype, cudaStream_t st, int *nlaunch) {
    if (dtype == kBF16) {
        if (s.vec == 8) run<__nv_bfloat16, 8>(back, a, s, st);
        else if (s.vec == 2) run<__nv_bfloat16, 2>(back, a, s, st);
        else run<__nv_bfloat16, 1>(back, a, s, st);
    } else {
        if (s.vec == 4) run<float, 4>(back, a, s, st);
        else if (s.vec == 2) run<float, 2>(back, a, s, st);
        else run<float, 1>(back, a, s, st);
    }
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) *nlaunch += 1;
    return e;
}

}  // namespace

cudaError_t launch_norm_fwd(const NormArgs &a, int dtype, cudaStream_t s, int *nlaunch) {
    return launch(false, a, norm_shape(a.M, a.H, a.d, dtype, false), dtype, s, nlaunch);
}

size_t norm_bwd_workspace(int M, int H, int d, int dtype) {
    return (size_t)norm_shape(M, H, d, dtype, true).p.gm * 2 * H * d * sizeof(float);
}

cudaError_t launch_norm_bwd(const NormArgs &a, int dtype, cudaStream_t s, int *nlaunch) {
    const NormShape sh = norm_shape(a.M, a.H, a.d, dtype, true);
    if (a.M > 0) {
        const cudaError_t e = launch(true, a, sh, dtype, s, nlaunch);
        if (e != cudaSuccess) return e;
    }
    if (!a.dw && !a.db) return cudaSuccess;
    const int64_t HD = (int64_t)a.H * a.d;
    return launch_sum_rows(a.part, sh.p.gm, 2 * HD, a.dw, HD, a.db, HD, nullptr, s, nlaunch);
}

}  // namespace qd
