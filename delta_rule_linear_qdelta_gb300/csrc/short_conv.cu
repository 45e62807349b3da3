// Short causal convolution over tokens, one filter of W taps per channel, with a bias and
// an optional SiLU: forward over a sequence, one token in place, and the backward.
//
//   pre_t = bias + sum_j w_j x_{t-W+1+j},  y_t = pre_t or SiLU(pre_t)
//   dx_s = sum_j w_j dpre_{s+W-1-j},  dw_j = sum_t dpre_t x_{t-W+1+j},  dbias = sum_t dpre_t
//
// All three are bound by memory: W + 4 operations per element against 4 to 12 bytes.  A
// thread owns VEC neighbouring channels and walks a run of tokens with the last W - 1
// inputs in registers, so x is read once but for the W - 1 tokens before (backward: and
// after) each run, which neighbouring threads have just brought into the caches.
#include "layer_common.cuh"

namespace qd {
namespace {

constexpr int kThreads = 128;
constexpr int kBatch = 4;             // tokens in flight while as many are computed

// `rows` consecutive channels' filters, w[c * W + j]; 16-byte loads when VEC > 1.
template <int VEC, int W> __device__ __forceinline__ void load_filter(const float *w, float (&f)[VEC][W]) {
    if constexpr (VEC > 1) {
        float flat[VEC * W];
#pragma unroll
        for (int i = 0; i < VEC * W / 4; ++i) {
            const float4 v = reinterpret_cast<const float4 *>(w)[i];
            flat[4 * i] = v.x; flat[4 * i + 1] = v.y; flat[4 * i + 2] = v.z; flat[4 * i + 3] = v.w;
        }
#pragma unroll
        for (int c = 0; c < VEC; ++c)
#pragma unroll
            for (int j = 0; j < W; ++j) f[c][j] = flat[c * W + j];
    } else {
#pragma unroll
        for (int j = 0; j < W; ++j) f[0][j] = w[j];
    }
}

__device__ __forceinline__ int seq_len(const int *lens, int b, int T) {
    return lens ? min(max(lens[b], 0), T) : T;
}

// Thread i: channel vector i % ncv, run i / ncv of the B * nruns runs of `run` tokens.  Run
// 0 alone reads S0 (run >= W - 1) and afterwards writes S_final, so the two may be one buffer.
template <typename T, int VEC, int W>
__global__ void __launch_bounds__(kThreads) conv_fwd_kernel(ConvArgs a, int run, int nruns) {
    using P = Pack<T, VEC>;
    const int ncv = a.D / VEC;
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (i >= (int64_t)a.B * nruns * ncv) return;
    const int cv = (int)(i % ncv);
    const int64_t br = i / ncv;
    const int b = (int)(br / nruns), r = (int)(br % nruns);
    const int D = a.D, n = seq_len(a.lens, b, a.T), c0 = cv * VEC;
    const int t0 = r * run, t1 = min(t0 + run, a.T);
    const T *x = (const T *)a.x + (size_t)b * a.T * D + c0;
    T *y = (T *)a.y + (size_t)b * a.T * D + c0;

    float w[VEC][W], bias[VEC];
    load_filter<VEC, W>(a.w + (size_t)c0 * W, w);
#pragma unroll
    for (int c = 0; c < VEC; ++c) bias[c] = a.bias ? a.bias[c0 + c] : 0.f;

    P head[W - 1];                                     // the W - 1 inputs before t0
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
        const int t = t0 - (W - 1) + k;
        head[k].zero();
        if (t >= 0) {
            if (t < n) head[k].load(x + (size_t)t * D);
        } else if (a.S0) {
            head[k].load((const T *)a.S0 + ((size_t)b * (W - 1) + (t + W - 1)) * D + c0);
        }
    }
    float win[W][VEC];                                 // the inputs t - W + 1 .. t
#pragma unroll
    for (int k = 0; k < W - 1; ++k) head[k].get(win[k + 1]);

    P in[kBatch], next[kBatch];
    auto fetch = [&](P(&to)[kBatch], int t) {
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            to[u].zero();
            if (t + u < t1 && t + u < n) to[u].load(x + (size_t)(t + u) * D);
        }
    };
    fetch(next, t0);
    for (int t = t0; t < t1; t += kBatch) {
#pragma unroll
        for (int u = 0; u < kBatch; ++u) in[u] = next[u];
        fetch(next, t + kBatch);
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
#pragma unroll
            for (int k = 0; k < W - 1; ++k)
#pragma unroll
                for (int c = 0; c < VEC; ++c) win[k][c] = win[k + 1][c];
            in[u].get(win[W - 1]);
            if (t + u < t1) {
                float o[VEC];
#pragma unroll
                for (int c = 0; c < VEC; ++c) {
                    float p = bias[c];
#pragma unroll
                    for (int j = 0; j < W; ++j) p = fmaf(w[c][j], win[j][c], p);
                    if (a.silu) p *= sigmoid_f(p);
                    o[c] = t + u < n ? p : 0.f;
                }
                P out;
                out.set(o);
                out.store(y + (size_t)(t + u) * D);
            }
        }
    }
    if (r == 0 && a.S_final) {                         // the last W - 1 inputs of S0 followed by x
#pragma unroll
        for (int k = 0; k < W - 1; ++k) {
            const int t = n - (W - 1) + k;
            P v;
            if (t >= 0) {
                v.load(x + (size_t)t * D);
            } else {
                v.zero();                              // t = k' - (W - 1) for the k'-th row of S0
#pragma unroll
                for (int m = 0; m < W - 1; ++m)
                    if (m == t + W - 1) v = head[m];
            }
            v.store((T *)a.S_final + ((size_t)b * (W - 1) + k) * D + c0);
        }
    }
}

template <typename T, int VEC, int W>
__global__ void __launch_bounds__(kThreads) conv_step_kernel(ConvArgs a) {
    using P = Pack<T, VEC>;
    const int ncv = a.D / VEC;
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (i >= (int64_t)a.B * ncv) return;
    const int c0 = (int)(i % ncv) * VEC;
    const size_t b = (size_t)(i / ncv);
    const int D = a.D;
    T *S = (T *)a.S_final + b * (W - 1) * D + c0;
    P in[W];
#pragma unroll
    for (int k = 0; k < W - 1; ++k) in[k].load(S + (size_t)k * D);
    in[W - 1].load((const T *)a.x + b * D + c0);
    float w[VEC][W], p[VEC];
    load_filter<VEC, W>(a.w + (size_t)c0 * W, w);
#pragma unroll
    for (int c = 0; c < VEC; ++c) p[c] = a.bias ? a.bias[c0 + c] : 0.f;
#pragma unroll
    for (int j = 0; j < W; ++j) {
        float v[VEC];
        in[j].get(v);
#pragma unroll
        for (int c = 0; c < VEC; ++c) p[c] = fmaf(w[c][j], v[c], p[c]);
    }
    if (a.silu) {
#pragma unroll
        for (int c = 0; c < VEC; ++c) p[c] *= sigmoid_f(p[c]);
    }
    P out;
    out.set(p);
    out.store((T *)a.y + b * D + c0);
#pragma unroll
    for (int k = 0; k < W - 1; ++k) in[k + 1].store(S + (size_t)k * D);
}

// Backward.  A CTA of 256 threads is CV channel vectors by 256 / CV consecutive runs of
// tokens.  A thread walks its run and the W - 1 tokens after it: each token's dpre adds to
// the W pending dx (acc[j] belongs to token t - W + 1 + j; acc[0] is complete and leaves),
// and, inside the run, to dw and dbias, which the CTA then sums over its runs in shared
// memory and leaves as one row of partials ([D][W] of dw, then [D] of dbias).
constexpr int kBwdThreads = 256;

template <typename T, int VEC, int W>
__global__ void __launch_bounds__(kBwdThreads) conv_bwd_kernel(ConvBwdArgs a, int CV, int run, int nrb, int ncb) {
    using P = Pack<T, VEC>;
    const int D = a.D, RB = kBwdThreads / CV;
    const int cvl = threadIdx.x % CV, rl = threadIdx.x / CV;
    const int cb = blockIdx.x % ncb, row = blockIdx.x / ncb;
    const int c0 = (cb * CV + cvl) * VEC;
    const int b = row / nrb, rb = row % nrb;
    const int r = rb * RB + rl;
    const bool on = c0 < D;
    const int n = seq_len(a.lens, b, a.T);
    const int64_t t0l = (int64_t)r * run;
    const int t0 = (int)(t0l < a.T ? t0l : a.T), t1 = min(t0 + run, a.T);
    const size_t base = (size_t)b * a.T * D + c0;
    const T *x = (const T *)a.x + base, *dy = (const T *)a.dy + base;
    T *dx = (T *)a.dx + base;

    float w[VEC][W], bias[VEC], dw[VEC][W], db[VEC], win[W][VEC], acc[W][VEC];
#pragma unroll
    for (int c = 0; c < VEC; ++c) {
        db[c] = 0.f;
#pragma unroll
        for (int j = 0; j < W; ++j) dw[c][j] = acc[j][c] = win[j][c] = 0.f;
    }
    if (on && (t0 < t1 || r == 0)) {
        load_filter<VEC, W>(a.w + (size_t)c0 * W, w);
#pragma unroll
        for (int c = 0; c < VEC; ++c) bias[c] = a.bias ? a.bias[c0 + c] : 0.f;
#pragma unroll
        for (int k = 0; k < W - 1; ++k) {
            const int t = t0 - (W - 1) + k;
            P v;
            v.zero();
            if (t >= 0) {
                if (t < n) v.load(x + (size_t)t * D);
            } else if (a.S0) {
                v.load((const T *)a.S0 + ((size_t)b * (W - 1) + (t + W - 1)) * D + c0);
            }
            v.get(win[k + 1]);
        }
        const int end = t1 + W - 1;                    // tokens t1 .. end - 1 complete the run's last dx
        P xi[kBatch], gi[kBatch], xn[kBatch], gn[kBatch];
        auto fetch = [&](int t) {
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                xn[u].zero();
                gn[u].zero();
                if (t + u < end && t + u < n) {
                    xn[u].load(x + (size_t)(t + u) * D);
                    gn[u].load(dy + (size_t)(t + u) * D);
                }
            }
        };
        fetch(t0);
        for (int t = t0; t < end; t += kBatch) {
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                xi[u] = xn[u];
                gi[u] = gn[u];
            }
            fetch(t + kBatch);
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const int tt = t + u;
                if (tt < end) {
                    float g[VEC];
#pragma unroll
                    for (int k = 0; k < W - 1; ++k)
#pragma unroll
                        for (int c = 0; c < VEC; ++c) win[k][c] = win[k + 1][c];
                    xi[u].get(win[W - 1]);
                    gi[u].get(g);
#pragma unroll
                    for (int c = 0; c < VEC; ++c) {
                        if (a.silu) {
                            float p = bias[c];
#pragma unroll
                            for (int j = 0; j < W; ++j) p = fmaf(w[c][j], win[j][c], p);
                            g[c] *= silu_grad(p, sigmoid_f(p));
                        }
                        if (tt >= n) g[c] = 0.f;
#pragma unroll
                        for (int j = 0; j < W; ++j) acc[j][c] = fmaf(w[c][j], g[c], acc[j][c]);
                        if (tt < t1) {
                            db[c] += g[c];
#pragma unroll
                            for (int j = 0; j < W; ++j) dw[c][j] = fmaf(g[c], win[j][c], dw[c][j]);
                        }
                    }
                    // token s = tt - (W - 1) is complete: it is this run's, or (run 0) a row of S0
                    const int s = tt - (W - 1);
                    if (s >= t0 || r == 0) {
                        float o[VEC];
                        const int kf = s - (n - (W - 1));          // its row in S_final, if any
#pragma unroll
                        for (int c = 0; c < VEC; ++c) o[c] = acc[0][c];
                        if (a.dS_final && kf >= 0 && kf < W - 1) {
                            P v;
                            float f[VEC];
                            v.load((const T *)a.dS_final + ((size_t)b * (W - 1) + kf) * D + c0);
                            v.get(f);
#pragma unroll
                            for (int c = 0; c < VEC; ++c) o[c] += f[c];
                        }
                        P out;
                        out.set(o);
                        if (s >= 0) out.store(dx + (size_t)s * D);
                        else if (a.dS0) out.store((T *)a.dS0 + ((size_t)b * (W - 1) + (s + W - 1)) * D + c0);
                    }
#pragma unroll
                    for (int j = 0; j < W; ++j)
#pragma unroll
                        for (int c = 0; c < VEC; ++c) acc[j][c] = j + 1 < W ? acc[j + 1 < W ? j + 1 : j][c] : 0.f;
                }
            }
        }
    }
    // sum the CTA's runs: [run][channel vector][VEC * (W + 1)], then one thread per column
    constexpr int C = VEC * (W + 1);
    extern __shared__ float sp[];
    float *mine = sp + (size_t)(rl * CV + cvl) * C;
#pragma unroll
    for (int c = 0; c < VEC; ++c) {
#pragma unroll
        for (int j = 0; j < W; ++j) mine[c * W + j] = dw[c][j];
        mine[VEC * W + c] = db[c];
    }
    __syncthreads();
    float *part = a.part + (size_t)row * D * (W + 1);
    for (int m = threadIdx.x; m < CV * C; m += kBwdThreads) {
        const int v = m / C, k = m % C, ch = (cb * CV + v) * VEC;
        if (ch >= D) continue;
        float t = 0.f;
        for (int q = 0; q < RB; ++q) t += sp[(size_t)q * CV * C + m];
        if (k < VEC * W) part[(size_t)ch * W + k] = t;
        else part[(size_t)D * W + ch + (k - VEC * W)] = t;
    }
}

template <typename T, int VEC, int W> void run_fwd(const ConvArgs &a, cudaStream_t s) {
    // The longest run (16, 8 or 4 tokens) that still leaves about 1024 threads per SM: a
    // longer run reads its W - 1 tokens of overlap less often, more threads keep more loads
    // in flight.
    const int64_t vecs = (int64_t)a.B * (a.D / VEC);
    int run = 16;
    while (run > 4 && vecs * ((a.T + run - 1) / run) < (int64_t)kSMs * 1024) run /= 2;
    const int nruns = a.T > 0 ? (a.T + run - 1) / run : 1;
    const int64_t n = vecs * nruns;
    conv_fwd_kernel<T, VEC, W><<<(unsigned)((n + kThreads - 1) / kThreads), kThreads, 0, s>>>(a, run, nruns);
}
template <typename T, int VEC, int W> void run_step(const ConvArgs &a, cudaStream_t s) {
    const int64_t n = (int64_t)a.B * (a.D / VEC);
    conv_step_kernel<T, VEC, W><<<(unsigned)((n + kThreads - 1) / kThreads), kThreads, 0, s>>>(a);
}

struct BwdPlan {
    int vec, CV, run, nrb;     // elements a thread, channel vectors a CTA, tokens a run, CTAs a sequence
    int ncb, rows;             // CTAs along the channels; rows of partials (one per CTA along the tokens)
};
// A thread of the backward takes four channels (its filter, its gradient, the window and
// the pending outputs are 16 W floats); channels that are no multiple of four go one by one.
BwdPlan bwd_plan(int B, int T, int D) {
    BwdPlan p;
    p.vec = D % 4 == 0 ? 4 : 1;
    const int ncv = D / p.vec;
    p.CV = 32;
    while (p.CV > 1 && p.CV / 2 >= ncv) p.CV /= 2;
    const int RB = kBwdThreads / p.CV;
    p.run = 32;
    const int64_t cols = (int64_t)B * ((ncv + p.CV - 1) / p.CV);
    while (p.run > 4 && cols * ((T + p.run * RB - 1) / (p.run * RB)) < 2 * kSMs) p.run /= 2;
    p.nrb = T > 0 ? (T + p.run * RB - 1) / (p.run * RB) : 1;
    p.ncb = (ncv + p.CV - 1) / p.CV;
    p.rows = B * p.nrb;
    return p;
}

template <typename T, int VEC, int W> void run_bwd(const ConvBwdArgs &a, const BwdPlan &p, cudaStream_t s) {
    conv_bwd_kernel<T, VEC, W><<<(unsigned)p.ncb * p.rows, kBwdThreads, kBwdThreads * VEC * (W + 1) * sizeof(float), s>>>(
        a, p.CV, p.run, p.nrb, p.ncb);
}

template <typename T_, int VEC_, int W_> struct Inst {
    using T = T_;
    static constexpr int VEC = VEC_, W = W_;
};

// Calls f(Inst<T, VEC, W>) for the call's dtype, elements per access and tap count.
template <typename T, int VEC, typename F> void with_taps(int W, F f) {
    if (W == 2) f(Inst<T, VEC, 2>());
    else if (W == 3) f(Inst<T, VEC, 3>());
    else f(Inst<T, VEC, 4>());
}
// Channels that fill 16-byte accesses in every row go VECB (bf16) or 4 (fp32) at a time.
template <int VECB, typename F> void with_inst(int dtype, int D, int W, F f) {
    if (dtype == kBF16) {
        if (D % VECB == 0) with_taps<__nv_bfloat16, VECB>(W, f);
        else with_taps<__nv_bfloat16, 1>(W, f);
    } else {
        if (D % 4 == 0) with_taps<float, 4>(W, f);
        else with_taps<float, 1>(W, f);
    }
}

cudaError_t launched(int *nlaunch) {
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) *nlaunch += 1;
    return e;
}

}  // namespace

cudaError_t launch_conv_fwd(const ConvArgs &a, int dtype, cudaStream_t s, int *nlaunch) {
    with_inst<8>(dtype, a.D, a.W, [&](auto i) { run_fwd<typename decltype(i)::T, i.VEC, i.W>(a, s); });
    return launched(nlaunch);
}

cudaError_t launch_conv_step(const ConvArgs &a, int dtype, cudaStream_t s, int *nlaunch) {
    with_inst<8>(dtype, a.D, a.W, [&](auto i) { run_step<typename decltype(i)::T, i.VEC, i.W>(a, s); });
    return launched(nlaunch);
}

size_t conv_bwd_workspace(int B, int T, int D, int W) {
    return (size_t)bwd_plan(B, T, D).rows * D * (W + 1) * sizeof(float);
}

cudaError_t launch_conv_bwd(const ConvBwdArgs &a, int dtype, cudaStream_t s, int *nlaunch) {
    const BwdPlan p = bwd_plan(a.B, a.T, a.D);
    if (p.rows > 0) {
        with_inst<4>(dtype, a.D, a.W, [&](auto i) { run_bwd<typename decltype(i)::T, i.VEC, i.W>(a, p, s); });
        const cudaError_t e = launched(nlaunch);
        if (e != cudaSuccess) return e;
    }
    return launch_sum_rows(a.part, p.rows, (int64_t)a.D * (a.W + 1), a.dw, (int64_t)a.D * a.W, a.dbias, a.D, nullptr, s,
                           nlaunch);
}

}  // namespace qd
