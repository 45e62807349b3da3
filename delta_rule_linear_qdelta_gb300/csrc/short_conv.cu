// Short causal convolution over tokens, one filter of W taps per channel, with a bias and
// an optional SiLU: forward over a sequence, one token in place, and the backward.
//
//   pre_t = bias + sum_j w_j x_{t-W+1+j},  y_t = pre_t or SiLU(pre_t)
//   dx_s = sum_j w_j dpre_{s+W-1-j},  dw_j = sum_t dpre_t x_{t-W+1+j},  dbias = sum_t dpre_t
//
// All three are bound by memory: W + 4 operations per element against 4 to 12 bytes.  A
// thread owns VEC neighbouring channels and walks a run of tokens with the last W - 1
// inputs in registers, so x is read once but for the W - 1 tokens before (backward: and
// after) each run.  The tokens ahead arrive by asynchronous copies in a ring of shared memory
// that only this thread uses: no barrier, and registers hold the filters, not the loads.
// 8 x 2048 tokens x 2048 channels, 4 taps, bf16: forward 28.7 us (4670 GB/s, 69 % of the copy
// bandwidth; four CTAs an SM, five spill: 30.7 us), backward 55 us with the sum of the partials
// (3640 GB/s; loads prefetched into registers: 225 us at one CTA an SM).
#include <type_traits>

#include "layer_common.cuh"

namespace qd {
namespace {

constexpr int kBatch = 4, kRing = 3;  // tokens computed together; batches in the ring
constexpr int kFwdThreads = 128, kBwdThreads = 256, kStepThreads = 128;
constexpr int kFwdCtas = 4, kBwdCtas = 2;    // resident on an SM

// The filters of VEC channels (w[c][j]) as pairs of channels per tap.
template <int VEC, int W> __device__ __forceinline__ void load_filter(const float *w, f32x2 (&f)[W][(VEC + 1) / 2]) {
    float flat[(VEC + 1) * W];
    if constexpr (VEC == 2) {
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const float2 v = reinterpret_cast<const float2 *>(w)[i];
            flat[2 * i] = v.x; flat[2 * i + 1] = v.y;
        }
    } else if constexpr (VEC > 2) {
#pragma unroll
        for (int i = 0; i < VEC * W / 4; ++i) {
            const float4 v = reinterpret_cast<const float4 *>(w)[i];
            flat[4 * i] = v.x; flat[4 * i + 1] = v.y; flat[4 * i + 2] = v.z; flat[4 * i + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int j = 0; j < W; ++j) {
            flat[j] = w[j];
            flat[W + j] = 0.f;
        }
    }
#pragma unroll
    for (int j = 0; j < W; ++j)
#pragma unroll
        for (int i = 0; i < (VEC + 1) / 2; ++i) f[j][i] = pk(flat[2 * i * W + j], flat[(2 * i + 1) * W + j]);
}
template <int VEC> __device__ __forceinline__ void load_bias(const float *bias, int c0, f32x2 (&f)[(VEC + 1) / 2]) {
#pragma unroll
    for (int i = 0; i < (VEC + 1) / 2; ++i)
        f[i] = bias ? pk(bias[c0 + 2 * i], 2 * i + 1 < VEC ? bias[c0 + 2 * i + 1] : 0.f) : 0;
}

__device__ __forceinline__ int seq_len(const int *lens, int b, int T) {
    return lens ? min(max(lens[b], 0), T) : T;
}

// One array's tokens ahead: slot u of batch i of this thread's ring, or zeros past `end`.  Single
// 16-bit elements are below what a copy can move.
template <typename T, int VEC, int THREADS> struct Ahead {
    using P = Pack<T, VEC>;
    static constexpr bool ASYNC = VEC * sizeof(T) >= 4;
    static constexpr size_t BYTES = ASYNC ? (size_t)kRing * kBatch * THREADS * VEC * sizeof(T) : 0;
    __device__ __forceinline__ static T *slot(T *ring, int buf, int u) {
        return ring + ((size_t)(buf * kBatch + u) * THREADS + threadIdx.x) * VEC;
    }
    // The batch at t, from src (its first token), and src to the next one; `any`: an address to read nothing from.
    __device__ __forceinline__ static void issue(T *ring, int buf, const T *&src, size_t D, int t, int end, const T *any) {
        if constexpr (ASYNC) {
            T *to = slot(ring, buf, 0);
            if (t + kBatch <= end) {
#pragma unroll
                for (int u = 0; u < kBatch; ++u) copy_async<VEC * sizeof(T)>(to + u * THREADS * VEC, src + u * D);
            } else {
#pragma unroll
                for (int u = 0; u < kBatch; ++u)
                    copy_async<VEC * sizeof(T)>(to + u * THREADS * VEC, t + u < end ? src + u * D : any, t + u < end);
            }
            src += kBatch * D;
        }
    }
    // What cannot be copied is loaded a batch at a time instead.
    __device__ __forceinline__ static void arrive(P (&now)[kBatch], const T *src, int D, int t, int end) {
        if constexpr (!ASYNC) {
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                now[u].zero();
                if (t + u < end) now[u].load(src + (size_t)(t + u) * D);
            }
        }
    }
    __device__ __forceinline__ static void get(T *ring, int buf, int u, const P (&now)[kBatch], f32x2 (&f)[(VEC + 1) / 2]) {
        P v;
        if constexpr (ASYNC) v.load(slot(ring, buf, u));
        else v = now[u];
        v.get2(f);
    }
};

// Thread i: channel vector i % ncv, run i / ncv of the B * nruns runs of `run` tokens.  Run
// 0 alone reads S0 (run >= W - 1) and afterwards writes S_final, so the two may be one buffer.
template <typename T, int VEC, int W>
__global__ void __launch_bounds__(kFwdThreads, kFwdCtas) conv_fwd_kernel(ConvArgs a, int run, int nruns) {
    using P = Pack<T, VEC>;
    using In = Ahead<T, VEC, kFwdThreads>;
    constexpr int HV = (VEC + 1) / 2;
    extern __shared__ float4 smem4[];
    T *ring = reinterpret_cast<T *>(smem4);
    const int ncv = a.D / VEC;
    const int64_t i = (int64_t)blockIdx.x * kFwdThreads + threadIdx.x;
    if (i >= (int64_t)a.B * nruns * ncv) return;
    const int cv = (int)(i % ncv);
    const int64_t br = i / ncv;
    const int b = (int)(br / nruns), r = (int)(br % nruns);
    const int D = a.D, n = seq_len(a.lens, b, a.T), c0 = cv * VEC;
    const int t0 = (int)min((int64_t)r * run, (int64_t)a.T), t1 = min(t0 + run, a.T), end = min(t1, n);
    const T *x = (const T *)a.x + (size_t)b * a.T * D + c0;
    T *y = (T *)a.y + (size_t)b * a.T * D + c0;

    const T *next = x + (size_t)t0 * D;
#pragma unroll
    for (int i = 0; i + 1 < kRing; ++i) {
        In::issue(ring, i, next, D, t0 + i * kBatch, end, x);
        copies_issued();
    }
    f32x2 w[W][HV], bias[HV];
    load_filter<VEC, W>(a.w + (size_t)c0 * W, w);
    load_bias<VEC>(a.bias, c0, bias);

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
    f32x2 win[W][HV];                                  // the inputs t - W + 1 .. t
#pragma unroll
    for (int k = 0; k < W - 1; ++k) head[k].get2(win[k + 1]);

    int buf = 0;
    T *yt = y + (size_t)t0 * D;
    for (int t = t0; t < t1; t += kBatch, buf = buf + 1 < kRing ? buf + 1 : 0) {
        In::issue(ring, buf ? buf - 1 : kRing - 1, next, D, t + (kRing - 1) * kBatch, end, x);
        copies_issued();
        copies_done<kRing - 1>();
        P now[kBatch];
        In::arrive(now, x, D, t, end);
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
#pragma unroll
            for (int k = 0; k < W - 1; ++k)
#pragma unroll
                for (int h = 0; h < HV; ++h) win[k][h] = win[k + 1][h];
            In::get(ring, buf, u, now, win[W - 1]);
            f32x2 o[HV];
#pragma unroll
            for (int h = 0; h < HV; ++h) {
                o[h] = bias[h];
#pragma unroll
                for (int j = 0; j < W; ++j) o[h] = fma2(w[j][h], win[j][h], o[h]);
            }
            if (a.silu) {
#pragma unroll
                for (int h = 0; h < HV; ++h) o[h] = mul2(o[h], sigmoid2(o[h]));
            }
            if (t + u < t1) {
                P out;
                out.set2(o);
                if (t + u >= n) out.zero();
                out.store(yt + u * (size_t)D);
            }
        }
        yt += kBatch * (size_t)D;
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
__global__ void __launch_bounds__(kStepThreads) conv_step_kernel(ConvArgs a) {
    using P = Pack<T, VEC>;
    constexpr int HV = (VEC + 1) / 2;
    const int ncv = a.D / VEC;
    const int64_t i = (int64_t)blockIdx.x * kStepThreads + threadIdx.x;
    if (i >= (int64_t)a.B * ncv) return;
    const int c0 = (int)(i % ncv) * VEC;
    const size_t b = (size_t)(i / ncv);
    const int D = a.D;
    T *S = (T *)a.S_final + b * (W - 1) * D + c0;
    P in[W];
#pragma unroll
    for (int k = 0; k < W - 1; ++k) in[k].load(S + (size_t)k * D);
    in[W - 1].load((const T *)a.x + b * D + c0);
    f32x2 w[W][HV], p[HV];
    load_filter<VEC, W>(a.w + (size_t)c0 * W, w);
    load_bias<VEC>(a.bias, c0, p);
#pragma unroll
    for (int j = 0; j < W; ++j) {
        f32x2 v[HV];
        in[j].get2(v);
#pragma unroll
        for (int h = 0; h < HV; ++h) p[h] = fma2(w[j][h], v[h], p[h]);
    }
    if (a.silu) {
#pragma unroll
        for (int h = 0; h < HV; ++h) p[h] = mul2(p[h], sigmoid2(p[h]));
    }
    P out;
    out.set2(p);
    out.store((T *)a.y + b * D + c0);
#pragma unroll
    for (int k = 0; k < W - 1; ++k) in[k + 1].store(S + (size_t)k * D);
}

// Backward.  A CTA of 256 threads is CV channel vectors by 256 / CV consecutive runs of
// tokens.  A thread walks its run and the W - 1 tokens after it: each token's dpre adds to
// the W pending dx (acc[j] belongs to token t - W + 1 + j; acc[0] is complete and leaves),
// and, inside the run, to dw and dbias, which the CTA then sums over its runs in shared
// memory and leaves as one row of partials ([D][W] of dw, then [D] of dbias).
template <typename T, int VEC, int W>
__global__ void __launch_bounds__(kBwdThreads, kBwdCtas) conv_bwd_kernel(ConvBwdArgs a, int CV, int run, int nrb, int ncb) {
    using P = Pack<T, VEC>;
    using In = Ahead<T, VEC, kBwdThreads>;
    constexpr int HV = (VEC + 1) / 2;
    extern __shared__ float4 smem4[];
    T *rx = reinterpret_cast<T *>(smem4), *rg = rx + In::BYTES / sizeof(T);
    const int D = a.D, RB = kBwdThreads / CV;
    const int cvl = threadIdx.x % CV, rl = threadIdx.x / CV;
    const int cb = blockIdx.x % ncb, row = blockIdx.x / ncb;
    const int c0 = (cb * CV + cvl) * VEC;
    const int b = row / nrb, rb = row % nrb;
    const int r = rb * RB + rl;
    const int n = seq_len(a.lens, b, a.T);
    const int t0 = (int)min((int64_t)r * run, (int64_t)a.T), t1 = min(t0 + run, a.T);
    const size_t base = (size_t)b * a.T * D + c0;
    const T *x = (const T *)a.x + base, *dy = (const T *)a.dy + base;
    T *dx = (T *)a.dx + base;

    f32x2 dw[W][HV] = {}, db[HV] = {};
    if (c0 < D && (t0 < t1 || r == 0)) {
        const int stop = t1 + W - 1, end = min(stop, n);       // tokens t1 .. stop - 1 complete the run's last dx
        const T *xn = x + (size_t)t0 * D, *gn = dy + (size_t)t0 * D;
        auto issue = [&](int t, int buf) {
            In::issue(rx, buf, xn, D, t, end, x);
            In::issue(rg, buf, gn, D, t, end, dy);
            copies_issued();
        };
#pragma unroll
        for (int i = 0; i + 1 < kRing; ++i) issue(t0 + i * kBatch, i);
        f32x2 w[W][HV], bias[HV], win[W][HV], acc[W][HV] = {};
        load_filter<VEC, W>(a.w + (size_t)c0 * W, w);
        load_bias<VEC>(a.bias, c0, bias);
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
            v.get2(win[k + 1]);
        }
        int buf = 0;
        T *xs = nullptr;                                       // where the batch's first complete token goes
        P xnow[kBatch], gnow[kBatch];
        // One token; INSIDE: it and its W - 1 predecessors are plain tokens of this run.
        auto token = [&](auto inside, int t, int u) {
            constexpr bool INSIDE = decltype(inside)::value;
            const int tt = t + u, s = tt - (W - 1);
            f32x2 g[HV];
#pragma unroll
            for (int k = 0; k < W - 1; ++k)
#pragma unroll
                for (int h = 0; h < HV; ++h) win[k][h] = win[k + 1][h];
            In::get(rx, buf, u, xnow, win[W - 1]);
            In::get(rg, buf, u, gnow, g);
            if (a.silu) {
#pragma unroll
                for (int h = 0; h < HV; ++h) {
                    f32x2 p = bias[h];
#pragma unroll
                    for (int j = 0; j < W; ++j) p = fma2(w[j][h], win[j][h], p);
                    g[h] = mul2(g[h], silu_grad2(p, sigmoid2(p)));
                }
            }
            // padding adds nothing, not even 0 times what the window still holds
            if (INSIDE || tt < n) {
#pragma unroll
                for (int j = 0; j < W; ++j)
#pragma unroll
                    for (int h = 0; h < HV; ++h) acc[j][h] = fma2(w[j][h], g[h], acc[j][h]);
            }
            if (INSIDE || tt < min(t1, n)) {
#pragma unroll
                for (int h = 0; h < HV; ++h) {
                    db[h] = add2(db[h], g[h]);
#pragma unroll
                    for (int j = 0; j < W; ++j) dw[j][h] = fma2(g[h], win[j][h], dw[j][h]);
                }
            }
            // token s is complete: it is this run's, or (run 0) a row of S0
            if (INSIDE || (tt < stop && (s >= t0 || r == 0))) {
                f32x2 o[HV];
#pragma unroll
                for (int h = 0; h < HV; ++h) o[h] = acc[0][h];
                const int kf = s - (n - (W - 1));              // its row in S_final, if any
                if (!INSIDE && a.dS_final && kf >= 0 && kf < W - 1) {
                    P v;
                    f32x2 f[HV];
                    v.load((const T *)a.dS_final + ((size_t)b * (W - 1) + kf) * D + c0);
                    v.get2(f);
#pragma unroll
                    for (int h = 0; h < HV; ++h) o[h] = add2(o[h], f[h]);
                }
                P out;
                out.set2(o);
                if (INSIDE) out.store(xs + u * (size_t)D);
                else if (s >= 0) out.store(dx + (size_t)s * D);
                else if (a.dS0) out.store((T *)a.dS0 + ((size_t)b * (W - 1) + (s + W - 1)) * D + c0);
            }
#pragma unroll
            for (int j = 0; j < W; ++j)
#pragma unroll
                for (int h = 0; h < HV; ++h) acc[j][h] = j + 1 < W ? acc[j + 1 < W ? j + 1 : j][h] : 0;
        };
        for (int t = t0; t < stop; t += kBatch, buf = buf + 1 < kRing ? buf + 1 : 0) {
            issue(t + (kRing - 1) * kBatch, buf ? buf - 1 : kRing - 1);
            copies_done<kRing - 1>();
            In::arrive(xnow, x, D, t, end);
            In::arrive(gnow, dy, D, t, end);
            if (t >= t0 + W - 1 && t + kBatch <= min(t1, n)) {
                xs = dx + (size_t)(t - (W - 1)) * D;
#pragma unroll
                for (int u = 0; u < kBatch; ++u) token(std::true_type{}, t, u);
            } else {
#pragma unroll
                for (int u = 0; u < kBatch; ++u) token(std::false_type{}, t, u);
            }
        }
        copies_done<0>();
    }
    // sum the CTA's runs: [run][channel vector][VEC * (W + 1)], then one thread per column
    constexpr int C = VEC * (W + 1);
    float *sp = reinterpret_cast<float *>(smem4);
    __syncthreads();                                           // every ring is read out
    float *mine = sp + (size_t)(rl * CV + cvl) * C;
#pragma unroll
    for (int h = 0; h < HV; ++h) {
#pragma unroll
        for (int j = 0; j <= W; ++j) {
            float lo, hi;
            unpk(j < W ? dw[j < W ? j : 0][h] : db[h], lo, hi);
            mine[j < W ? 2 * h * W + j : VEC * W + 2 * h] = lo;
            if (2 * h + 1 < VEC) mine[j < W ? (2 * h + 1) * W + j : VEC * W + 2 * h + 1] = hi;
        }
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

// The run (a multiple of the batch) of the least time: rounds of `slots` resident CTAs, each
// as long as a run and what it costs beside its tokens (`extra`: overlap, filters, first copies).
template <typename F> int best_run(int T, int64_t slots, int extra, F ctas) {
    int best = kBatch;
    int64_t least = INT64_MAX;
    for (int run = kBatch; run <= 256 && run < T + kBatch; run += kBatch) {
        const int64_t cost = (ctas(run) + slots - 1) / slots * (run + extra);
        if (cost < least) {
            least = cost;
            best = run;
        }
    }
    return best;
}

template <typename T, int VEC, int W> void run_fwd(const ConvArgs &a, cudaStream_t s) {
    const int64_t vecs = (int64_t)a.B * (a.D / VEC);
    auto ctas = [&](int run) { return (vecs * ((a.T + run - 1) / run) + kFwdThreads - 1) / kFwdThreads; };
    const int run = best_run(a.T, kFwdCtas * kSMs, 12, ctas);
    const int nruns = a.T > 0 ? (a.T + run - 1) / run : 1;
    const int64_t n = vecs * nruns;
    conv_fwd_kernel<T, VEC, W><<<(unsigned)((n + kFwdThreads - 1) / kFwdThreads), kFwdThreads,
                                 Ahead<T, VEC, kFwdThreads>::BYTES, s>>>(a, run, nruns);
}
template <typename T, int VEC, int W> void run_step(const ConvArgs &a, cudaStream_t s) {
    const int64_t n = (int64_t)a.B * (a.D / VEC);
    conv_step_kernel<T, VEC, W><<<(unsigned)((n + kStepThreads - 1) / kStepThreads), kStepThreads, 0, s>>>(a);
}

// The channels of an access: the most, up to MOST (bf16) or 4 (fp32), that divide D and so start
// every row's accesses on a multiple of their size.
int access_size(int D, int most) {
    int v = most;
    while (D % v) v /= 2;
    return v;
}
struct BwdPlan {
    int vec, CV, run, nrb;     // elements a thread, channel vectors a CTA, tokens a run, CTAs a sequence
    int ncb;                   // CTAs along the channels
    int64_t rows;              // rows of partials (one per CTA along the tokens)
};
// A thread of the backward takes up to four channels: its filter, its gradient, the window and the
// pending outputs are then 16 W floats.
BwdPlan bwd_plan(int B, int T, int D) {
    BwdPlan p;
    p.vec = access_size(D, 4);
    const int ncv = D / p.vec;
    p.CV = 32;
    while (p.CV > 1 && p.CV / 2 >= ncv) p.CV /= 2;
    const int RB = kBwdThreads / p.CV;
    p.ncb = (ncv + p.CV - 1) / p.CV;
    p.run = best_run(T, kBwdCtas * kSMs, 24, [&](int run) { return (int64_t)B * p.ncb * ((T + run * RB - 1) / (run * RB)); });
    p.nrb = T > 0 ? (T + p.run * RB - 1) / (p.run * RB) : 1;
    p.rows = (int64_t)B * p.nrb;
    return p;
}

template <typename T, int VEC, int W> cudaError_t run_bwd(const ConvBwdArgs &a, const BwdPlan &p, cudaStream_t s) {
    const size_t ring = 2 * Ahead<T, VEC, kBwdThreads>::BYTES, sums = kBwdThreads * VEC * (W + 1) * sizeof(float);
    const size_t smem = ring > sums ? ring : sums;
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(conv_bwd_kernel<T, VEC, W>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    conv_bwd_kernel<T, VEC, W><<<(unsigned)(p.ncb * p.rows), kBwdThreads, smem, s>>>(a, p.CV, p.run, p.nrb, p.ncb);
    return cudaGetLastError();
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
template <int MOST, typename F> void with_inst(int dtype, int D, int W, F f) {
    const int v = access_size(D, dtype == kBF16 ? MOST : 4);
    if (dtype == kBF16) {
        if (v == 8) {
            if constexpr (MOST == 8) with_taps<__nv_bfloat16, 8>(W, f);
        }
        else if (v == 4) with_taps<__nv_bfloat16, 4>(W, f);
        else if (v == 2) with_taps<__nv_bfloat16, 2>(W, f);
        else with_taps<__nv_bfloat16, 1>(W, f);
    } else {
        if (v == 4) with_taps<float, 4>(W, f);
        else if (v == 2) with_taps<float, 2>(W, f);
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

double conv_bwd_ctas(int B, int T, int D) {
    const BwdPlan p = bwd_plan(B, T, D);
    return (double)p.ncb * (double)p.rows;
}

size_t conv_bwd_workspace(int B, int T, int D, int W) {
    return (size_t)bwd_plan(B, T, D).rows * D * (W + 1) * sizeof(float);
}

cudaError_t launch_conv_bwd(const ConvBwdArgs &a, int dtype, cudaStream_t s, int *nlaunch) {
    const BwdPlan p = bwd_plan(a.B, a.T, a.D);
    if (p.rows > 0) {
        cudaError_t e = cudaSuccess;
        with_inst<4>(dtype, a.D, a.W, [&](auto i) { e = run_bwd<typename decltype(i)::T, i.VEC, i.W>(a, p, s); });
        if (e != cudaSuccess) return e;
        *nlaunch += 1;
    }
    return launch_sum_rows(a.part, (int)p.rows, (int64_t)a.D * (a.W + 1), a.dw, (int64_t)a.D * a.W, a.dbias, a.D, nullptr, s,
                           nlaunch);
}

}  // namespace qd
