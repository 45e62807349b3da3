// Pieces of the selective scan's forward and backward: how channels and tokens are shared
// out, and the staging of a tile of tokens from global to shared memory.
#pragma once

#include "layer_common.cuh"

namespace qd {
namespace ssm {

constexpr int kThreads = 256;
constexpr int kTile = 32;             // tokens of one shared-memory tile of the forward

__host__ __device__ constexpr int padded_states(int N) { return N <= 8 ? 8 : N <= 16 ? 16 : N <= 32 ? 32 : N <= 64 ? 64 : 128; }
__host__ __device__ constexpr int lanes_for(int N) { return N <= 8 ? 2 : N <= 32 ? 4 : 8; }

// Channel blocks never cross a group of channels that share B and C.
__host__ __device__ inline int channel_blocks(int D, int G, int CPB) { return G * ((D / G + CPB - 1) / CPB); }

struct ChannelBlock {
    int group, first, count;          // its group, its first channel and how many it has
    __device__ __forceinline__ ChannelBlock(const SsmArgs &a, int block, int CPB) {
        const int per = a.D / a.G, nb = (per + CPB - 1) / CPB;
        group = block / nb;
        const int at = (block % nb) * CPB;
        first = group * per + at;
        count = min(CPB, per - at);
    }
};

// Tokens cut into S segments of `len` (a multiple of the tile): one when `ctas` CTAs already
// number `enough`, else about `want` CTAs in all, of at least `least` tokens.
struct Split {
    int S, len;
};
inline Split split_tokens(int64_t ctas, int T, int64_t enough, int64_t want, int least) {
    Split s{1, T > 0 ? T : 1};
    if (ctas <= 0 || ctas >= enough) return s;
    int64_t S = want / ctas, most = T / least;
    if (S > most) S = most;
    if (S < 2) return s;
    s.len = (int)(((T + S - 1) / S + kTile - 1) / kTile * kTile);
    s.S = (T + s.len - 1) / s.len;
    return s;
}

__device__ __forceinline__ int seq_len(const int *lens, int b, int T) { return lens ? min(max(lens[b], 0), T) : T; }

// A forward tile.  Each thread moves PER accesses of x and of delta (VEC channels of a token)
// and GPER of B and C together; what is beyond the sequence, the block's channels or N is
// staged as zero, so that padding leaves the state unchanged (a = 1, u x B = 0) whatever the
// padded values are.
template <typename T, int LN, int SPL, bool WIDE> struct Geo {
    static constexpr int CPB = kThreads / LN, NP = LN * SPL;
    static constexpr int VEC = WIDE ? 16 / (int)sizeof(T) : 1;
    static constexpr int ROW = CPB / VEC;                              // accesses a token
    static constexpr int PER = (kTile * ROW + kThreads - 1) / kThreads;
    static constexpr int GROW = NP / VEC, GALL = 2 * kTile * GROW;     // accesses a token of B; of both
    // prefetched in registers when they are wide; one by one, straight to shared memory, otherwise
    static constexpr int GPER = WIDE ? (GALL + kThreads - 1) / kThreads : 1;
    using Vec = Pack<T, VEC>;

    struct Stage {
        Vec x[PER], dl[PER], g[GPER];

        __device__ __forceinline__ void load(const SsmArgs &a, const ChannelBlock &cb, int b, int t0, int n, bool both) {
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int e = threadIdx.x + i * kThreads, t = e / ROW, c = e % ROW * VEC;
                x[i].zero();
                dl[i].zero();
                if (t < kTile && t0 + t < n && c < cb.count) {
                    const size_t at = ((size_t)b * a.T + t0 + t) * a.D + cb.first + c;
                    x[i].load((const T *)a.x + at);
                    dl[i].load((const T *)a.delta + at);
                }
            }
            if constexpr (WIDE) {
#pragma unroll
                for (int i = 0; i < GPER; ++i) {
                    const int e = threadIdx.x + i * kThreads, which = e / (kTile * GROW), r = e % (kTile * GROW);
                    const int t = r / GROW, k = r % GROW * VEC;
                    g[i].zero();
                    if (e < (both ? GALL : GALL / 2) && t0 + t < n && k < a.N)
                        g[i].load((const T *)(which ? a.Cm : a.Bm) + (((size_t)b * a.T + t0 + t) * a.G + cb.group) * a.N + k);
                }
            }
        }
        __device__ __forceinline__ void store_tokens(const SsmArgs &a, const ChannelBlock &cb, int t0, int n, float2 *su) const {
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int e = threadIdx.x + i * kThreads, t = e / ROW, c = e % ROW * VEC;
                if (t >= kTile) break;
                float xf[VEC], df[VEC];
                x[i].get(xf);
                dl[i].get(df);
#pragma unroll
                for (int k = 0; k < VEC; ++k) {
                    float u = 0.f;
                    if (t0 + t < n && c + k < cb.count) {
                        u = df[k] + (a.delta_bias ? a.delta_bias[cb.first + c + k] : 0.f);
                        if (a.softplus) u = softplus_f(u);
                    }
                    su[t * CPB + c + k] = make_float2(u, u * xf[k]);
                }
            }
        }
        __device__ __forceinline__ void store_groups(const SsmArgs &a, const ChannelBlock &cb, int b, int t0, int n, float *sB,
                                                     float *sC, bool both) const {
            if constexpr (WIDE) {
#pragma unroll
                for (int i = 0; i < GPER; ++i) {
                    const int e = threadIdx.x + i * kThreads, which = e / (kTile * GROW), r = e % (kTile * GROW);
                    if (e >= (both ? GALL : GALL / 2)) break;
                    float f[VEC];
                    g[i].get(f);
                    float *to = (which ? sC : sB) + r * VEC;
#pragma unroll
                    for (int k = 0; k < VEC; k += 4) *reinterpret_cast<float4 *>(to + k) = make_float4(f[k], f[k + 1], f[k + 2], f[k + 3]);
                }
            } else {
                for (int e = threadIdx.x; e < (both ? 2 : 1) * kTile * NP; e += kThreads) {
                    const int which = e / (kTile * NP), r = e % (kTile * NP), t = r / NP, k = r % NP;
                    float f = 0.f;
                    if (t0 + t < n && k < a.N)
                        f = to_f(((const T *)(which ? a.Cm : a.Bm))[(((size_t)b * a.T + t0 + t) * a.G + cb.group) * a.N + k]);
                    (which ? sC : sB)[r] = f;
                }
            }
        }
    };

    // y = the staged sums + D x, zero on padding; `any` false: the whole tile is padding.
    __device__ __forceinline__ static void write_y(const SsmArgs &a, const ChannelBlock &cb, int b, int t0, int t_end, int n,
                                                   bool any, const Vec (&xk)[PER], const float *sy, int YS) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = threadIdx.x + i * kThreads, t = e / ROW, c = e % ROW * VEC;
            if (t >= kTile || t0 + t >= t_end || c >= cb.count) continue;
            float f[VEC];
#pragma unroll
            for (int k = 0; k < VEC; ++k) f[k] = 0.f;
            if (any && t0 + t < n) {
                float xf[VEC];
                xk[i].get(xf);
#pragma unroll
                for (int k = 0; k < VEC; ++k)
                    f[k] = sy[t * YS + c + k] + (a.Dskip ? a.Dskip[cb.first + c + k] * xf[k] : 0.f);
            }
            Vec v;
            v.set(f);
            v.store((T *)a.y + ((size_t)b * a.T + t0 + t) * a.D + cb.first + c);
        }
    }
};

}  // namespace ssm
}  // namespace qd
