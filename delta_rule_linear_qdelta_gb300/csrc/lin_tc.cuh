// What the tensor-core kernels of linear attention share: the decays of a chunk of 128 tokens.
#pragma once

#include "mix_tc.cuh"

namespace qd {
namespace mix {

constexpr int kBlock = 32, kBlocks = kRows / kBlock;
// Below this sum of log decays over a chunk its decays are not factored.  The factors go up to its exp(): 2^58, which leaves products
// of inputs (and their sums) from 2^-68 to 2^70 inside the range of the types.  At -64, gradients of 2^56 were NaN and outputs of
// 2^-56 lost.  Decays of -0.4 a token, which fall between: 8 x 2048 tokens of 16 heads 59 us with factors, 70 without; the
// backward of 4 x 4096, 8 heads, 150 and 176.
constexpr float kLight = -40.f;

// The decays of one chunk in shared memory.  In a light chunk (no dropping token, not too strong) the weight of token
// j in token i's output factors, exp(P_i - P_j) = exp(P_i - P_end) exp(P_end - P_j), and the second factor, at most 1, is
// the one with which token j enters the state: weights cost one product a pair and outputs one a value.
struct alignas(16) Gates {
    float P[kRows];           // sums of the log decays from the chunk's start, times log2 e (dropping tokens add nothing)
    float write[kRows];       // the walk's factor: exp(P_end - P_j), 0 if dropped in between; walked backwards exp(P_j)
    unsigned char seen[kRows];// 0: token i sees the entering state; else one more than the first token it sees
    float total;              // across the chunk
    int light;
};

// One warp's share of the decays of a chunk, tokens 4 lane .. 4 lane + 3, before they are stored.
struct LaneGates {
    float x[4];               // log decays, then P
    float write[4], total;
    unsigned seen;            // four bytes
    int light;

    __device__ __forceinline__ void load(const void *g, int g_token, size_t row0, int t0, int n, int H, int h) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int t = t0 + 4 * (threadIdx.x & 31) + u;
            x[u] = g && t < n ? (g_token ? to_f(static_cast<const __nv_bfloat16 *>(g)[(row0 + t) * H + h]) : static_cast<const float *>(g)[h]) : 0.f;
        }
    }
    // Sums from the chunk's start, and for the factors of a forward walk from its end: a factor is then as exact as its own
    // exponent, however large the sums before.  A pair's, exp(P_i - P_j), is as exact as the sums: 3e-5 at worst with half to one and
    // a half nats a token, 2e-4 with up to ten, 3e-3 where most tokens of the chunk lose 86 each, just short
    // of dropping the state, and the last few nothing (in a simulation of these sums); its product is rounded to bf16, 2^-8.
    __device__ __forceinline__ void compute(bool back) {
        const int lane = threadIdx.x & 31;
        float own[4], sum = 0.f, rest[4];
        int last = -1, own_last[4];                         // the last dropping token
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            if (x[u] < kDrop) {
                last = 4 * lane + u;
                x[u] = 0.f;
            }
            sum += x[u];
            own[u] = sum;
            own_last[u] = last;
        }
        float upto = sum, from = sum;
        int last_upto = last;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const float v = __shfl_up_sync(0xffffffffu, upto, off), d = __shfl_down_sync(0xffffffffu, from, off);
            const int l = __shfl_up_sync(0xffffffffu, last_upto, off);
            if (lane >= off) {
                upto += v;
                last_upto = max(last_upto, l);
            }
            if (lane + off < 32) from += d;
        }
        const float all = __shfl_sync(0xffffffffu, upto, 31);
        const int drop = __shfl_sync(0xffffffffu, last_upto, 31);
        float before = __shfl_up_sync(0xffffffffu, upto, 1), after = __shfl_down_sync(0xffffffffu, from, 1);
        int last_before = __shfl_up_sync(0xffffffffu, last_upto, 1);
        if (lane == 0) before = 0.f, last_before = -1;
        if (lane == 31) after = 0.f;
#pragma unroll
        for (int u = 3; u >= 0; --u) {
            rest[u] = after;
            after += x[u];
        }
        seen = 0;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int i = 4 * lane + u, l = max(last_before, own_last[u]);
            const float P = before + own[u];
            x[u] = P * kLog2e;
            write[u] = back ? (l < 0 ? expf(P) : 0.f) : (i >= drop ? expf(rest[u]) : 0.f);
            seen |= (unsigned)(l + 1) << (8 * u);
        }
        total = drop < 0 ? expf(all) : 0.f;
        light = drop < 0 && all > kLight;
    }
    __device__ __forceinline__ void store(Gates &s) const {
        const int lane = threadIdx.x & 31;
        *reinterpret_cast<float4 *>(s.P + 4 * lane) = make_float4(x[0], x[1], x[2], x[3]);
        *reinterpret_cast<float4 *>(s.write + 4 * lane) = make_float4(write[0], write[1], write[2], write[3]);
        *reinterpret_cast<unsigned *>(s.seen + 4 * lane) = seen;
        if (lane == 0) s.total = total, s.light = light;
    }
};

}  // namespace mix
}  // namespace qd
