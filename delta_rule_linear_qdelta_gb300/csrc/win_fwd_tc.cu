// Windowed attention's forward on the sm_103a tensor cores (bf16; tcgen05, TMEM, TMA).  The mathematics is
// win_attn_simt.cu's: running maximum and sum over the key tiles that a query tile sees.
//
// A CTA has two tiles of 128 queries -- two heads that share a key head where their number is even (both see the
// same keys), else two consecutive blocks of one head -- and walks the union of their key tiles, 128 keys each.
//   warps 0-7, 8-15   softmax of tile 0, 1: two threads a row (a TMEM lane), 64 columns each; S to P in place
//   warp 16           TMA: Q once, then K and V tiles through a ring
//   warps 17, 18      the products of tile 0, 1: S_t(i) = Q_t K_i^T and O_t += P_t(i) V_i; while one tile's softmax runs, the
//                     tensor core has the other tile's products
// TMEM: S_0, S_1 (128 fp32 columns each; P packed over the first half of each thread's columns), O_0, O_1 (DP columns each).
//
// The running maximum of a row is renewed only when a score passes it by more than 2^8 (P then stays below 2^8, in
// bf16 as exact as below 1, and sums are fp32): the rescaling of O, a round trip through TMEM that has to wait for
// the products under way, is rare after the first tiles.
//
// Bound by the tensor core: 4 d flop a pair of a query and a key in the tiles, of which a window of W keys needs
// W / (W + 128).  (A tile of up to 32 sinks is taken as one of 32 keys.)  Measured: 8 x 2048 tokens, 16 heads on 4, window 512, 4
// sinks: 107 us (565 TFLOP/s of what is seen, 29 % of the measured rate); 1 x 32768, window 2048: 468 us (1.14 PFLOP/s, 59 %).
// At the first of them issue slots are 42 % busy, tensor cores 37 %, the exponential unit 20 %: what is left is the latency of
// the chain scores, softmax, product over the five or six tiles of a CTA's walk, its start and its way out.
//
// Every wait is bounded; on a timeout the kernel sets its error word, waits (bounded) for its own copies and
// products, frees TMEM and returns.
#include "mix_tc.cuh"

namespace qd {

__device__ unsigned int g_win_fwd_timeout = 0;

namespace {

using namespace mix;

constexpr int kThreads = 608, kLoader = 512, kIssueWarp = 17;
constexpr uint32_t TM_S = 0, TM_O = 256;
constexpr float kSlack = 8.f;                               // log2 of what a probability may pass 1 by

template <int DP> struct Layout {
    static constexpr uint32_t kTile = DP / 64 * kPanel;
    static constexpr int kSlots = DP == 128 ? 5 : 8;
    static constexpr uint32_t kRing = 2 * kTile, kRest = kRing + kSlots * kTile, kBytes = kRest + 2560;
};

struct Params {
    const int *lens;
    float *lse;
    int B, T, past, H, Hkv, d, window, sinks, blocks, by_head, together;
    float scale;
};

template <int DP>
__global__ void __launch_bounds__(kThreads, 1)
win_fwd_tc_kernel(const Params p, const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                  const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mo) {
    typedef Layout<DP> L;
    extern __shared__ __align__(1024) uint8_t sm[];         // Q_0 | Q_1 | ring of K_0, V_0, K_1, .. | the rest
    struct Rest {
        float other[2][2][kRows];                           // of a row's two threads: maxima, sums
        uint64_t q, full[L::kSlots], free[L::kSlots], s[2], p[2], o[2], turn[2], done[2];
        uint32_t tmem;
        int abort;
    };
    Rest &rest = *reinterpret_cast<Rest *>(sm + L::kRest);
    static_assert(L::kRest + sizeof(Rest) <= L::kBytes && L::kBytes <= 232448, "shared memory");
    auto &other = rest.other;
    auto &bar_full = rest.full, &bar_free = rest.free;
    auto &bar_s = rest.s, &bar_p = rest.p, &bar_o = rest.o, &bar_turn = rest.turn, &bar_done = rest.done;
    uint64_t &bar_q = rest.q;
    uint32_t &tmem_base = rest.tmem;
    int &abort_flag = rest.abort;
    if (smem_u32(sm) & 1023) {                              // (the swizzle's alignment; shared memory starts on it)
        if (threadIdx.x == 0) atomicExch(&g_win_fwd_timeout, 1u);
        return;
    }

    const int tid = threadIdx.x, warp = uniform(tid >> 5);
    // which tiles: heads of a key head next to each other (they share its tiles in L2), later blocks first (where
    // the window does not cut, they have the most keys); of all streams together, or stream by stream
    const int r = p.H / p.Hkv, per = p.by_head ? r / 2 : r, nblocks = p.by_head ? p.blocks : (p.blocks + 1) / 2;
    int u = blockIdx.x;
    const int pair = u % per;
    u /= per;
    const int streams = p.B * p.Hkv, blk = nblocks - 1 - (p.together ? u / streams : u % nblocks);
    u = p.together ? u % streams : u / nblocks;
    const int hk = u % p.Hkv, b = u / p.Hkv;
    const int n = real_tokens(p.lens, b, p.T), keys = p.past + n;
    const int head0 = hk * r + (p.by_head ? 2 * pair : pair), head1 = head0 + p.by_head;
    const int first0 = (p.by_head ? blk : 2 * blk) * kRows, first1 = p.by_head ? first0 : first0 + kRows;

    if (first0 >= n) {                                      // nothing but padding
        for (int t = 0; t < 2; ++t) {
            const int t0 = t ? first1 : first0, h = t ? head1 : head0, rows = min(kRows, p.T - t0);
            if (tid < rows && p.lse) p.lse[((size_t)b * p.T + t0 + tid) * p.H + h] = 0.f;
        }
        for (int i = tid; i < (int)(2 * L::kTile / 16); i += kThreads) reinterpret_cast<uint4 *>(sm)[i] = make_uint4(0u, 0u, 0u, 0u);
        fence_proxy_async();
        __syncthreads();
        if (tid == 0) {
            store_tile<DP>(&mo, sm, head0, first0, b);
            if (first1 < p.T) store_tile<DP>(&mo, sm + L::kTile, head1, first1, b);
            tma_store_commit();
            tma_store_wait_read0();
        }
        return;
    }
    // the key tiles: [0, early) and [from, from + count - early)
    const int last = min(n, (p.by_head ? first0 : first1) + kRows) - 1;
    const int from = max(0, p.past + first0 - p.window + 1) / kRows, to = (p.past + last) / kRows + 1;
    const int early = min((int)(((unsigned)p.sinks + kRows - 1) / kRows), from), count = early + to - from;
    auto key0 = [&](int i) { return (i < early ? i : from + i - early) * kRows; };

    if (tid == 0) {
        mbar_init(&bar_q, 1);
        for (int i = 0; i < L::kSlots; ++i) {
            mbar_init(&bar_full[i], 1);
            mbar_init(&bar_free[i], 2);                     // (both tiles' products)
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(&bar_s[t], 1);
            mbar_init(&bar_p[t], 256);
            mbar_init(&bar_o[t], 1);
            mbar_init(&bar_turn[t], 1);
            mbar_init(&bar_done[t], 1);
        }
        abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 0) {
        tmem_alloc(&tmem_base, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = tmem_base;

    int loaded = 0;                                         // ring loads issued (the loader's)
    if (tid == kLoader) {
        mbar_arrive_expect_tx(&bar_q, 2 * L::kTile);
        load_tile<DP>(sm, &mq, &bar_q, head0, first0, b);
        load_tile<DP>(sm + L::kTile, &mq, &bar_q, head1, first1, b);
        for (int i = 0; i < 2 * count; ++i, ++loaded) {     // K_0, V_0, K_1, V_1, ..
            const int slot = i % L::kSlots;
            if (i >= L::kSlots && !one_wait(&bar_free[slot], (i / L::kSlots - 1) & 1, &abort_flag)) break;
            mbar_arrive_expect_tx(&bar_full[slot], L::kTile);
            load_tile<DP>(sm + L::kRing + slot * L::kTile, i & 1 ? &mv : &mk, &bar_full[slot], hk, key0(i >> 1), b);
        }
    } else if (warp == kIssueWarp || warp == kIssueWarp + 1) {
        const int t = warp - kIssueWarp;
        const uint32_t base = smem_u32(sm), q = base + t * L::kTile, S = tm + TM_S + 128 * t;
        const bool leader = elect_one();
        auto tile = [&](int i) { return base + L::kRing + (i % L::kSlots) * L::kTile; };
        auto arrived = [&](int i) { return warp_wait(&bar_full[i % L::kSlots], (i / L::kSlots) & 1, &abort_flag); };
        // the tiles take turns, so that one's products run while the other's softmax does: turn k of tile 1 follows tile 0's,
        // that of tile 0 tile 1's before
        auto my_turn = [&](int k) { return t ? warp_wait(&bar_turn[1], k & 1, &abort_flag) : k == 0 || warp_wait(&bar_turn[0], (k - 1) & 1, &abort_flag); };
        auto next_turn = [&]() { if (leader) mbar_arrive(&bar_turn[t ^ 1]); };
        const bool few = early == 1 && p.sinks <= 32;       // the first tile: few sinks, its first 32 keys
        auto issue_s = [&](int i) {
            const uint64_t a = desc_rows(q), x = desc_rows(tile(2 * i));
            const uint32_t shape = few && i == 0 ? idesc_bf16(128, 32, false, false) : idesc_bf16(128, 128, false, false);
            if (leader) {
#pragma unroll
                for (int k = 0; k < DP / 16; ++k) umma_bf16(S, a + step_rows(k), x + step_rows(k), shape, k > 0);
            }
            commit(leader, &bar_s[t]);
            commit(leader, &bar_free[2 * i % L::kSlots]);
        };
        bool ok = warp_wait(&bar_q, 0, &abort_flag) && arrived(0) && my_turn(0);
        if (ok) {
            issue_s(0);
            next_turn();
        }
        for (int i = 0; ok && i < count; ++i) {
            const int vi = 2 * i + 1;
            ok = arrived(vi) && (i + 1 == count || arrived(vi + 1)) && warp_wait(&bar_p[t], i & 1, &abort_flag) && my_turn(i + 1);
            if (!ok) break;
            tc_fence_after();
            const uint64_t v = desc_cols(tile(vi));
            if (leader) {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (k < 2 || !few || i > 0)
                        umma_bf16_ta(tm + TM_O + DP * t, S + step_halves(k), v + step_cols(k), idesc_bf16(128, DP, false, true), k > 0 || i > 0);
            }
            commit(leader, &bar_o[t]);
            commit(leader, &bar_free[vi % L::kSlots]);
            if (i + 1 < count) issue_s(i + 1);              // (over P, which the product above reads before)
            next_turn();
        }
        commit(leader, &bar_done[t]);
    } else if (tid < 512) {
        const int t = warp >> 3, half = (warp >> 2) & 1, row = tid & 127, t0 = t ? first1 : first0, head = t ? head1 : head0;
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t sS = tm + TM_S + 128 * t + 64 * half + lanes, sO = tm + TM_O + DP * t + DP / 2 * half + lanes;
        const int pos = p.past + t0 + row;
        const float c = p.scale * kLog2e;
        float m = -INFINITY, l = 0.f;                       // of this row, in log2 units; of this thread's columns
        bool ok = true;
        for (int i = 0; i < count; ++i) {
            const int j0 = key0(i);
            ok = warp_wait(&bar_s[t], i & 1, &abort_flag);
            tc_fence_after();
            float s[64];
            tmem_ld32(sS, *reinterpret_cast<float(*)[32]>(s));
            tmem_ld32(sS + 32, *reinterpret_cast<float(*)[32]>(s + 32));
            tmem_ld_wait();
            // every row of the tile sees every key of the tile: its scores are only scaled
            const bool inner = j0 + kRows - 1 <= p.past + t0 && (p.past + t0 + kRows - 1 - j0 < p.window || j0 + kRows - 1 < p.sinks);
            float ce = c, top = -INFINITY;
            if (inner) {
                float best[4];                              // (four short chains)
                if (c >= 0.f) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) best[k] = fmaxf(s[k], s[k + 4]);
#pragma unroll
                    for (int j = 8; j < 64; j += 8)
#pragma unroll
                        for (int k = 0; k < 4; ++k) best[k] = fmaxf(best[k], fmaxf(s[j + k], s[j + k + 4]));
                    top = fmaxf(fmaxf(best[0], best[1]), fmaxf(best[2], best[3]));
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k) best[k] = fminf(s[k], s[k + 4]);
#pragma unroll
                    for (int j = 8; j < 64; j += 8)
#pragma unroll
                        for (int k = 0; k < 4; ++k) best[k] = fminf(best[k], fminf(s[j + k], s[j + k + 4]));
                    top = fminf(fminf(best[0], best[1]), fminf(best[2], best[3]));
                }
                top *= c;
            } else {
                const int hi = pos - j0, lo = max(0, pos - p.window + 1) - j0, early_hi = min(hi, p.sinks - 1 - j0);
                ce = 1.f;
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    // bits of this thread's columns 32 w .. 32 w + 31 that the row sees: [lo, hi] and [0, early_hi]
                    auto upto = [&](int x) { x -= 64 * half + 32 * w; return x < 0 ? 0u : x >= 31 ? ~0u : (2u << x) - 1u; };
                    const uint32_t bits = (upto(hi) & ~upto(lo - 1)) | upto(early_hi);
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        s[32 * w + j] = (bits >> j) & 1u ? c * s[32 * w + j] : -INFINITY;
                        top = fmaxf(top, s[32 * w + j]);
                    }
                }
            }
            // the tile's 256 threads agree on whether anything has to be renewed (or ended)
            if (tc::named_sync_or(1 + t, 256, top > m + kSlack || (m == -INFINITY && top > m) || !ok)) {
                other[t][half][row] = top;
                if (i > 0 && ok) ok = warp_wait(&bar_o[t], (i - 1) & 1, &abort_flag);
                if (tc::named_sync_or(1 + t, 256, !ok)) {
                    ok = false;
                    break;
                }
                top = fmaxf(top, other[t][half ^ 1][row]);
                const bool renew = top > m + kSlack || (m == -INFINITY && top > m);
                const float f = renew ? exp2_fast(m - top) : 1.f;
                if (renew) m = top;
                l *= f;
                if (i > 0) {
                    tc_fence_after();
#pragma unroll 1
                    for (int k = 0; k < DP / 32; ++k) {
                        float o[16];
                        tmem_ld16(sO + 16 * k, o);
                        tmem_ld_wait();
#pragma unroll
                        for (int j = 0; j < 16; ++j) o[j] *= f;
                        tmem_st16(sO + 16 * k, reinterpret_cast<const uint32_t(&)[16]>(o));
                    }
                }
            }
            const float base = m == -INFINITY ? 0.f : -m;   // (nothing seen yet)
            const f32x2 ce2 = pk(ce, ce), base2 = pk(base, base);
            f32x2 sum[2] = {pk(0.f, 0.f), pk(0.f, 0.f)};
#pragma unroll
            for (int part = 0; part < 2; ++part) {
                uint32_t packed[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const f32x2 e = exp2_2(fma2(pk(s[32 * part + 2 * j], s[32 * part + 2 * j + 1]), ce2, base2));
                    sum[j & 1] = add2(sum[j & 1], e);
                    float e0, e1;
                    unpk(e, e0, e1);
                    packed[j] = pack_bf16x2(e0, e1);        // probabilities in bf16, as their products' other factor
                }
                tmem_st16(sS + 16 * part, packed);
            }
            l += sum2(add2(sum[0], sum[1]));
            if (j0 + kRows > keys && keys < p.past + p.T) {
                // rows of V behind the last key are padding, whatever they hold: 0 times them has to be 0
                const int vi = 2 * i + 1, slot = vi % L::kSlots;
                ok = warp_wait(&bar_full[slot], (vi / L::kSlots) & 1, &abort_flag);
                if (j0 + row >= keys)
#pragma unroll
                    for (int k = 0; k < DP / 16; ++k) {
                        const int chunk = DP / 16 * half + k;
                        *reinterpret_cast<uint4 *>(sm + L::kRing + slot * L::kTile + (chunk >> 3) * kPanel + row * 128 + (chunk & 7) * 16) =
                            make_uint4(0u, 0u, 0u, 0u);
                    }
                fence_proxy_async();
            }
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive(&bar_p[t]);
        }
        if (ok) ok = warp_wait(&bar_o[t], (count - 1) & 1, &abort_flag);
        other[t][half][row] = l;
        named_sync(1 + t, 256);
        l += other[t][half ^ 1][row];
        const bool real = t0 + row < n;
        if (ok) {
            tc_fence_after();
            const float inv = real ? 1.f / l : 0.f;
#pragma unroll 1
            for (int k = 0; k < DP / 64; ++k) {             // into the tile's Q, which the last S has read
                float o[32];
                const int c0 = DP / 2 * half + 32 * k;
                tmem_ld32(sO + 32 * k, o);
                tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 32; ++j) o[j] = real ? o[j] * inv : 0.f;
#pragma unroll
                for (int j = 0; j < 32; j += 8)
                    *reinterpret_cast<uint4 *>(sm + t * L::kTile + (c0 >> 6) * kPanel + sw128_off(row, (c0 & 63) + j)) = tc::pack8p(o + j);
            }
            if (half == 0 && p.lse && t0 + row < p.T)
                p.lse[((size_t)b * p.T + t0 + row) * p.H + head] = real ? kLn2 * (m + __log2f(l)) : 0.f;
        }
        fence_proxy_async();
        named_sync(1 + t, 256);
        if ((tid & 255) == 0 && t0 < p.T && !*reinterpret_cast<volatile int *>(&abort_flag)) {
            store_tile<DP>(&mo, sm + t * L::kTile, head, t0, b);
            tma_store_commit();
            tma_store_wait_read0();
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (abort_flag) {
        if (tid == kLoader) {                               // its copies: the last of each slot
            mbar_wait(&bar_q, 0, kWaitNs);
            for (int i = max(0, loaded - L::kSlots); i < loaded; ++i) mbar_wait(&bar_full[i % L::kSlots], (i / L::kSlots) & 1, kWaitNs);
        }
        if (warp == kIssueWarp && elect_one()) {
            mbar_wait(&bar_done[0], 0, kWaitNs);            // (committed behind all the products)
            mbar_wait(&bar_done[1], 0, kWaitNs);
            atomicExch(&g_win_fwd_timeout, 1u);
        }
        __syncwarp();
        __syncthreads();
    }
    if (warp == 0) tmem_dealloc(tm, 512);
}

template <int DP> cudaError_t run(const WinArgs &a, cudaStream_t s) {
    CUtensorMap mq, mk, mv, mo;
    const int keys = a.past + a.T;
    if (!token_map(&mq, a.q, a.B, a.T, a.H, a.d) || !token_map(&mk, a.k, a.B, keys, a.Hkv, a.d) ||
        !token_map(&mv, a.v, a.B, keys, a.Hkv, a.d) || !token_map(&mo, a.o, a.B, a.T, a.H, a.d))
        return cudaErrorInvalidValue;
    constexpr int bytes = Layout<DP>::kBytes;
    const cudaError_t e = cudaFuncSetAttribute(win_fwd_tc_kernel<DP>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    const int r = a.H / a.Hkv;
    Params p{a.lens, a.lse, a.B, a.T, a.past, a.H, a.Hkv, a.d, a.window, a.sinks, (a.T + kRows - 1) / kRows, r % 2 == 0,
             blocks_together(a), a.scale};
    const size_t pairs = p.by_head ? (size_t)p.blocks * (r / 2) : (size_t)((p.blocks + 1) / 2) * r;
    win_fwd_tc_kernel<DP><<<(unsigned)(a.B * a.Hkv * pairs), kThreads, bytes, s>>>(p, mq, mk, mv, mo);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_win_fwd_tc(const WinArgs &a, cudaStream_t s, int *n) {
    const cudaError_t e = a.d > 64 ? run<128>(a, s) : run<64>(a, s);
    if (e == cudaSuccess) *n += 1;
    return e;
}

bool win_fwd_read_and_clear_timeout() {
    unsigned int v = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&v, g_win_fwd_timeout, sizeof v) != cudaSuccess) return false;
    if (v) cudaMemcpyToSymbol(g_win_fwd_timeout, &zero, sizeof zero);
    return v != 0;
}

}  // namespace qd
