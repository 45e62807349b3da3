// Windowed attention's backward on the sm_103a tensor cores (bf16; tcgen05, TMEM, TMA).  The mathematics is
// win_attn_simt.cu's; probabilities come from the forward's lse.  Two kernels, so that every sum has one owner and needs
// no atomic: seven products of 128 x 128 x d a pair of tiles in the place of five.
//
// Both: warps 0-15 take the four quarters of a tile's columns (a thread: a row, 32 columns); warp 16 TMA; warps 17 and 18 the
// products, of which those of one chain come from one of them, in order; the second kernel's warp 19 the rows' lse and D.
//
//   dq    a CTA has 128 queries of a head.  S = Q K^T, dP = dO V^T, dS = P (dP - D) packed over S, dQ += dS K.  S of the next
//         tile but one waits in the second of two places; D = rowsum(dO . o) is formed first and left in the workspace.
//         TMEM: S 0-255, dP 256-383, dQ 384-511.
//   dk dv a CTA has 128 keys of a key head and walks the heads that share it and the queries that see them, with the lanes
//         along the keys: S^T = K Q^T, P^T packed over it, dV += P^T dO (one chain); dP^T = V dO^T, dS^T over it, dK += dS^T Q
//         (the other).  TMEM: S^T 0-127, dP^T 128-255, dV 256-383, dK 384-511.
//
// Tiles of sinks are seen by every later query: those beyond the tile's window are cut into slices of their own CTAs, which
// leave fp32 parts of the sinks' rows to be summed in order (win_sinks_kernel); more than two tiles of sinks are not cut.  Walks that are long for the number of SMs are
// cut into pieces, summed likewise (win_pieces_kernel).
//
// Bound by the tensor core: 14 d flop a pair of the tiles.  4 x 4096 tokens, 8 heads on 2, window 1024, 4 sinks: 253 us (597
// TFLOP/s of the 10 d a pair that is seen), of which under a profiler dq has 115, dk dv 132, the sinks' sums 6; tensor cores
// active 47 and 64 %.
//
// Every wait is bounded; on a timeout the kernel sets its error word, waits (bounded) for its own copies and products,
// frees TMEM and returns.
#include "mix_tc.cuh"

#include <algorithm>

namespace qd {

__device__ unsigned int g_win_bwd_timeout = 0;

namespace {

using namespace mix;

constexpr int kWorkers = 512, kLoader = 512, kIssueWarp = 17, kStatWarp = 19, kThreadsQ = 608, kThreadsK = 640;
constexpr int kMostSlices = 64;

struct Params {
    const float *lse;
    const int *lens;
    float *delta, *parts, *pieces; // [B][T][H]; [B][Hkv][sink tile][slice][128][2][d]; [piece][B][past + T][Hkv][2][d]
    int B, T, past, H, Hkv, d, window, sinks, blocks, key_tiles, sink_tiles, slices, near, together;
    float scale;
};

template <int DP> struct Layout {
    static constexpr uint32_t kTile = DP / 64 * kPanel;
    static constexpr int kSlots = DP == 128 ? 5 : 8;
    static constexpr uint32_t kRing = 2 * kTile, kRest = kRing + kSlots * kTile, kBytes = kRest + 2560;
    static_assert(kBytes <= 232448, "shared memory");
};

// Bits of the columns 32 w .. 32 w + 31 that lie in [lo, hi].
__device__ __forceinline__ uint32_t bits_between(int lo, int hi, int w) {
    auto upto = [&](int x) { return x < 32 * w ? 0u : x >= 32 * w + 31 ? ~0u : (2u << (x - 32 * w)) - 1u; };
    return upto(hi) & ~upto(lo - 1);
}

// 32 probabilities' gradients, packed: dS = P (dP - D), 0 where P is (whatever the other factor).
__device__ __forceinline__ uint32_t pack_ds(float p0, float p1, float d0, float d1) {
    return pack_bf16x2(p0 == 0.f ? 0.f : p0 * d0, p1 == 0.f ? 0.f : p1 * d1);
}

template <int DP>
__global__ void __launch_bounds__(kThreadsQ, 1)
win_dq_tc_kernel(const Params p, const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                 const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap md,
                 const __grid_constant__ CUtensorMap mo, const __grid_constant__ CUtensorMap mdq) {
    typedef Layout<DP> L;
    constexpr uint32_t TM_S = 0, TM_DP = 256, TM_DQ = 384;
    extern __shared__ __align__(1024) uint8_t sm[];         // Q | dO | ring of K_0, V_0, K_1, .. | the rest
    struct Rest {
        float part[4][kRows];                               // of the rows' D
        uint64_t qd, full[L::kSlots], free[L::kSlots], s[2], dp, ds, dq[2], o, all[2];
        uint32_t tmem;
        int abort;
    };
    Rest &rest = *reinterpret_cast<Rest *>(sm + L::kRest);
    static_assert(L::kRest + sizeof(Rest) <= L::kBytes, "shared memory");
    auto &bar_full = rest.full, &bar_free = rest.free;
    uint32_t &tmem_base = rest.tmem;
    int &abort_flag = rest.abort;
    if (smem_u32(sm) & 1023) {                              // (the swizzle's alignment; shared memory starts on it)
        if (threadIdx.x == 0) atomicExch(&g_win_bwd_timeout, 1u);
        return;
    }

    const int tid = threadIdx.x, warp = uniform(tid >> 5);
    const int r = p.H / p.Hkv;
    int u = blockIdx.x;
    const int head_in = u % r;
    u /= r;
    const int streams = p.B * p.Hkv, blk = p.blocks - 1 - (p.together ? u / streams : u % p.blocks);
    u = p.together ? u % streams : u / p.blocks;
    const int hk = u % p.Hkv, b = u / p.Hkv, h = hk * r + head_in, t0 = blk * kRows;
    const int n = real_tokens(p.lens, b, p.T), keys = p.past + n, rows = min(kRows, n - t0);
    const size_t tok = ((size_t)b * p.T + t0) * p.H + h;
    if (rows <= 0) {                                        // nothing but padding
        for (int i = tid; i < (int)(L::kTile / 16); i += kThreadsQ) reinterpret_cast<uint4 *>(sm)[i] = make_uint4(0u, 0u, 0u, 0u);
        fence_proxy_async();
        __syncthreads();
        if (tid == 0) {
            store_tile<DP>(&mdq, sm, h, t0, b);
            tma_store_commit();
            tma_store_wait_read0();
        }
        return;
    }
    const int from = max(0, p.past + t0 - p.window + 1) / kRows, to = (p.past + t0 + rows - 1) / kRows + 1;
    const int early = min((int)(((unsigned)p.sinks + kRows - 1) / kRows), from), count = early + to - from;
    auto key0 = [&](int i) { return (i < early ? i : from + i - early) * kRows; };

    if (tid == 0) {
        mbar_init(&rest.qd, 1);
        for (int i = 0; i < L::kSlots; ++i) {
            mbar_init(&bar_full[i], 1);
            mbar_init(&bar_free[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&rest.s[i], 1);
            mbar_init(&rest.dq[i], 1);
            mbar_init(&rest.all[i], 1);
        }
        mbar_init(&rest.dp, 1);
        mbar_init(&rest.ds, kWorkers);
        mbar_init(&rest.o, 1);
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
    const uint32_t tm = tmem_base, base = smem_u32(sm);
    auto ring = [](int i) { return (uint32_t)(i / L::kSlots) & 1u; };

    int loaded = 0;
    if (tid == kLoader) {
        mbar_arrive_expect_tx(&rest.qd, 3 * L::kTile);
        load_tile<DP>(sm, &mq, &rest.qd, h, t0, b);
        load_tile<DP>(sm + L::kTile, &md, &rest.qd, h, t0, b);
        load_tile<DP>(sm + L::kRing + (L::kSlots - 1) * L::kTile, &mo, &rest.qd, h, t0, b);   // o, in the ring's last place at first
        for (int i = 0; i < 2 * count; ++i, ++loaded) {     // K_0, V_0, K_1, ..
            const int slot = i % L::kSlots;
            if (i == L::kSlots - 1 && !one_wait(&rest.o, 0, &abort_flag)) break;
            if (i >= L::kSlots && !one_wait(&bar_free[slot], ring(i - L::kSlots), &abort_flag)) break;
            mbar_arrive_expect_tx(&bar_full[slot], L::kTile);
            load_tile<DP>(sm + L::kRing + slot * L::kTile, i & 1 ? &mv : &mk, &bar_full[slot], hk, key0(i >> 1), b);
        }
    } else if (warp == kIssueWarp || warp == kIssueWarp + 1) {
        const bool leader = elect_one(), second = warp > kIssueWarp;
        auto tile = [&](int i) { return base + L::kRing + (i % L::kSlots) * L::kTile; };
        auto arrived = [&](int i) { return warp_wait(&bar_full[i % L::kSlots], ring(i), &abort_flag); };
        bool ok = warp_wait(&rest.qd, 0, &abort_flag);
        if (!second) {                                      // S of every tile, into its place once dQ has read dS of the last but one
            for (int i = 0; ok && i < count; ++i) {
                ok = arrived(2 * i) && (i < 2 || warp_wait(&rest.dq[i & 1], ((i >> 1) - 1) & 1, &abort_flag));
                if (!ok) break;
                tc_fence_after();
                mma_rows_rows<DP, 128>(leader, tm + TM_S + 128 * (i & 1), base, tile(2 * i), false);
                commit(leader, &rest.s[i & 1]);
            }
        } else {
            // step i: dP(i), whose place has been read when dS(i - 1) is there, then dQ += dS(i - 1) K(i - 1)
            for (int i = 0; ok && i <= count; ++i) {
                ok = (i == count || arrived(2 * i + 1)) && (i == 0 || warp_wait(&rest.ds, (i - 1) & 1, &abort_flag));
                if (!ok) break;
                tc_fence_after();
                if (i < count) {
                    mma_rows_rows<DP, 128>(leader, tm + TM_DP, base + L::kTile, tile(2 * i + 1), false);
                    commit(leader, &rest.dp);
                    commit(leader, &bar_free[(2 * i + 1) % L::kSlots]);
                }
                if (i > 0) {
                    mma_tmem_cols<DP, 4>(leader, tm + TM_DQ, tm + TM_S + 128 * ((i - 1) & 1), tile(2 * i - 2), i > 1);
                    commit(leader, &rest.dq[(i - 1) & 1]);
                    commit(leader, &bar_free[(2 * i - 2) % L::kSlots]);
                }
            }
        }
        commit(leader, &rest.all[second]);
    } else if (tid < kWorkers) {
        const int quarter = warp >> 2, row = tid & 127;
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const bool real = row < rows;
        const int pos = p.past + t0 + row;
        const bool alone = sees_itself_alone(pos, p.window, p.sinks);
        const float c = p.scale * kLog2e, lse = real ? kLog2e * p.lse[tok + (size_t)row * p.H] : 0.f;
        bool ok = warp_wait(&rest.qd, 0, &abort_flag);
        {
            float t = 0.f;
#pragma unroll
            for (int k = 0; k < DP / 32; ++k) {             // this thread's quarter of the row of dO . o
                const int col = DP / 4 * quarter + 8 * k;
                const uint32_t at = (col >> 6) * kPanel + sw128_off(row, col & 63);
                float x[8], y[8];
                tc::unpack8(*reinterpret_cast<const uint4 *>(sm + L::kRing + (L::kSlots - 1) * L::kTile + at), x);
                tc::unpack8(*reinterpret_cast<const uint4 *>(sm + L::kTile + at), y);
#pragma unroll
                for (int e = 0; e < 8; ++e) t = fmaf(x[e], y[e], t);
            }
            rest.part[quarter][row] = t;
        }
        named_sync(1, kWorkers);
        if (tid == 0) mbar_arrive(&rest.o);                 // (the sums are formed: o has been read)
        const float delta = (rest.part[0][row] + rest.part[1][row]) + (rest.part[2][row] + rest.part[3][row]);
        if (quarter == 0 && real && ok) p.delta[tok + (size_t)row * p.H] = delta;
        for (int i = 0; ok && i < count; ++i) {
            const int j0 = key0(i);
            const uint32_t sS = tm + TM_S + 128 * (i & 1) + 32 * quarter + lanes;
            ok = warp_wait(&rest.s[i & 1], (i >> 1) & 1, &abort_flag);
            if (!ok) break;
            tc_fence_after();
            float s[32];
            tmem_ld32(sS, s);
            tmem_ld_wait();
            const f32x2 c2 = pk(c, c), l2 = pk(-lse, -lse);
#pragma unroll
            for (int j = 0; j < 32; j += 2) unpk(exp2_2(fma2(pk(s[j], s[j + 1]), c2, l2)), s[j], s[j + 1]);
            const bool inner = j0 + kRows - 1 <= p.past + t0 && (p.past + t0 + kRows - 1 - j0 < p.window || j0 + kRows - 1 < p.sinks);
            if (!inner) {
                const int hi = pos - j0, lo = max(0, pos - p.window + 1) - j0, early_hi = min(hi, p.sinks - 1 - j0);
                const uint32_t bits = bits_between(lo, hi, quarter) | bits_between(0, early_hi, quarter);
#pragma unroll
                for (int j = 0; j < 32; ++j) s[j] = (bits >> j) & 1u ? s[j] : 0.f;
            }
            ok = warp_wait(&rest.dp, i & 1, &abort_flag);
            if (!ok) break;
            tc_fence_after();
            uint32_t packed[16];
            float dp[32];
            tmem_ld32(tm + TM_DP + 32 * quarter + lanes, dp);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 32; j += 2) packed[j / 2] = pack_ds(s[j], s[j + 1], dp[j] - delta, dp[j + 1] - delta);
            tmem_st16(sS, packed);
            if (j0 + kRows > keys && keys < p.past + p.T) {
                // rows of K behind the last key are padding, whatever they hold: 0 times them has to be 0
                const int slot = (2 * i) % L::kSlots;
                if (j0 + row >= keys)
#pragma unroll
                    for (int k = 0; k < DP / 32; ++k) {
                        const int chunk = DP / 32 * quarter + k;
                        *reinterpret_cast<uint4 *>(sm + L::kRing + slot * L::kTile + (chunk >> 3) * kPanel + row * 128 + (chunk & 7) * 16) =
                            make_uint4(0u, 0u, 0u, 0u);
                    }
                fence_proxy_async();
            }
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive(&rest.ds);
        }
        ok = ok && warp_wait(&rest.all[1], 0, &abort_flag);
        if (ok) {
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < DP / 64; ++k) {             // this quarter's columns into Q's place, which S has read
                float x[16];
                const int c0 = DP / 4 * quarter + 16 * k;
                tmem_ld16(tm + TM_DQ + c0 + lanes, x);
                tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 16; ++j) x[j] = real && !alone ? p.scale * x[j] : 0.f;
#pragma unroll
                for (int j = 0; j < 16; j += 8)
                    *reinterpret_cast<uint4 *>(sm + (c0 >> 6) * kPanel + sw128_off(row, (c0 & 63) + j)) = tc::pack8p(x + j);
            }
        }
        fence_proxy_async();
        named_sync(1, kWorkers);
        if (tid == 0 && !*reinterpret_cast<volatile int *>(&abort_flag)) {
            store_tile<DP>(&mdq, sm, h, t0, b);
            tma_store_commit();
            tma_store_wait_read0();
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (abort_flag) {
        if (tid == kLoader) {
            mbar_wait(&rest.qd, 0, kWaitNs);
            for (int i = max(0, loaded - L::kSlots); i < loaded; ++i) mbar_wait(&bar_full[i % L::kSlots], ring(i), kWaitNs);
        }
        if (warp == kIssueWarp && elect_one()) {
            mbar_wait(&rest.all[0], 0, kWaitNs);            // (committed behind all the products)
            mbar_wait(&rest.all[1], 0, kWaitNs);
            atomicExch(&g_win_bwd_timeout, 1u);
        }
        __syncwarp();
        __syncthreads();
    }
    if (warp == 0) tmem_dealloc(tm, 512);
}

template <int DP>
__global__ void __launch_bounds__(kThreadsK, 1)
win_dkdv_tc_kernel(const Params p, const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                   const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap md,
                   const __grid_constant__ CUtensorMap mdk, const __grid_constant__ CUtensorMap mdv) {
    typedef Layout<DP> L;
    constexpr uint32_t TM_S = 0, TM_DP = 128, TM_DV = 256, TM_DK = 384;
    extern __shared__ __align__(1024) uint8_t sm[];         // K | V | ring of Q_0, dO_0, Q_1, .. | the rest
    struct Rest {
        float lse_of[2][kRows], delta_of[2][kRows];
        uint64_t kv, full[L::kSlots], free[L::kSlots], s, p, dp, ds, all[2], stat[2], sfree[2], clean[2];
        uint32_t tmem;
        int abort;
    };
    Rest &rest = *reinterpret_cast<Rest *>(sm + L::kRest);
    static_assert(L::kRest + sizeof(Rest) <= L::kBytes, "shared memory");
    auto &lse_of = rest.lse_of, &delta_of = rest.delta_of;
    uint64_t &bar_kv = rest.kv, &bar_s = rest.s, &bar_p = rest.p, &bar_dp = rest.dp, &bar_ds = rest.ds;
    auto &bar_full = rest.full, &bar_free = rest.free;
    auto &bar_all = rest.all;
    auto &bar_stat = rest.stat, &bar_sfree = rest.sfree, &bar_clean = rest.clean;
    uint32_t &tmem_base = rest.tmem;
    int &abort_flag = rest.abort;
    if (smem_u32(sm) & 1023) {                              // (the swizzle's alignment; shared memory starts on it)
        if (threadIdx.x == 0) atomicExch(&g_win_bwd_timeout, 1u);
        return;
    }

    const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
    const int r = p.H / p.Hkv;
    // the key tile; of a tile of sinks, the queries of its window (slice 0, or a piece of it) or a part of those beyond.  All
    // streams' long ones come first: the last tiles have the fewest queries
    const int streams = p.B * p.Hkv, far = p.sink_tiles * (p.slices - 1);
    const int stream = blockIdx.x % streams, hk = stream % p.Hkv, b = stream / p.Hkv;
    int item = blockIdx.x / streams, tile_j, slice = 0, piece = 0;
    if (item < far) {
        tile_j = item / (p.slices - 1);
        slice = 1 + item % (p.slices - 1);
    } else {
        item -= far;
        tile_j = item / p.near;
        piece = item % p.near;
    }
    const int j0 = tile_j * kRows, Tk = p.past + p.T, n = real_tokens(p.lens, b, p.T), keys = p.past + n;
    const bool cut = tile_j < p.sink_tiles && p.slices > 1; // its rows of sinks are summed from parts
    // tiles of queries, [first, end); iterations [it0, it1) over heads and those
    int first = max(0, j0 - p.past) / kRows, end = (n + kRows - 1) / kRows;
    const long long last = (long long)j0 + kRows - 1 + p.window - 1 - p.past;                // the window's last token
    const int window_end = last < 0 ? 0 : (int)min((long long)end, last / kRows + 1);
    if (j0 >= p.sinks || (cut && slice == 0)) end = window_end;
    if (slice > 0) first = max(first, window_end);
    if (j0 >= keys) end = first;
    const int tiles = max(0, end - first);
    int it0 = 0, it1 = tiles * r;
    if (slice > 0) {
        const int all = it1, each = (all + p.slices - 2) / (p.slices - 1);
        it0 = min(all, (slice - 1) * each);
        it1 = min(all, it0 + each);
    } else {
        it0 = (int)((long long)it1 * piece / p.near);
        it1 = (int)((long long)it1 * (piece + 1) / p.near);
    }
    const int count = it1 - it0;
    auto head_of = [&](int i) { return hk * r + (it0 + i) / tiles; };
    auto token_of = [&](int i) { return (first + (it0 + i) % tiles) * kRows; };

    if (tid == 0) {
        mbar_init(&bar_kv, 1);
        for (int i = 0; i < L::kSlots; ++i) {
            mbar_init(&bar_full[i], 1);
            mbar_init(&bar_free[i], 1);
        }
        mbar_init(&bar_s, 1);
        mbar_init(&bar_p, kWorkers);
        mbar_init(&bar_dp, 1);
        mbar_init(&bar_ds, kWorkers);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar_all[i], 1);
            mbar_init(&bar_stat[i], 1);
            mbar_init(&bar_sfree[i], kWorkers);
            mbar_init(&bar_clean[i], kWorkers);
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
    const uint32_t tm = tmem_base, base = smem_u32(sm);
    auto ring = [](int i) { return (uint32_t)(i / L::kSlots) & 1u; };
    // a tile whose last rows are padding: they are cleared before the products see them (both are summed over)
    auto ragged = [&](int i) { return n < p.T && token_of(i) + kRows > n; };

    int loaded = 0;
    if (tid == kLoader && count > 0) {
        mbar_arrive_expect_tx(&bar_kv, 2 * L::kTile);
        load_tile<DP>(sm, &mk, &bar_kv, hk, j0, b);
        load_tile<DP>(sm + L::kTile, &mv, &bar_kv, hk, j0, b);
        for (int i = 0; i < 2 * count; ++i, ++loaded) {     // Q_0, dO_0, Q_1, ..
            const int slot = i % L::kSlots;
            if (i >= L::kSlots && !one_wait(&bar_free[slot], ring(i - L::kSlots), &abort_flag)) break;
            mbar_arrive_expect_tx(&bar_full[slot], L::kTile);
            load_tile<DP>(sm + L::kRing + slot * L::kTile, i & 1 ? &md : &mq, &bar_full[slot], head_of(i >> 1), token_of(i >> 1), b);
        }
    } else if (warp == kIssueWarp) {
        const bool leader = elect_one();
        auto tile = [&](int i) { return base + L::kRing + (i % L::kSlots) * L::kTile; };
        auto arrived = [&](int i) { return warp_wait(&bar_full[i % L::kSlots], ring(i), &abort_flag); };
        // Step i of a chain: the product with what has been packed of tile i - 1, then the next scores over it.  First chain:
        // dV += P^T dO, S^T = K Q^T; second: dK += dS^T Q, dP^T = V dO^T.  In turn: while one's scores are worked on the tensor
        // core has the other's products.
        int cleaned = 0;                                    // ragged tiles so far
        auto step = [&](int i, bool second) {
            const int with = 2 * i - 1 - second, next = 2 * i + second;          // dO or Q of the last tile; Q or dO of the next
            const uint32_t scores = tm + (second ? TM_DP : TM_S), sum = tm + (second ? TM_DK : TM_DV), keys_tile = base + (second ? L::kTile : 0);
            if (i < count) {
                if (!arrived(next)) return false;
                if (!second && ragged(i)) {
                    if (!warp_wait(&bar_clean[cleaned & 1], (cleaned >> 1) & 1, &abort_flag)) return false;
                    ++cleaned;
                }
            }
            if (i > 0) {
                if (!warp_wait(second ? &bar_ds : &bar_p, (i - 1) & 1, &abort_flag)) return false;
                tc_fence_after();
                mma_tmem_cols<DP, 4>(leader, sum, scores, tile(with), i > 1);
                commit(leader, &bar_free[with % L::kSlots]);
            }
            tc_fence_after();
            if (i < count) {
                mma_rows_rows<DP, 128>(leader, scores, keys_tile, tile(next), false);
                commit(leader, second ? &bar_dp : &bar_s);
            }
            return true;
        };
        bool ok = count > 0 && warp_wait(&bar_kv, 0, &abort_flag);
        for (int i = 0; ok && i <= count; ++i) ok = step(i, false) && step(i, true);
        commit(leader, &bar_all[0]);
        commit(leader, &bar_all[1]);
    } else if (warp == kStatWarp) {
        for (int i = 0; i < count; ++i) {
            const int t0 = token_of(i);
            const size_t tok = ((size_t)b * p.T + t0) * p.H + head_of(i);
            float4 l, d;
            float *lv = reinterpret_cast<float *>(&l), *dv = reinterpret_cast<float *>(&d);
#pragma unroll
            for (int e = 0; e < 4; ++e) {                   // padding: P = exp2(0 - inf)
                const int t = 4 * lane + e;
                const bool real = t0 + t < n;
                lv[e] = real ? kLog2e * p.lse[tok + (size_t)t * p.H] : INFINITY;
                dv[e] = real ? p.delta[tok + (size_t)t * p.H] : 0.f;
            }
            if (i >= 2 && !warp_wait(&bar_sfree[i & 1], ((i >> 1) - 1) & 1, &abort_flag)) break;
            *reinterpret_cast<float4 *>(lse_of[i & 1] + 4 * lane) = l;
            *reinterpret_cast<float4 *>(delta_of[i & 1] + 4 * lane) = d;
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar_stat[i & 1]);
        }
    } else if (tid < kWorkers) {
        const int quarter = warp >> 2, row = tid & 127, j = j0 + row;
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t sS = tm + TM_S + 32 * quarter + lanes, sD = tm + TM_DP + 32 * quarter + lanes;
        const float c = p.scale * kLog2e;
        bool ok = true;
        int cleaned = 0;
        auto clear = [&](int i) {                           // of a ragged tile: Q's rows by two quarters, dO's by the others
            const int k0 = 2 * i + (quarter >> 1), slot = k0 % L::kSlots;
            if (!warp_wait(&bar_full[slot], ring(k0), &abort_flag)) return false;
            if (token_of(i) + row >= n)
#pragma unroll
                for (int k = 0; k < DP / 16; ++k) {
                    const int chunk = DP / 16 * (quarter & 1) + k;
                    *reinterpret_cast<uint4 *>(sm + L::kRing + slot * L::kTile + (chunk >> 3) * kPanel + row * 128 + (chunk & 7) * 16) =
                        make_uint4(0u, 0u, 0u, 0u);
                }
            fence_proxy_async();
            mbar_arrive(&bar_clean[cleaned & 1]);
            ++cleaned;
            return true;
        };
        if (count > 0 && ragged(0)) ok = clear(0);
        for (int i = 0; ok && i < count; ++i) {
            const int q0 = p.past + token_of(i);            // position of column 0
            ok = warp_wait(&bar_stat[i & 1], (i >> 1) & 1, &abort_flag) && warp_wait(&bar_s, i & 1, &abort_flag);
            if (!ok) break;
            tc_fence_after();
            float s[32];
            tmem_ld32(sS, s);
            tmem_ld_wait();
            const f32x2 c2 = pk(c, c);
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
                const float4 l = *reinterpret_cast<const float4 *>(lse_of[i & 1] + 32 * quarter + e);
                unpk(exp2_2(fma2(pk(s[e], s[e + 1]), c2, pk(-l.x, -l.y))), s[e], s[e + 1]);
                unpk(exp2_2(fma2(pk(s[e + 2], s[e + 3]), c2, pk(-l.z, -l.w))), s[e + 2], s[e + 3]);
            }
            const bool inner = j0 + kRows - 1 <= q0 && (q0 + kRows - 1 - j0 < p.window || j0 + kRows - 1 < p.sinks);
            if (!inner) {
                const int lo = j - q0;
                const long long see = (long long)j + p.window - 1 - q0;
                const int hi = j < p.sinks || see > kRows ? kRows : see < -1 ? -1 : (int)see;
                const uint32_t bits = bits_between(lo, hi, quarter);
#pragma unroll
                for (int e = 0; e < 32; ++e) s[e] = (bits >> e) & 1u ? s[e] : 0.f;
            }
            uint32_t packed[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) packed[e] = pack_bf16x2(s[2 * e], s[2 * e + 1]);
            tmem_st16(sS, packed);
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive(&bar_p);
            if (i + 1 < count && ragged(i + 1)) {
                ok = clear(i + 1);
                if (!ok) break;
            }
            ok = warp_wait(&bar_dp, i & 1, &abort_flag);
            if (!ok) break;
            tc_fence_after();
            float dp[32];
            tmem_ld32(sD, dp);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
                const float4 d = *reinterpret_cast<const float4 *>(delta_of[i & 1] + 32 * quarter + e);
                packed[e / 2] = pack_ds(s[e], s[e + 1], dp[e] - d.x, dp[e + 1] - d.y);
                packed[e / 2 + 1] = pack_ds(s[e + 2], s[e + 3], dp[e + 2] - d.z, dp[e + 3] - d.w);
            }
            tmem_st16(sD, packed);
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive(&bar_sfree[i & 1]);
            mbar_arrive(&bar_ds);
        }
        const int of = quarter >> 1;                        // dV by two quarters, dK by the others, over V and K
        if (ok && count > 0) ok = warp_wait(&bar_all[0], 0, &abort_flag) && warp_wait(&bar_all[1], 0, &abort_flag);
        if (ok) {
            tc_fence_after();
            const bool real = j < keys;
            const float f = !of ? 1.f : sees_itself_alone(Tk - 1, p.window, p.sinks) ? 0.f : p.scale;
            float *part = nullptr;
            if (slice == 0 && p.near > 1) {
                if (j < Tk) part = p.pieces + ((((size_t)piece * p.B + b) * Tk + j) * p.Hkv + hk) * 2 * p.d + (of ? 0 : p.d);
            } else if (cut && j < p.sinks && j < Tk) {
                part = p.parts + (((((size_t)b * p.Hkv + hk) * p.sink_tiles + tile_j) * p.slices + slice) * kRows + row) * 2 * p.d + (of ? 0 : p.d);
            }
            uint8_t *to = sm + (of ? 0 : L::kTile);
#pragma unroll 1
            for (int k = 0; k < DP / 64; ++k) {
                float x[32];
                const int c0 = DP / 2 * (quarter & 1) + 32 * k;
                tmem_ld32(tm + (of ? TM_DK : TM_DV) + c0 + lanes, x);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 32; ++e) x[e] = real && count > 0 ? f * x[e] : 0.f;
                if (part)
#pragma unroll
                    for (int e = 0; e < 32; e += 4)
                        if (c0 + e < p.d) *reinterpret_cast<float4 *>(part + c0 + e) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
#pragma unroll
                for (int e = 0; e < 32; e += 8)
                    *reinterpret_cast<uint4 *>(to + (c0 >> 6) * kPanel + sw128_off(row, (c0 & 63) + e)) = tc::pack8p(x + e);
            }
        }
        fence_proxy_async();
        named_sync(1, kWorkers);
        if (tid == 0 && slice == 0 && p.near == 1 && !*reinterpret_cast<volatile int *>(&abort_flag)) {
            store_tile<DP>(&mdk, sm, hk, j0, b);
            store_tile<DP>(&mdv, sm + L::kTile, hk, j0, b);
            tma_store_commit();
            tma_store_wait_read0();
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (abort_flag) {
        if (tid == kLoader && count > 0) {
            mbar_wait(&bar_kv, 0, kWaitNs);
            for (int i = max(0, loaded - L::kSlots); i < loaded; ++i) mbar_wait(&bar_full[i % L::kSlots], ring(i), kWaitNs);
        }
        if (warp == kIssueWarp && elect_one()) {
            mbar_wait(&bar_all[0], 0, kWaitNs);             // (committed behind all the products)
            mbar_wait(&bar_all[1], 0, kWaitNs);
            atomicExch(&g_win_bwd_timeout, 1u);
        }
        __syncwarp();
        __syncthreads();
    }
    if (warp == 0) tmem_dealloc(tm, 512);
}

// The rows of the sinks: their parts summed in order.  One CTA a (row, key head, sequence).
__global__ void win_sinks_kernel(Params p, __nv_bfloat16 *dk, __nv_bfloat16 *dv) {
    const int rows = min(p.sinks, p.past + p.T), j = blockIdx.x % rows, u = blockIdx.x / rows, hk = u % p.Hkv, b = u / p.Hkv;
    const int c = threadIdx.x;
    if (c >= 2 * p.d) return;
    const float *part = p.parts + ((((size_t)b * p.Hkv + hk) * p.sink_tiles + j / kRows) * p.slices * kRows + j % kRows) * 2 * p.d + c;
    float t = 0.f;
#pragma unroll 8
    for (int s = 0; s < p.slices; ++s) t += part[(size_t)s * kRows * 2 * p.d];
    const size_t at = (((size_t)b * (p.past + p.T) + j) * p.Hkv + hk) * p.d;
    if (c < p.d) dk[at + c] = __float2bfloat16_rn(t);
    else dv[at + c - p.d] = __float2bfloat16_rn(t);
}

// The same for keys whose tiles are cut: a CTA a row of dk and dv, its pieces in order, then a sink's slices.
__global__ void win_pieces_kernel(Params p, __nv_bfloat16 *dk, __nv_bfloat16 *dv) {
    const int Tk = p.past + p.T, hk = blockIdx.x % p.Hkv, u = blockIdx.x / p.Hkv, j = u % Tk, b = u / Tk, c = threadIdx.x;
    if (c >= 2 * p.d) return;
    const size_t row = blockIdx.x, rows = (size_t)p.B * Tk * p.Hkv;
    float t = 0.f;
#pragma unroll 4
    for (int s = 0; s < p.near; ++s) t += p.pieces[(s * rows + row) * 2 * p.d + c];
    if (j < p.sinks && p.slices > 1) {
        const float *part = p.parts + ((((size_t)b * p.Hkv + hk) * p.sink_tiles + j / kRows) * p.slices * kRows + j % kRows) * 2 * p.d + c;
#pragma unroll 4
        for (int s = 1; s < p.slices; ++s) t += part[(size_t)s * kRows * 2 * p.d];
    }
    if (c < p.d) dk[row * p.d + c] = __float2bfloat16_rn(t);
    else dv[row * p.d + c - p.d] = __float2bfloat16_rn(t);
}

// How the second kernel is cut.  Tiles of sinks: where the queries beyond the window outnumber the window's, as many slices
// as leave each about a window's work (1: nothing is cut).  More than two such tiles are left whole, CTAs that walk every later
// query, which is slow where the window is short: 1 x 32768 tokens, 16 heads on 4, window 512: 4 sinks 691 us, 256 795, 257
// 2192.  All tiles: where the longest walk, of the queries of a window and the
// heads that share the keys, is more than one and a half times an SM's share of all, into `near` pieces of about half a share, of
// at least eight pairs of tiles; a kernel of its own adds the pieces up.  Both directions, us, without and with pieces:
// 1 x 4096 tokens, 16 heads on 1, all keys: 867, 219; 2 x 4096, 16 on 2: 579, 423; 1 x 300, 16 on 1: 96, 41; a window of 2048 of
// 16384 tokens, 4 heads on 1 (128 walks of one length), in two pieces 186, as the rule has it 172.
struct Cut {
    int tiles, slices, near;
};
Cut cut_of(int B, int T, int past, int H, int Hkv, int window, int sinks) {
    const long long keys = (long long)past + T, blocks = (T + kRows - 1) / kRows, key_tiles = (keys + kRows - 1) / kRows;
    const long long tiles = (sinks < keys ? sinks + kRows - 1 : keys + kRows - 1) / kRows, seen = (window < keys ? window : keys) / kRows + 2;
    const long long r = H / Hkv, streams = (long long)B * Hkv, ctas = std::max(1LL, streams * key_tiles);
    // query blocks see `most` tiles each, but for the first `fewer`, which see 1 + past / 128, one more, ..
    const long long most = std::min(seen, key_tiles), lack = std::max(0LL, most - 1 - past / kRows), fewer = std::min(lack, blocks);
    const long long pairs = streams * r * (blocks * most - fewer * lack + fewer * (fewer - 1) / 2), longest = r * std::min(blocks, most);
    const long long share = std::max(1LL, pairs / kSMs);
    Cut c{0, 1, 1};
    if (2 * longest > 3 * share)
        c.near = (int)std::max(1LL, std::min({longest / 8, 2LL * kSMs / ctas, (2 * longest + share - 1) / share}));
    if (sinks == 0 || tiles > 2 || blocks - seen <= seen) return c;
    const long long slices = 1 + c.near * ((blocks - seen + seen - 1) / seen);
    c.tiles = (int)tiles;
    c.slices = (int)(slices < kMostSlices ? slices : kMostSlices);
    return c;
}

size_t parts_bytes(const Cut &c, int B, int Hkv, int d) {
    return c.slices > 1 ? sizeof(float) * (size_t)B * Hkv * c.tiles * c.slices * kRows * 2 * d : 0;
}
size_t delta_bytes(int B, int T, int H) { return (sizeof(float) * (size_t)B * T * H + 255) / 256 * 256; }

template <int DP> cudaError_t run(const WinArgs &a, cudaStream_t s, int *n) {
    CUtensorMap mq, mk, mv, md, mo, mdq, mdk, mdv;
    const int keys = a.past + a.T;
    if (!token_map(&mq, a.q, a.B, a.T, a.H, a.d) || !token_map(&mk, a.k, a.B, keys, a.Hkv, a.d) ||
        !token_map(&mv, a.v, a.B, keys, a.Hkv, a.d) || !token_map(&md, a.dO, a.B, a.T, a.H, a.d) || !token_map(&mo, a.o, a.B, a.T, a.H, a.d) ||
        !token_map(&mdq, a.dq, a.B, a.T, a.H, a.d) || !token_map(&mdk, a.dk, a.B, keys, a.Hkv, a.d) ||
        !token_map(&mdv, a.dv, a.B, keys, a.Hkv, a.d))
        return cudaErrorInvalidValue;
    constexpr int bytes = Layout<DP>::kBytes;
    cudaError_t e = cudaFuncSetAttribute(win_dq_tc_kernel<DP>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(win_dkdv_tc_kernel<DP>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    const Cut cut = cut_of(a.B, a.T, a.past, a.H, a.Hkv, a.window, a.sinks);
    // (dq's blocks together where the window does not make them alike: 1 x 8192 tokens, 8 heads on 8, all keys 418 us, 370 so; a window
    // of 1024 of 4 x 4096 tokens the same either way)
    Params p{a.lse, a.lens, static_cast<float *>(a.ws), nullptr, nullptr, a.B, a.T, a.past, a.H, a.Hkv, a.d, a.window, a.sinks,
             (a.T + kRows - 1) / kRows, (keys + kRows - 1) / kRows, cut.tiles, cut.slices, cut.near,
             2.0 * a.window > keys && blocks_together(a), a.scale};
    p.parts = reinterpret_cast<float *>(static_cast<uint8_t *>(a.ws) + delta_bytes(a.B, a.T, a.H));
    p.pieces = p.parts + parts_bytes(cut, a.B, a.Hkv, a.d) / sizeof(float);
    win_dq_tc_kernel<DP><<<(unsigned)((size_t)a.B * a.H * p.blocks), kThreadsQ, bytes, s>>>(p, mq, mk, mv, md, mo, mdq);
    *n += 1;
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const size_t items = (size_t)p.key_tiles * cut.near + (size_t)cut.tiles * (cut.slices - 1);
    win_dkdv_tc_kernel<DP><<<(unsigned)((size_t)a.B * a.Hkv * items), kThreadsK, bytes, s>>>(p, mq, mk, mv, md, mdk, mdv);
    *n += 1;
    e = cudaGetLastError();
    if (e == cudaSuccess && cut.near > 1) {
        win_pieces_kernel<<<(unsigned)((size_t)a.B * keys * a.Hkv), 256, 0, s>>>(p, static_cast<__nv_bfloat16 *>(a.dk),
                                                                                 static_cast<__nv_bfloat16 *>(a.dv));
        *n += 1;
        return cudaGetLastError();
    }
    if (e != cudaSuccess || cut.slices == 1) return e;
    const size_t rows = a.sinks < keys ? a.sinks : keys;
    win_sinks_kernel<<<(unsigned)(rows * a.Hkv * a.B), 256, 0, s>>>(p, static_cast<__nv_bfloat16 *>(a.dk), static_cast<__nv_bfloat16 *>(a.dv));
    *n += 1;
    return cudaGetLastError();
}

}  // namespace

// The rows' D, the parts of the sinks' rows, the pieces.
size_t win_bwd_tc_workspace(int B, int T, int past, int H, int Hkv, int d, int window, int sinks) {
    const Cut cut = cut_of(B, T, past, H, Hkv, window, sinks);
    return delta_bytes(B, T, H) + parts_bytes(cut, B, Hkv, d) +
           (cut.near > 1 ? sizeof(float) * cut.near * (size_t)B * (past + T) * Hkv * 2 * d : 0);
}

cudaError_t launch_win_bwd_tc(const WinArgs &a, cudaStream_t s, int *n) { return a.d > 64 ? run<128>(a, s, n) : run<64>(a, s, n); }

bool win_bwd_read_and_clear_timeout() {
    unsigned int v = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&v, g_win_bwd_timeout, sizeof v) != cudaSuccess) return false;
    if (v) cudaMemcpyToSymbol(g_win_bwd_timeout, &zero, sizeof zero);
    return v != 0;
}

}  // namespace qd
