// Linear attention on the sm_103a tensor cores (bf16; tcgen05, TMEM, TMA): the forward, and the pass that leaves
// the states between chunks for the backward.  The mathematics is lin_attn_simt.cu's, in chunks of 128 tokens:
//     A = Q K^T,  P = A . M,  O = P V + (gamma Q) S^T,  S <- a S + (kappa V)^T K
// One CTA of 20 warps walks a stream's chunks:
//   warps 0-3, 12-15   halves of the columns of P (in bf16 over A in TMEM; a thread: a row, a token), then of the tokens of the next
//                chunk's (kappa V)^T, through transposing loads and stores of 8x8 fragments
//   warps 4-11   the state: a thread has a row of S (of d_v) and half its columns in registers, in fp32; the bf16 copy
//                of S that the outputs read; the outputs' way out
//   warp 16      TMA loads, two chunks ahead;  warp 17  the products;  warp 18  the decays;  warp 19  the outputs' copies
// TMEM: A 0-127 (P over 0-31 and 64-95), O 128-255, the chunk's (kappa V)^T K 256-383, (kappa V)^T 384-511 (64 columns of high
// parts, 64 of low parts).
//
// In a light chunk (lin_tc.cuh) P is A kappa_j below the diagonal, S is copied times a, Q enters as it is, and the
// rows of O are multiplied by exp(P_i - P_end) on their way out.  Otherwise P takes an exponential a pair, gamma Q is
// formed in bf16 over the rest of A, and O is done.
//
// The state leaves in fp32 and has to be fp32: kappa V is split into two bf16 numbers (16 bits and more of it; K
// is exact), at the cost of a fifth product of 128^3, and added to S in registers, rounded to nearest.  The other
// factors are rounded to bf16 once (P and S; gamma Q), their products' other factors being bf16 themselves.
//
// By its bytes memory bound (1 KB a token and head at d = 128: 41 us at the measured copy rate for 8 x 2048 tokens of 16 heads);
// a chunk's products take 2560 cycles of the tensor core.  Measured there: 56 us, 73 % of that rate, on 128 of the 152 SMs:
// 4600 cycles a chunk, of which the chain turned tile, state's product, state, its copy, outputs is the longest part.
//
// Few streams are cut into segments: each segment's own state from zero (this kernel without outputs), the states
// that enter the segments (lin_join_kernel), then the outputs of all of them.  1 x 32768 tokens, 16 heads: 153 us, 53 the first
// pass, 5 the join, 92 the outputs (16 streams in one pass would keep 16 SMs busy).
//
// Backwards (for the gradient of the state): X = dO in v's place, Y = q in k's, gamma in kappa's, chunks from the last.  The
// backward's walks, without outputs, run both ways in one launch, with two places in TMEM for X^T and for the product and three
// in shared memory for tiles.  4 x 4096 tokens, 8 heads: 33 us for each of the two passes.
//
// Every wait is bounded; on a timeout the kernel sets its error word, waits (bounded) for its own copies and products,
// frees TMEM and returns.
#include "lin_tc.cuh"

namespace qd {

__device__ unsigned int g_lin_tc_timeout = 0;

namespace {

using namespace mix;

constexpr int kStateFirst = 128, kStateThreads = 256, kTurnWarp = 12, kLoader = 512, kIssuer = 544, kGateWarp = 18;
constexpr int kStoreWarp = 19, kTurnThreads = 256, kThreads = 640;
constexpr uint32_t TM_A = 0, TM_O = 128, TM_DS = 256, TM_X = 384;

struct Params {
    const void *g;
    const int *lens;
    const float *first_state, *entering;      // of a stream in one piece (null: zero); of the segments of the others
    float *last_state, *leaving, *decay;      // of the last one; of the others, with their decays (null: not written)
    uint8_t *chk;                             // states entering the chunks (leaving ones' gradients), as operand tiles
    void *o;
    // segments: walked by a stream's CTAs here, in all, their chunks; states that end one of the first pass (`joints` a stream: with
    // the first, joints + 1 entering ones), `pieces` to a segment
    int g_token, T, H, nk, nv, walked, segs, seg_chunks, joints, pieces, back;
};

// Stages of {Y, X, Q}: two; without outputs three of {Y, X}.
template <int DK, int DV, bool OUT> struct Layout {
    static constexpr int kStages = OUT ? 2 : 3;
    static constexpr uint32_t kY = DK / 64 * kPanel, kX = DV / 64 * kPanel;      // a tile of k or q, of v or dO
    static constexpr uint32_t kStage = (OUT ? 2 : 1) * kY + kX, kBytes = kY + kStages * kStage + 2 * sizeof(Gates) + 288;
    static constexpr uint32_t kChk = DV * DK * 2;
};

struct Bars {
    uint64_t fy[3], fx[3], fq[2], ey[3], ex[3], eq[2];      // tiles of K (Q), V (dO), Q: there; free again
    uint64_t gates[2], gfree[2], x[2], ds[2], dsread[2], a, p, s, o, oread, staged, drain;
    uint32_t tmem;
    int abort;
};

template <int DK, int DV, bool OUT>
__global__ void __launch_bounds__(kThreads, 1)
lin_tc_kernel(const __grid_constant__ Params there, const __grid_constant__ Params back, const __grid_constant__ CUtensorMap mq,
              const __grid_constant__ CUtensorMap my_there, const __grid_constant__ CUtensorMap mx_there,
              const __grid_constant__ CUtensorMap mo, const __grid_constant__ CUtensorMap my_back,
              const __grid_constant__ CUtensorMap mx_back, int forward) {
    typedef Layout<DK, DV, OUT> L;
    // the first `forward` CTAs walk forward
    const bool backwards = !OUT && blockIdx.x >= forward;
    const Params &p = backwards ? back : there;
    const CUtensorMap &my = backwards ? my_back : my_there, &mx = backwards ? mx_back : mx_there;
    const int cta = backwards ? blockIdx.x - forward : blockIdx.x;
    extern __shared__ __align__(1024) uint8_t sm[];         // S (its copy on the way out) | stages | decays | barriers
    uint8_t *stages = sm + L::kY;
    Gates *gates = reinterpret_cast<Gates *>(stages + L::kStages * L::kStage);
    Bars &bar = *reinterpret_cast<Bars *>(gates + 2);
    constexpr uint32_t OY = 0, OX = L::kY, OQ = L::kY + L::kX;
    // where outputs are staged: in q's place if they fit (V is then free earlier: its way is the longer one), else v's
    constexpr bool kInQ = DK >= DV;
    static_assert(L::kChk <= L::kY, "the state's copy");
    static_assert(sizeof(Bars) <= 288 && L::kBytes <= 232448, "shared memory");

    const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
    if (smem_u32(sm) & 1023) {                              // (the swizzle's alignment; shared memory starts on it)
        if (tid == 0) atomicExch(&g_lin_tc_timeout, 1u);
        return;
    }
    const int w = cta % p.walked, bh = cta / p.walked, b = bh / p.H, h = bh % p.H;
    const int seg = p.back ? p.segs - 1 - w : w, n = real_tokens(p.lens, b, p.T);
    const int chunks = (p.T + kRows - 1) / kRows, c_first = seg * p.seg_chunks, c_end = min(chunks, c_first + p.seg_chunks);
    const int live = max(0, min(c_end, (n + kRows - 1) / kRows) - c_first);      // chunks with real tokens
    auto chunk = [&](int i) { return p.back ? c_first + live - 1 - i : c_first + i; };

    if (tid == 0) {
        for (int i = 0; i < 3; ++i) {
            mbar_init(&bar.fy[i], 1);
            mbar_init(&bar.fx[i], 1);
            mbar_init(&bar.ey[i], 1);
            mbar_init(&bar.ex[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar.fq[i], 1);
            mbar_init(&bar.eq[i], 1);
            mbar_init(&bar.gates[i], 1);
            mbar_init(&bar.gfree[i], kStateThreads);
            mbar_init(&bar.x[i], kTurnThreads);
            mbar_init(&bar.ds[i], 1);
            mbar_init(&bar.dsread[i], kStateThreads);
        }
        mbar_init(&bar.a, 1);
        mbar_init(&bar.p, kTurnThreads);
        mbar_init(&bar.s, kStateThreads);
        mbar_init(&bar.o, 1);
        mbar_init(&bar.oread, kStateThreads);
        mbar_init(&bar.staged, kStateThreads);
        mbar_init(&bar.drain, 1);
        bar.abort = 0;
        fence_mbar_init();
    }
    if (warp == 0) {
        tmem_alloc(&bar.tmem, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = bar.tmem, base = smem_u32(sm);
    constexpr int kN = L::kStages;
    auto stage = [&](int i) { return stages + (i % kN) * L::kStage; };
    auto stage_addr = [&](int i) { return base + L::kY + (i % kN) * L::kStage; };
    auto use = [](int i) { return (uint32_t)(i / kN) & 1u; };                     // parity of index i's use of its stage
    auto ring = [](int i) { return (uint32_t)(i >> 1) & 1u; };                   // parity of index i's use of one of two places
    // the places in TMEM of X^T and of the product, and the last chunk that had index i's
    auto x_place = [&](int i) { return tm + (!OUT && (i & 1) ? TM_A : TM_X); };
    auto ds_place = [&](int i) { return tm + (!OUT && (i & 1) ? TM_O : TM_DS); };
    constexpr int kBefore = OUT ? 1 : 2;

    int loaded = 0;
    if (tid == kLoader) {
        for (int i = 0; i < live; ++i) {
            const int s = i % kN, t0 = chunk(i) * kRows;
            if (i >= kN && !one_wait(&bar.ey[s], use(i - kN), &bar.abort)) break;
            mbar_arrive_expect_tx(&bar.fy[s], L::kY);
            load_tile<DK>(stage(i) + OY, &my, &bar.fy[s], h, t0, b);
            loaded = 3 * i + 1;
            if (i >= kN && !one_wait(&bar.ex[s], use(i - kN), &bar.abort)) break;
            mbar_arrive_expect_tx(&bar.fx[s], L::kX);
            load_tile<DV>(stage(i) + OX, &mx, &bar.fx[s], h, t0, b);
            loaded = 3 * i + 2;
            if (OUT) {                                      // (last: its place is the last to be free, when the outputs are out of it)
                if (i >= kN && !one_wait(&bar.eq[s], use(i - kN), &bar.abort)) break;
                mbar_arrive_expect_tx(&bar.fq[s], L::kY);
                load_tile<DK>(stage(i) + OQ, &mq, &bar.fq[s], h, t0, b);
            }
            loaded = 3 * i + 3;
        }
    } else if (warp == kIssuer / 32) {
        const bool leader = elect_one();
        auto issue_a = [&](int i) {
            if (!warp_wait(&bar.fy[i % kN], use(i), &bar.abort) || !warp_wait(&bar.fq[i % kN], use(i), &bar.abort)) return false;
            mma_rows_rows<DK, 128>(leader, tm + TM_A, stage_addr(i) + OQ, stage_addr(i) + OY, false);
            commit(leader, &bar.a);
            return true;
        };
        bool ok = live > 0;
        if (OUT && ok) ok = issue_a(0);
        for (int i = 0; ok && i < live; ++i) {
            ok = warp_wait(&bar.x[i & 1], ring(i), &bar.abort) && warp_wait(&bar.fy[i % kN], use(i), &bar.abort) &&
                 (i < kBefore || warp_wait(&bar.dsread[(i - kBefore) & 1], ring(i - kBefore), &bar.abort));
            if (!ok) break;
            tc_fence_after();
            mma_tmem_cols<DK>(leader, ds_place(i), x_place(i), stage_addr(i) + OY, false);
            mma_tmem_cols<DK>(leader, ds_place(i), x_place(i) + 64, stage_addr(i) + OY, true);
            commit(leader, &bar.ds[i & 1]);
            commit(leader, &bar.ey[i % kN]);
            if (!OUT) {
                commit(leader, &bar.ex[i % kN]);
                continue;
            }
            ok = warp_wait(&bar.p, i & 1, &bar.abort) && warp_wait(&bar.s, i & 1, &bar.abort) &&
                 (i == 0 || warp_wait(&bar.oread, (i - 1) & 1, &bar.abort));
            if (!ok) break;
            tc_fence_after();
            mma_tmem_cols<DV, 2>(leader, tm + TM_O, tm + TM_A, stage_addr(i) + OX, false);
            if (gates[i & 1].light) {
                mma_rows_rows<DK, DV>(leader, tm + TM_O, stage_addr(i) + OQ, base, true);
            } else {
                const uint64_t ds = desc_rows(base);
                if (leader) {
#pragma unroll
                    for (int k = 0; k < DK / 16; ++k)
                        umma_bf16_ta(tm + TM_O, tm + TM_A + 32 + step_halves(k), ds + step_rows(k), idesc_bf16(128, DV, false, false), 1);
                }
            }
            commit(leader, &bar.o);
            commit(leader, kInQ ? &bar.ex[i & 1] : &bar.eq[i & 1]);
            if (i + 1 < live) ok = issue_a(i + 1);
        }
        commit(leader, &bar.drain);
    } else if ((OUT || p.chk) && tid == 32 * kStoreWarp) {  // (whose waits for the copies out are nobody else's)
        for (int i = 0; i < live; ++i) {
            if (!one_wait(&bar.staged, i & 1, &bar.abort)) break;
            if (OUT) store_tile<DV>(&mo, stage(i) + (kInQ ? OQ : OX), h, chunk(i) * kRows, b);
            else bulk_store(p.chk + ((size_t)bh * chunks + chunk(i)) * L::kChk, sm, L::kChk);
            tma_store_commit();
            tma_store_wait_read0();
            mbar_arrive(!OUT ? &bar.eq[0] : kInQ ? &bar.eq[i & 1] : &bar.ex[i & 1]);
        }
    } else if (warp == kGateWarp) {
        LaneGates g;
        if (live) g.load(p.g, p.g_token, (size_t)b * p.T, chunk(0) * kRows, n, p.H, h);
        for (int i = 0; i < live; ++i) {
            g.compute(p.back);
            if (i >= 2 && !warp_wait(&bar.gfree[i & 1], ring(i - 2), &bar.abort)) break;
            g.store(gates[i & 1]);
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.gates[i & 1]);
            if (i + 1 < live) g.load(p.g, p.g_token, (size_t)b * p.T, chunk(i + 1) * kRows, n, p.H, h);
        }
    } else if (warp < 4 || (warp >= kTurnWarp && warp < kTurnWarp + 4)) {
        const int half = warp >= 4, row = tid & 127, own = (warp & 3) - 2 * half;    // (own: the row's block, of the half's two)
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        // (f X)^T of chunk i in two bf16 parts, tokens 64 half .. 64 half + 63
        auto turn = [&](int i) {
            const Gates &g = gates[i & 1];
            if (!warp_wait(&bar.gates[i & 1], ring(i), &bar.abort) || !warp_wait(&bar.fx[i % kN], use(i), &bar.abort)) return false;
            const int rows = n - chunk(i) * kRows;          // real tokens, if fewer than the chunk's
            const bool cut = rows < kRows && n < p.T;
            if (cut) {                                      // padding, whatever it holds, is 0: K's rows by one half, V's by the other
                if (!warp_wait(&bar.fy[i % kN], use(i), &bar.abort)) return false;
                if (row >= rows)
                    for (int k = 0; k < (half ? DV : DK) / 8; ++k)
                        *reinterpret_cast<uint4 *>(stage(i) + (half ? OX : OY) + (k >> 3) * kPanel + row * 128 + (k & 7) * 16) =
                            make_uint4(0u, 0u, 0u, 0u);
                fence_proxy_async();
            }
            if (i >= kBefore && !warp_wait(&bar.ds[(i - kBefore) & 1], ring(i - kBefore), &bar.abort)) return false;     // its place in TMEM
            tc_fence_after();
            if (32 * (warp & 3) < DV) {
                // a load gives 8 tokens of this warp's 32 columns; four of them make a store's columns
                const int c0 = 32 * (warp & 3) + (lane & 24);
                const uint32_t from = smem_u32(stage(i) + OX + (c0 >> 6) * kPanel) + (lane & 7) * 128 + ((((c0 >> 3) & 7) ^ (lane & 7)) << 4);
#pragma unroll 1
                for (int t8 = 8 * half; t8 < 8 * half + 8; t8 += 4) {
                    uint32_t v[4][4], hi[2][8], lo[2][8];
#pragma unroll
                    for (int u = 0; u < 4; ++u) ldmatrix_x4_trans(from + (t8 + u) * 1024, v[u]);
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const int t = 8 * (t8 + u) + 2 * (lane & 3);
                        const float2 f = *reinterpret_cast<const float2 *>(g.write + t);
                        const uint32_t keep = !cut ? ~0u : (t < rows ? 0xffffu : 0u) | (t + 1 < rows ? 0xffff0000u : 0u);
#pragma unroll
                        for (int m = 0; m < 4; ++m) {
                            const uint32_t x2 = v[u][m] & keep;
                            const f32x2 x = mul2(pk(__uint_as_float(x2 << 16), __uint_as_float(x2 & 0xffff0000u)), pk(f.x, f.y));
                            float x0, x1, r0, r1;
                            unpk(x, x0, x1);
                            const uint32_t top = pack_bf16x2(x0, x1);
                            unpk(fma2(pk(__uint_as_float(top << 16), __uint_as_float(top & 0xffff0000u)), pk(-1.f, -1.f), x), r0, r1);
                            hi[m >> 1][2 * u + (m & 1)] = top;
                            lo[m >> 1][2 * u + (m & 1)] = pack_bf16x2(r0, r1);
                        }
                    }
#pragma unroll
                    for (int hl = 0; hl < 2; ++hl) {
                        const uint32_t to = x_place(i) + lanes + ((uint32_t)(16 * hl) << 16) + 4 * t8;
                        tmem_st16x128_x4(to, hi[hl]);
                        tmem_st16x128_x4(to + 64, lo[hl]);
                    }
                }
                tmem_st_wait();
            }
            tc_fence_before();
            mbar_arrive(&bar.x[i & 1]);
            return true;
        };
        // P of chunk i, columns 64 half .. 64 half + 63, packed over the first half of them
        auto weights = [&](int i) {
            const Gates &g = gates[i & 1];
            const uint32_t sA = tm + TM_A + 64 * half + lanes;
            if (!warp_wait(&bar.gates[i & 1], ring(i), &bar.abort) || !warp_wait(&bar.a, i & 1, &bar.abort)) return false;
            tc_fence_after();
            const bool light = g.light;
            const float Pi = g.P[row];
            const int seen = g.seen[row];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                uint32_t packed[16];
                const int c = 64 * half + 32 * k;
                if (k > own) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) packed[j] = 0u;
                } else {
                    float x[32];
                    tmem_ld32(sA + 32 * k, x);
                    tmem_ld_wait();
                    // columns up to the row's own, and those that it sees (of a light chunk: all)
                    uint32_t bits = k < own ? ~0u : (2u << lane) - 1u;
                    if (light) {
#pragma unroll
                        for (int j = 0; j < 32; j += 4) {
                            const float4 f = *reinterpret_cast<const float4 *>(g.write + c + j);
                            unpk(mul2(pk(x[j], x[j + 1]), pk(f.x, f.y)), x[j], x[j + 1]);
                            unpk(mul2(pk(x[j + 2], x[j + 3]), pk(f.z, f.w)), x[j + 2], x[j + 3]);
                        }
                    } else {
                        const int lo = max(0, seen - 1 - c);
                        bits = lo > 31 ? 0u : bits & ~((1u << lo) - 1u);
#pragma unroll
                        for (int j = 0; j < 32; j += 4) {
                            const float4 f = *reinterpret_cast<const float4 *>(g.P + c + j);
                            const float e[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
                            for (int u = 0; u < 4; ++u) x[j + u] = (bits >> (j + u)) & 1u ? x[j + u] * exp2_fast(Pi - e[u]) : 0.f;
                        }
                    }
                    if (k == own)
#pragma unroll
                        for (int j = 0; j < 32; ++j) x[j] = (bits >> j) & 1u ? x[j] : 0.f;
#pragma unroll
                    for (int j = 0; j < 16; ++j) packed[j] = pack_bf16x2(x[2 * j], x[2 * j + 1]);
                }
                tmem_st16(sA + 16 * k, packed);
            }
            if (!light && 64 * half < DK) {                 // gamma Q, 64 of its columns over the second half of these
                const uint8_t *q = stage(i) + OQ + half * kPanel;
                const float gamma = seen ? 0.f : exp2_fast(Pi);
#pragma unroll 1
                for (int k = 0; k < 2; ++k) {
                    uint32_t gq[16];
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        float f[8];
                        tc::unpack8(*reinterpret_cast<const uint4 *>(q + sw128_off(row, 32 * k + 8 * c)), f);
#pragma unroll
                        for (int e = 0; e < 4; ++e) gq[4 * c + e] = gamma == 0.f ? 0u : pack_bf16x2(gamma * f[2 * e], gamma * f[2 * e + 1]);
                    }
                    tmem_st16(sA + 32 + 16 * k, gq);
                }
            }
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive(&bar.p);
            return true;
        };
        bool ok = live == 0 || turn(0);
        for (int i = 0; ok && i < live; ++i) ok = (!OUT || weights(i)) && (i + 1 == live || turn(i + 1));
    } else if (tid >= kStateFirst && tid < kStateFirst + kStateThreads) {
        constexpr int SC = DK / 2, OC = DV / 2;             // columns of a thread: of S, of O
        const int half = (warp - 4) >> 2, row = 32 * (warp & 3) + lane;
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const bool mine = row < DV, real_row = row < p.nv;
        float S[SC];
        {
            const float *from = p.entering ? p.entering : p.first_state;
            if (from) from += ((p.entering ? (size_t)bh * (p.joints + 1) + w * p.pieces : (size_t)bh) * p.nv + row) * p.nk;
#pragma unroll
            for (int c = 0; c < SC; c += 4) {
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                if (from && real_row && SC * half + c < p.nk) v = *reinterpret_cast<const float4 *>(from + SC * half + c);
                S[c] = v.x, S[c + 1] = v.y, S[c + 2] = v.z, S[c + 3] = v.w;
            }
        }
        // f times the state in bf16: the outputs' operand, or a checkpoint of the same layout (rows of d_v, panels of d_k)
        auto copy_state = [&](uint8_t *to, uint32_t panel, float f) {
            if (!mine) return;
#pragma unroll
            for (int c = 0; c < SC; c += 8) {
                const int col = SC * half + c;
                float x[8];
#pragma unroll
                for (int e = 0; e < 8; e += 2) unpk(mul2(pk(S[c + e], S[c + e + 1]), pk(f, f)), x[e], x[e + 1]);
                const uint4 v = tc::pack8(x);
                *reinterpret_cast<uint4 *>(to + (col >> 6) * panel + sw128_off(row, col & 63)) = v;
            }
        };
        auto scaled_for = [&](int i) { return gates[i & 1].light ? gates[i & 1].total : 1.f; };
        float decay = 1.f;
        bool ok = true;
        if (OUT && live) {
            ok = warp_wait(&bar.gates[0], 0, &bar.abort);
            if (ok) {
                copy_state(sm, kPanel, scaled_for(0));
                fence_proxy_async();
                mbar_arrive(&bar.s);
            }
        }
        for (int i = 0; ok && i < live; ++i) {
            ok = warp_wait(&bar.gates[i & 1], ring(i), &bar.abort);
            if (!ok) break;
            if (!OUT && p.chk) {                            // on the way out; a forward walk's as the outputs' operand: times a
                ok = i == 0 || warp_wait(&bar.eq[0], (i - 1) & 1, &bar.abort);
                if (!ok) break;
                copy_state(sm, DV * 128, p.back ? 1.f : scaled_for(i));
                fence_proxy_async();
                mbar_arrive(&bar.staged);
            }
            // (read before a wait: the decays' place is handed back below without another use of it)
            const volatile Gates &g = gates[i & 1];
            const float total = g.total, out = OUT && g.light ? exp2_fast(g.P[row] - g.P[kRows - 1]) : 1.f;
            ok = warp_wait(&bar.ds[i & 1], ring(i), &bar.abort);
            if (!ok) break;
            tc_fence_after();
            decay *= total;
            if (total == 0.f)                               // (0 also times what is not finite)
#pragma unroll
                for (int c = 0; c < SC; ++c) S[c] = 0.f;
            if (mine) {
                const f32x2 a2 = pk(total, total);
#pragma unroll
                for (int c = 0; c < SC; c += 32) {
                    float d[2][16];
                    tmem_ld16(ds_place(i) + lanes + SC * half + c, d[0]);
                    tmem_ld16(ds_place(i) + lanes + SC * half + c + 16, d[1]);
                    tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 32; e += 2)
                        unpk(fma2(a2, pk(S[c + e], S[c + e + 1]), pk(d[e >> 4][e & 15], d[e >> 4][(e & 15) + 1])), S[c + e], S[c + e + 1]);
                }
            }
            tc_fence_before();
            mbar_arrive(&bar.dsread[i & 1]);
            if (!OUT) {
                mbar_arrive(&bar.gfree[i & 1]);
                continue;
            }
            float f = 1.f;
            if (i + 1 < live) {
                ok = warp_wait(&bar.gates[(i + 1) & 1], ring(i + 1), &bar.abort);
                if (!ok) break;
                f = scaled_for(i + 1);
            }
            ok = warp_wait(&bar.o, i & 1, &bar.abort);      // the outputs of this chunk have read the last copy
            if (!ok) break;
            tc_fence_after();
            mbar_arrive(&bar.gfree[i & 1]);                 // (the outputs' products come after all else that reads the decays)
            const int t0 = chunk(i) * kRows;
            uint8_t *to = stage(i) + (kInQ ? OQ : OX);      // (the products have read it)
            const bool real = t0 + row < n;
#pragma unroll
            for (int c = 0; c < OC; c += 32) {
                float o[2][16];
                tmem_ld16(tm + TM_O + lanes + OC * half + c, o[0]);
                tmem_ld16(tm + TM_O + lanes + OC * half + c + 16, o[1]);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 32; e += 8) {
                    const int col = OC * half + c + e;
                    float x[8];
#pragma unroll
                    for (int u = 0; u < 8; u += 2)
                        unpk(mul2(pk(o[e >> 4][(e & 15) + u], o[e >> 4][(e & 15) + u + 1]), pk(out, out)), x[u], x[u + 1]);
                    uint4 v = tc::pack8(x);
                    if (!real) v = make_uint4(0u, 0u, 0u, 0u);
                    *reinterpret_cast<uint4 *>(to + (col >> 6) * kPanel + sw128_off(row, col & 63)) = v;
                }
            }
            tc_fence_before();
            mbar_arrive(&bar.oread);
            fence_proxy_async();
            mbar_arrive(&bar.staged);
            copy_state(sm, kPanel, f);                      // (the next chunk's outputs are not near yet)
            fence_proxy_async();
            mbar_arrive(&bar.s);
        }
        if (!bar.abort && real_row) {
            float *to = w == p.segs - 1 ? p.last_state : p.leaving;
            if (to) {
                to += ((w == p.segs - 1 ? (size_t)bh : (size_t)bh * (p.joints + 1) + w + 1) * p.nv + row) * p.nk + SC * half;
#pragma unroll
                for (int c = 0; c < SC; c += 4)
                    if (SC * half + c < p.nk) *reinterpret_cast<float4 *>(to + c) = make_float4(S[c], S[c + 1], S[c + 2], S[c + 3]);
            }
            if (tid == kStateFirst && w < p.segs - 1 && p.decay) p.decay[(size_t)bh * p.joints + w] = decay;
        }
    }
    __syncwarp();
    if (OUT) {                                              // the rows of chunks that are all padding
        const int t0 = (c_first + live) * kRows, t1 = min(p.T, c_end * kRows), per = p.nv / 8;
        for (int u = tid; u < (t1 - t0) * per; u += kThreads)
            *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.o) + (((size_t)b * p.T + t0 + u / per) * p.H + h) * p.nv + 8 * (u % per)) =
                make_uint4(0u, 0u, 0u, 0u);
    }
    tc_fence_before();
    __syncthreads();
    if (bar.abort) {
        if (tid == kLoader)                                 // its copies: the last of each place
            for (int i = max(0, loaded - 3 * kN); i < loaded; ++i) {
                const int c = i / 3, kind = i % 3;
                if (kind == 0) mbar_wait(&bar.fy[c % kN], use(c), kWaitNs);
                if (kind == 1) mbar_wait(&bar.fx[c % kN], use(c), kWaitNs);
                if (kind == 2 && OUT) mbar_wait(&bar.fq[c % kN], use(c), kWaitNs);
            }
        if (tid == kIssuer) {
            mbar_wait(&bar.drain, 0, kWaitNs);              // (committed behind all the products)
            atomicExch(&g_lin_tc_timeout, 1u);
        }
        __syncwarp();
        __syncthreads();
    }
    if (warp == 0) tmem_dealloc(tm, 512);
}

// The states that enter the segments: the first one, which the last pass reads here alone (the state that leaves may have its
// place, and nothing orders the CTAs of a stream's first and last segment), then, in the place of the segments' own,
// S <- a_w S + own_w, walked in order.  A row of the grid is a stream of one direction.
__global__ void lin_join_kernel(const float *first_there, const float *first_back, float *states, const float *decay, int joints, int elements,
                                int streams) {
    const size_t row = blockIdx.y, bh = row % streams;
    const float *first = row < streams ? first_there : first_back;
    const int e = 4 * (blockIdx.x * blockDim.x + threadIdx.x);
    if (e >= elements) return;
    float4 S = first ? *reinterpret_cast<const float4 *>(first + bh * elements + e) : make_float4(0.f, 0.f, 0.f, 0.f);
    states += row * (joints + 1) * elements + e;
    *reinterpret_cast<float4 *>(states) = S;
#pragma unroll 4
    for (int w = 0; w < joints; ++w) {
        float4 *at = reinterpret_cast<float4 *>(states + (size_t)(w + 1) * elements);
        const float a = decay[row * joints + w];
        float4 v = *at;
        if (a != 0.f) v = make_float4(fmaf(a, S.x, v.x), fmaf(a, S.y, v.y), fmaf(a, S.z, v.z), fmaf(a, S.w, v.w));
        *at = v;
        S = v;
    }
}

// Segments of a walk: as many as there are SMs for, of at least 4 chunks each; and the pieces of a segment in the pass that finds
// the states between them, which has one segment a walk less to do.
struct Cut {
    int segs, chunks, pieces; // segments, chunks of one, pieces of one
};
Cut cut_of(long long walks, int T) {
    const int chunks = (T + kRows - 1) / kRows;
    long long segs = walks >= kSMs ? 1 : kSMs / walks;
    const int most = chunks / 4 > 1 ? chunks / 4 : 1;
    if (segs > most) segs = most;
    Cut c;
    c.chunks = (int)((chunks + segs - 1) / segs);
    if (c.chunks < 1) c.chunks = 1;
    c.segs = chunks ? (chunks + c.chunks - 1) / c.chunks : 1;
    c.pieces = 1;
    if (c.segs > 1)
        for (int r = (int)(kSMs / (walks * (c.segs - 1))); r > 1 && c.pieces == 1; --r)
            if (c.chunks % r == 0 && c.chunks / r >= 4) c.pieces = r;
    return c;
}

struct Walks {
    Params p[2];              // forward, backward
    CUtensorMap q, y[2], x[2], o;
    int streams;
};

template <int DK, int DV, bool OUT> cudaError_t launch(const Walks &w, cudaStream_t s, int *n, int ctas) {
    constexpr int bytes = Layout<DK, DV, OUT>::kBytes;
    const cudaError_t e = cudaFuncSetAttribute(lin_tc_kernel<DK, DV, OUT>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    lin_tc_kernel<DK, DV, OUT><<<(unsigned)ctas, kThreads, bytes, s>>>(w.p[0], w.p[1], w.q, w.y[0], w.x[0], w.o, w.y[1], w.x[1],
                                                                       w.streams * w.p[0].walked);
    *n += 1;
    return cudaGetLastError();
}
template <bool OUT> cudaError_t launch(const Walks &w, cudaStream_t s, int *n, int ctas) {
    if (w.p[0].nk > 64) return w.p[0].nv > 64 ? launch<128, 128, OUT>(w, s, n, ctas) : launch<128, 64, OUT>(w, s, n, ctas);
    return w.p[0].nv > 64 ? launch<64, 128, OUT>(w, s, n, ctas) : launch<64, 64, OUT>(w, s, n, ctas);
}

// The walks of all streams (without outputs: both ways), cut or not.
cudaError_t walk(Walks &w, bool out, float *ws, cudaStream_t s, int *n) {
    const int ways = out ? 1 : 2;
    const Cut cut = cut_of((long long)ways * w.streams, w.p[0].T);
    const int joints = (cut.segs - 1) * cut.pieces, elements = w.p[0].nk * w.p[0].nv;
    const size_t each = (size_t)w.streams * (joints + 1) * elements;     // of one direction
    float *states = ws, *decay = ws + ways * each;
    if (joints) {
        Walks local = w;
        for (int d = 0; d < 2; ++d) {
            Params &p = local.p[d];
            p.segs = cut.segs * cut.pieces;
            p.seg_chunks = cut.chunks / cut.pieces;
            p.walked = p.joints = joints;
            p.first_state = p.entering = nullptr;
            p.last_state = nullptr;
            p.leaving = states + d * each;
            p.decay = decay + (size_t)d * w.streams * joints;
            p.chk = nullptr;
        }
        cudaError_t e = launch<false>(local, s, n, ways * w.streams * joints);   // (one way: without the other's CTAs)
        if (e != cudaSuccess) return e;
        lin_join_kernel<<<dim3((unsigned)((elements / 4 + 255) / 256), (unsigned)(ways * w.streams)), 256, 0, s>>>(
            w.p[0].first_state, w.p[1].first_state, states, decay, joints, elements, w.streams);
        *n += 1;
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    for (int d = 0; d < 2; ++d) {
        Params &p = w.p[d];
        p.segs = p.walked = cut.segs;
        p.seg_chunks = cut.chunks;
        p.joints = joints;
        p.pieces = cut.pieces;
        p.entering = joints ? states + d * each : nullptr;
    }
    return out ? launch<true>(w, s, n, w.streams * cut.segs) : launch<false>(w, s, n, 2 * w.streams * cut.segs);
}

Params params_of(const LinArgs &a) {
    Params p{};
    p.g = a.g; p.g_token = a.g_token; p.lens = a.lens; p.o = a.o; p.T = a.T; p.H = a.H; p.nk = a.nk; p.nv = a.nv;
    return p;
}

}  // namespace

// Of the forward (ways = 1) or of the backward's walks (2).
size_t lin_tc_workspace(int B, int T, int H, int nk, int nv, int ways) {
    const size_t walks = (size_t)ways * B * H;
    const Cut cut = cut_of(walks, T);
    const size_t joints = (size_t)(cut.segs - 1) * cut.pieces;
    return joints ? walks * ((joints + 1) * nk * nv + joints) * sizeof(float) : 0;
}

cudaError_t launch_lin_fwd_tc(const LinArgs &a, cudaStream_t s, int *n) {
    Walks w;
    if (!token_map(&w.q, a.q, a.B, a.T, a.H, a.nk) || !token_map(&w.y[0], a.k, a.B, a.T, a.H, a.nk) ||
        !token_map(&w.x[0], a.v, a.B, a.T, a.H, a.nv) || !token_map(&w.o, a.o, a.B, a.T, a.H, a.nv))
        return cudaErrorInvalidValue;
    w.y[1] = w.y[0];
    w.x[1] = w.x[0];
    w.p[0] = params_of(a);
    w.p[0].first_state = a.S0;
    w.p[0].last_state = a.S_final;
    w.p[1] = w.p[0];
    w.streams = a.B * a.H;
    return walk(w, true, static_cast<float *>(a.ws), s, n);
}

// The states that enter each chunk and the gradients of those that leave it, as bf16 operand tiles at chk and dchk; dS0.
cudaError_t launch_lin_states_tc(const LinArgs &a, uint8_t *chk, uint8_t *dchk, float *ws, cudaStream_t s, int *n) {
    Walks w;
    if (!token_map(&w.y[0], a.k, a.B, a.T, a.H, a.nk) || !token_map(&w.x[0], a.v, a.B, a.T, a.H, a.nv) ||
        !token_map(&w.y[1], a.q, a.B, a.T, a.H, a.nk) || !token_map(&w.x[1], a.dO, a.B, a.T, a.H, a.nv))
        return cudaErrorInvalidValue;
    w.q = w.y[0];
    w.o = w.x[0];
    w.p[0] = w.p[1] = params_of(a);
    w.p[0].chk = chk;
    w.p[0].first_state = a.S0;
    w.p[1].chk = dchk;
    w.p[1].back = 1;
    w.p[1].first_state = a.dS_final;
    w.p[1].last_state = a.dS0;
    w.streams = a.B * a.H;
    return walk(w, false, ws, s, n);
}

bool lin_tc_read_and_clear_timeout() {
    unsigned int v = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&v, g_lin_tc_timeout, sizeof v) != cudaSuccess) return false;
    if (v) cudaMemcpyToSymbol(g_lin_tc_timeout, &zero, sizeof zero);
    return v != 0;
}

}  // namespace qd
