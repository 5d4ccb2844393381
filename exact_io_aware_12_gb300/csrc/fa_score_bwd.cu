// Backward of attention whose scores are capped, biased by distance or masked (forward:
// fa_score_fwd.cu), with grouped heads and the gradient of a learned bias, for sm_103a.
//
// Mathematics: with x = tau q_i.k_j and y = cap tanh(x / cap) + b(h, i - j) (or x + b),
//   P = exp(y - LSE_i),  D_i = sum_j P_ij dP_ij,  dP = dO V^T,  dY = P o (dP - D),
//   dX = dY (1 - tanh^2(x / cap)),  dV = P^T dO,  dK = tau dX^T Q,  dQ = tau dX K,
// summed over the query heads that share a key head; the bias's gradient is the sum of dY
// over the pairs of each bucket.
//
// Kernels:
//   spans     documents' ranges (with documents)
//   expand    the table's biases by distance (with a table; log2 units)
//   rows      D_i and a zeroed fp32 dQ accumulator (fa_score_rows.cu)
//   main      one CTA per (128-key tile, key head).  It keeps K and V and walks the query
//             tiles that see its keys, head by head of the group, summing dK and dV in
//             tensor memory over all of them: shared heads need no sum afterwards.  Per step
//             S^T = K Q^T and dP^T = V dO^T (tcgen05), P^T and dX^T by elementwise warps (a
//             key row per thread, P^T to tensor memory, dX^T to shared memory), dV += P^T dO,
//             dQ = dX K (read out and added to the accumulator by TMA reductions), dK += dX^T Q.
//   post      dQ = bf16(tau * accumulator)
//   buckets, table   the bias's gradient (below), with a table
//
// (d = 64: the same in fa_score_bwd64.cu, with steps that overlap.)
//
// dX enters the products as bf16, rounded once from fp32; where registers are short, P (1 - tanh^2) waits for
// dP^T as fp16 of 2^15 times its value, which is off by 2^-11 of it down to 2^-29; dQ, dK, dV take
// the factor off.  With a cap and a table P itself, which dY takes, waits in the same form in tensor memory, in the
// columns that dX^T (d = 64: dQ) takes later.
//
// The bias's gradient: pairs at one distance lie on a diagonal.  A tile pair all of whose
// distances are `far` or more (most of them in a long sequence: the last bucket begins near)
// has one bucket, and its dY are summed in fp32 registers over the steps.  In the near ones
// each warp sums a 32 x 32 block's 63 diagonals: it turns column q's 32 values by q lanes (one
// shuffle), so that lane m holds the value at distance m or m - 32 of the block's.
// The sums go to memory, 64 per block, and two small kernels add them in a fixed order: no
// atomics.
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>

#include "fa_score_bwd.cuh"

namespace fa {
namespace {

constexpr int D = 128;

struct ScoreBwdLayout {
    static constexpr int kTile = kBK * D * 2;  // one bf16 [128 x D] tile
    static constexpr int kBox = 128 * 128;     // [128 rows x 64 bf16] or [128 x 32 fp32]
    static constexpr int kBoxes = D / 64;
    static constexpr int kK = 0;
    static constexpr int kV = kTile;
    static constexpr int kStage0 = 2 * kTile;    // stage s: Q at +0, dO at +kTile
    static constexpr int kStageBytes = 2 * kTile;
    static constexpr int kDS = kStage0 + 2 * kStageBytes;  // dX^T [128 keys x 128 queries] bf16
    static constexpr int kVec = kDS + 128 * 128 * 2;       // lse2[2][128], dvec[2][128]
    static constexpr int kBars = kVec + 4 * 128 * 4;
    static constexpr int kBytes = kBars + 256;
    // tensor-memory columns; dQ over dP^T, P^T and (dK's A operand) dX^T over S^T
    static constexpr uint32_t kTmDV = 0, kTmDK = D, kTmS = 2 * D, kTmDP = 2 * D + 128, kTmDQ = kTmDP;
};

struct ScoreBwdShared {
    uint64_t kv_full;
    uint64_t q_full[2];    // Q tile (and the LSE / D vectors) of stage s loaded
    uint64_t do_full[2];
    uint64_t q_empty[2];   // stage s's Q half free: MMAs done, staged dQ half read
    uint64_t do_empty[2];
    uint64_t s_full, dp_full, p_ready, ds_ready, dq_full, dq_drained;
    uint64_t dq_staged_q;   // dQ columns [0, D/2) staged over Q
    uint64_t dq_staged_do;  // dQ columns [D/2, D) staged over dO
    uint64_t dk_done;
    uint32_t tmem_base;
    int abort_flag;
};

enum : uint32_t {
    kSiteProd = 71, kSiteMmaKV = 72, kSiteMmaQ = 73, kSiteMmaP = 74, kSiteMmaDS = 75, kSiteMmaDrain = 76,
    kSiteDsS = 77, kSiteDsQ = 78, kSiteDsDP = 79, kSiteDsDQ = 80, kSiteDrain = 81, kSiteReduce = 82
};

template <int CAP, int BIAS>
__global__ void __launch_bounds__(kThreads, 1)
fa_score_bwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                    const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmdO,
                    const __grid_constant__ CUtensorMap tmdQacc, const __grid_constant__ CUtensorMap tmdK,
                    const __grid_constant__ CUtensorMap tmdV, const ScoreBwdParams p) {
    using L = ScoreBwdLayout;
    static_assert(sizeof(ScoreBwdShared) <= L::kBytes - L::kBars, "barrier block overflows its slot");
    constexpr int kProducerWarp = 4 * kNWG, kMmaWarp = 4 * kNWG + 1, kReducerWarp = 4 * kNWG + 2;
    constexpr int kDC = D / kNWG;        // d-columns of dQ, dK, dV per warpgroup
    constexpr int kEW = 128 * kNWG;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sbase = smem_addr(smem);
    ScoreBwdShared& sh = *reinterpret_cast<ScoreBwdShared*>(smem + L::kBars);
    float* lse2_s = reinterpret_cast<float*>(smem + L::kVec);        // [2][128]
    float* dvec_s = reinterpret_cast<float*>(smem + L::kVec + 1024);  // [2][128]
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int N = p.mask.N;
    // launch order: groups of head_group key heads, whose Q, dO and accumulator stay in L2; in a
    // group the key tiles in order (when causal the longest first), its heads interleaved
    int ikv, bkv;
    {
        const long long i = blockIdx.x, per_group = static_cast<long long>(p.head_group) * p.n_kv;
        const int BHkv = static_cast<int>(gridDim.x) / p.n_kv;
        const int g = static_cast<int>(i / per_group), j = static_cast<int>(i - g * per_group);
        const int heads = min(p.head_group, BHkv - g * p.head_group);
        ikv = j / heads;
        bkv = g * p.head_group + (j - ikv * heads);
    }
    const int b = bkv / p.H_kv, hkv = bkv - b * p.H_kv;
    if (sbase & 1023u) {  // the swizzled tiles need 1024-byte alignment
        if (threadIdx.x == 0) atomicCAS(p.err, 0u, 1u | (0xAAu << 8));
        return;
    }

    const uint32_t bar_kv = smem_addr(&sh.kv_full);
    const uint32_t bar_qf = smem_addr(&sh.q_full[0]);
    const uint32_t bar_df = smem_addr(&sh.do_full[0]);
    const uint32_t bar_qe = smem_addr(&sh.q_empty[0]);
    const uint32_t bar_de = smem_addr(&sh.do_empty[0]);
    const uint32_t bar_s = smem_addr(&sh.s_full);
    const uint32_t bar_dp = smem_addr(&sh.dp_full);
    const uint32_t bar_p = smem_addr(&sh.p_ready);
    const uint32_t bar_ds = smem_addr(&sh.ds_ready);
    const uint32_t bar_dq = smem_addr(&sh.dq_full);
    const uint32_t bar_dr = smem_addr(&sh.dq_drained);
    const uint32_t bar_sgq = smem_addr(&sh.dq_staged_q);
    const uint32_t bar_sgd = smem_addr(&sh.dq_staged_do);
    const uint32_t bar_dk = smem_addr(&sh.dk_done);
    if (threadIdx.x == 0) {
        sh.abort_flag = 0;
        mbar_init(bar_kv, 1);
        for (int s = 0; s < 2; ++s) {
            mbar_init(bar_qf + 8 * s, 32);
            mbar_init(bar_df + 8 * s, 1);
            mbar_init(bar_qe + 8 * s, 2);  // MMA commit + the reducer warp
            mbar_init(bar_de + 8 * s, 2);
        }
        mbar_init(bar_s, 1);
        mbar_init(bar_dp, 1);
        mbar_init(bar_p, kEW);
        mbar_init(bar_ds, kEW);
        mbar_init(bar_dq, 1);
        mbar_init(bar_dr, kEW);
        mbar_init(bar_sgq, kEW / 2);
        mbar_init(bar_sgd, kEW / 2);
        mbar_init(bar_dk, 1);
        mbar_init_fence();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(smem_addr(&sh.tmem_base), 512);
        tmem_relinquish();
    }
    if (warp == kProducerWarp && lane == 0) {
        tma_prefetch_map(&tmQ);
        tma_prefetch_map(&tmK);
        tma_prefetch_map(&tmV);
        tma_prefetch_map(&tmdO);
        tma_prefetch_map(&tmdQacc);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    griddep_launch_dependents();
    griddep_wait();  // D, the accumulator and the spans come from the kernels before
    const uint32_t tmem = sh.tmem_base;
    const Watchdog wd{p.err, &sh.abort_flag, p.wait_limit_ns};
    constexpr uint32_t FULL = 0xffffffffu;

    if (p.order) ikv = p.order[static_cast<long long>(b) * p.n_kv + ikv];
    const int kvs = ikv * kBK;
    // query tiles [first, first + per_head) see this key tile, in each of the G heads; the rows in
    // [clear_lo, clear_hi) see all of its keys.  A tile of keys that nothing sees has a step all the same
    // (its sums are 0).
    const int prefix = prefix_of(p.mask, b);
    const ScoreRange left = queries_of(p.mask, b, kvs, prefix);
    const ScoreRange right = queries_of(p.mask, b, min(kvs + kBK, N) - 1, prefix);
    const ScoreRange tiles = blocks_of(left.lo, right.hi, kBQ);
    const int clear_lo = right.lo, clear_hi = kvs + kBK > N ? 0 : left.hi;
    const int first = tiles.lo, per_head = tiles.hi - tiles.lo;
    const int steps = per_head * p.G;
    const int bh0 = b * p.H + hkv * p.G;  // the group's first query head

    if (warp == kProducerWarp) {
        // ------------------------------------------------------------ producer --
        if (lane == 0) {
            mbar_arrive_expect_tx(bar_kv, 2 * L::kTile);
            for (int x = 0; x < L::kBoxes; ++x) {
                tma_load_3d(sbase + L::kK + x * L::kBox, &tmK, bar_kv, x * 64, kvs, bkv);
                tma_load_3d(sbase + L::kV + x * L::kBox, &tmV, bar_kv, x * 64, kvs, bkv);
            }
        }
        int bh = bh0, qt = first;
        for (int s = 0; s < steps; ++s) {
            const int st = s & 1;
            const int q_start = qt * kBQ;
            const int64_t row0 = static_cast<int64_t>(bh) * N;
            // LSE and D into registers first: their latency overlaps the wait for the stage (negated,
            // for paired adds)
            float lv[4], dv[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int q = q_start + lane * 4 + e;
                lv[e] = q < N ? kLiftP - p.LSE[row0 + q] * kLog2e : -INFINITY;
                dv[e] = q < N ? -p.Dvec[row0 + q] : 0.f;
            }
            const uint32_t stage = sbase + L::kStage0 + st * L::kStageBytes;
            if (s >= 2 && !mbar_wait(bar_de + 8 * st, ((s >> 1) - 1) & 1, wd, kSiteProd)) break;
            if (lane == 0) {
                mbar_arrive_expect_tx(bar_df + 8 * st, L::kTile);
                for (int x = 0; x < L::kBoxes; ++x)
                    tma_load_3d(stage + L::kTile + x * L::kBox, &tmdO, bar_df + 8 * st, x * 64, q_start, bh);
            }
            if (s >= 2 && !mbar_wait(bar_qe + 8 * st, ((s >> 1) - 1) & 1, wd, kSiteProd)) break;
            if (lane == 0) {
                mbar_expect_tx(bar_qf + 8 * st, L::kTile);
                for (int x = 0; x < L::kBoxes; ++x)
                    tma_load_3d(stage + x * L::kBox, &tmQ, bar_qf + 8 * st, x * 64, q_start, bh);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                lse2_s[st * 128 + lane * 4 + e] = lv[e];
                dvec_s[st * 128 + lane * 4 + e] = dv[e];
            }
            mbar_arrive(bar_qf + 8 * st);  // 32 arrivals; the phase also waits for the copy
            if (++qt == first + per_head) {
                qt = first;
                ++bh;
            }
        }
    } else if (warp == kMmaWarp) {
        // ----------------------------------------------------------------- MMA --
        const uint32_t k_lo = sw128_desc_lo(sbase + L::kK, 16), k_mn = sw128_desc_lo(sbase + L::kK, kLboMN);
        const uint32_t v_lo = sw128_desc_lo(sbase + L::kV, 16);
        const uint32_t ds_mn = sw128_desc_lo(sbase + L::kDS, kLboMN);
        const uint32_t q_lo0 = sw128_desc_lo(sbase + L::kStage0, 16);
        const uint32_t q_mn0 = sw128_desc_lo(sbase + L::kStage0, kLboMN);
        const uint32_t do_lo0 = sw128_desc_lo(sbase + L::kStage0 + L::kTile, 16);
        const uint32_t do_mn0 = sw128_desc_lo(sbase + L::kStage0 + L::kTile, kLboMN);
        constexpr uint32_t kStageStep = L::kStageBytes >> 4;
        bool ok = __all_sync(FULL, mbar_wait(bar_kv, 0, wd, kSiteMmaKV) && mbar_wait(bar_qf, 0, wd, kSiteMmaQ));
        if (ok) {
            tc_fence_after();
            mma_rows_rows<D>(tmem + L::kTmS, k_lo, q_lo0);     // S^T
            mma_commit_warp(bar_s);
            ok = __all_sync(FULL, mbar_wait(bar_df, 0, wd, kSiteMmaQ));
            if (ok) {
                tc_fence_after();
                mma_rows_rows<D>(tmem + L::kTmDP, v_lo, do_lo0);   // dP^T
                mma_commit_warp(bar_dp);
            }
        }
        for (int s = 0; ok && s < steps; ++s) {
            const int st = s & 1;
            const uint32_t so = st * kStageStep;
            if (!(ok = __all_sync(FULL, mbar_wait(bar_p, s & 1, wd, kSiteMmaP)))) break;
            tc_fence_after();
            mma_tmem_a<D, kQC>(tmem + L::kTmDV, tmem + L::kTmS, do_mn0 + so, s > 0);   // dV
            mma_commit_warp(bar_de + 8 * st);  // the last MMA that reads this dO
            if (!(ok = __all_sync(FULL, mbar_wait(bar_ds, s & 1, wd, kSiteMmaDS)))) break;
            tc_fence_after();
            // dQ first: its drain is on the elementwise warps' path; dK and the next S^T run beside it
            mma_mn_mn<D>(tmem + L::kTmDQ, ds_mn, k_mn);                                // dQ
            mma_commit_warp(bar_dq);
            mma_tmem_a<D, kQC>(tmem + L::kTmDK, tmem + L::kTmS + kQC / 2, q_mn0 + so, s > 0);  // dK
            mma_commit_warp(bar_dk);
            mma_commit_warp(bar_qe + 8 * st);
            if (s + 1 < steps) {
                const int st1 = (s + 1) & 1;
                const uint32_t so1 = st1 * kStageStep;
                if (!(ok = __all_sync(FULL, mbar_wait(bar_qf + 8 * st1, ((s + 1) >> 1) & 1, wd, kSiteMmaQ)))) break;
                tc_fence_after();
                // S^T over P^T and dX^T, which only the MMAs above read (they run in issue order)
                mma_rows_rows<D>(tmem + L::kTmS, k_lo, q_lo0 + so1);
                mma_commit_warp(bar_s);
                // dP^T over the dQ tile, once it has been read out
                if (!(ok = __all_sync(FULL, mbar_wait(bar_dr, s & 1, wd, kSiteMmaDrain)))) break;
                tc_fence_after();
                if (!(ok = __all_sync(FULL, mbar_wait(bar_df + 8 * st1, ((s + 1) >> 1) & 1, wd, kSiteMmaQ)))) break;
                tc_fence_after();
                mma_rows_rows<D>(tmem + L::kTmDP, v_lo, do_lo0 + so1);
                mma_commit_warp(bar_dp);
            }
        }
        __syncwarp();
    } else if (warp == kReducerWarp) {
        // ------------------------------------------------------------- reducer --
        // adds each step's staged fp32 dQ tiles into the accumulator and hands the stage back
        if (lane == 0) {
            bool ok = true;
            int bh = bh0, qt = first;
            for (int s = 0; s < steps; ++s) {
                const int st = s & 1;
                const uint32_t src = sbase + L::kStage0 + st * L::kStageBytes;
                const int q_start = qt * kBQ;
                // dQ columns [D/2, D) were staged over dO (first), [0, D/2) over Q (once dK is done)
                if (ok) ok = mbar_wait(bar_sgd, s & 1, wd, kSiteReduce);
                if (ok) {
                    for (int x = D / 64; x < D / 32; ++x) tma_reduce_add_3d(&tmdQacc, src + x * L::kBox, x * 32, q_start, bh);
                    bulk_commit();
                }
                if (ok) ok = mbar_wait(bar_sgq, s & 1, wd, kSiteReduce);
                if (ok) {
                    for (int x = 0; x < D / 64; ++x) tma_reduce_add_3d(&tmdQacc, src + x * L::kBox, x * 32, q_start, bh);
                    bulk_commit();
                    bulk_wait_read<1>();
                }
                mbar_arrive(bar_de + 8 * st);
                if (ok) bulk_wait_read<0>();
                mbar_arrive(bar_qe + 8 * st);
                if (++qt == first + per_head) {
                    qt = first;
                    ++bh;
                }
            }
        }
        __syncwarp();
    } else {
        // ------------------------------------------ elementwise warpgroups 0 .. kNWG - 1 --
        // A failed wait poisons the rest of the work (ok = false) but every thread still reaches every
        // barrier.
        const int hw = warp >> 2;
        const int r = threadIdx.x & 127;  // key row (P^T, dX^T, dK, dV) / query row (dQ)
        const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + lane_off + L::kTmS + kQC * hw;
        const uint32_t tDP = tmem + lane_off + L::kTmDP + kQC * hw;
        const uint32_t tDQ = tmem + lane_off + L::kTmDQ + kDC * hw;
        uint8_t* ds_row = smem + L::kDS + (kQC * hw / 64) * (128 * 128) + r * 128;
        const int ds_chunk0 = (kQC * hw % 64) / 8;
        constexpr int kDrainChunks = kDC / 16;
        const int kg = kvs + r;
        // the queries that see this row's key (none past a ragged end)
        const ScoreRange mine = kg < N ? queries_of(p.mask, b, kg, prefix) : ScoreRange{0, 0};
        // the table gradient's sums of far pairs, kept while steps stay on one side
        [[maybe_unused]] uint64_t fsum = 0;
        [[maybe_unused]] int fside = 0;
        const bool grad = BIAS == kBiasTable && p.near_part != nullptr;
        [[maybe_unused]] const auto flush = [&](int bh) {
            const float2 f = f2_unpack(fsum);
            const float fs = warp_sum(f.x + f.y);
            if (lane == 0)
                p.far_part[((static_cast<long long>(bh) * p.n_kv + ikv) * (4 * kNWG) + warp) * kFarFloats + (fside > 0)] = fs;
            fsum = 0;
        };
        bool ok = true;
        int s = 0;
        for (int g = 0; g < p.G; ++g) {
            const int bh = bh0 + g;
            [[maybe_unused]] float slope2 = 0.f;
            [[maybe_unused]] const float* bias2 = nullptr;
            if constexpr (BIAS == kBiasSlopes) slope2 = p.slopes[hkv * p.G + g] * kLog2e;
            if constexpr (BIAS == kBiasTable) bias2 = p.bias2 + static_cast<long long>(hkv * p.G + g) * (2 * p.far + 1);
            if (grad) {
                // what no step of this head writes is zero
                const long long at = static_cast<long long>(bh) * p.n_kv + ikv;
                if (lane < kFarFloats) p.far_part[(at * (4 * kNWG) + warp) * kFarFloats + lane] = 0.f;
                __syncwarp();
                for (int x = 0; x < p.near_n; ++x) {
                    const int qt = ikv + p.near_lo + x;
                    if (qt >= 0 && qt < p.n_kv && (qt < first || qt >= first + per_head))
                        for (int i = threadIdx.x; i < kNearFloats; i += kEW)
                            p.near_part[(at * p.near_n + x) * kNearFloats + i] = 0.f;
                }
                fside = 0;
            }
            for (int t = 0; t < per_head; ++t, ++s) {
                const int st = s & 1;
                const int q_start = (first + t) * kBQ;
                const ulonglong2* nl4 = reinterpret_cast<const ulonglong2*>(lse2_s + st * 128 + kQC * hw);
                uint32_t keep[keep_regs(CAP, BIAS)];  // P (1 - tanh^2)
                [[maybe_unused]] const int side = far_side(q_start, kvs, kBQ, BIAS == kBiasTable ? p.far : 0);
                [[maybe_unused]] uint64_t far_bias = 0;
                if constexpr (BIAS == kBiasTable) {
                    if (side != 0) {
                        const float v = bias2[side > 0 ? 2 * p.far : 0];
                        far_bias = f2_pack(v, v);
                    }
                }
                if (ok)
                    ok = __all_sync(FULL, mbar_wait_sleep(bar_qf + 8 * st, (s >> 1) & 1, wd, kSiteDsQ) &&
                                              mbar_wait_sleep(bar_s, s & 1, wd, kSiteDsS));
                if (ok) {
                    tc_fence_after();
                    const int qh = q_start + kQC * hw;
                    const bool general = q_start < clear_lo || q_start + kBQ > clear_hi || (BIAS != kBiasNone && side == 0);
                    const BwdRow row{kg, mine.lo, static_cast<uint32_t>(mine.hi - mine.lo), general, side, slope2, bias2, far_bias};
                    uint32_t sv[32], pk[16], pw[16];
                    tmem_ld32(tS, sv);
                    tmem_ld_wait(sv);
                    bwd_weights<CAP, BIAS>(p, row, sv, nl4, qh, pk, keep, pw);
                    tmem_st16(tS, pk);
                    if constexpr (CAP && BIAS == kBiasTable) tmem_st16(tS + kQC / 2, pw);  // (until dX takes its columns)
                    tmem_st_wait();
                    tc_fence_before();
                }
                mbar_arrive(bar_p);

                const ulonglong2* nd4 = reinterpret_cast<const ulonglong2*>(dvec_s + st * 128 + kQC * hw);
                if (ok)
                    ok = __all_sync(FULL, mbar_wait_sleep(bar_dp, s & 1, wd, kSiteDsDP) &&
                                              (s == 0 || mbar_wait_sleep(bar_dq, (s - 1) & 1, wd, kSiteDsDQ)));
                if (ok) {
                    tc_fence_after();
                    if (grad && side != fside) {
                        if (fside != 0) flush(bh);
                        fside = side;
                    }
                    uint32_t dp[32], ds[16];
                    tmem_ld32(tDP, dp);
                    [[maybe_unused]] uint32_t pw[16];  // CAP: P itself, fp16
                    if constexpr (CAP && BIAS == kBiasTable) {
                        tmem_ld16(tS + kQC / 2, pw);
                        tmem_ld_wait(pw);
                    }
                    tmem_ld_wait(dp);
                    [[maybe_unused]] float ahead = 0.f, behind = 0.f;
                    if (BIAS == kBiasTable && grad && side != 0)
                        bwd_products<CAP, BIAS == kBiasTable>(dp, keep, pw, nd4, lane, ds, fsum, ahead, behind);
                    else if (BIAS == kBiasTable && grad)
                        bwd_products<CAP, BIAS == kBiasTable ? 2 : 0>(dp, keep, pw, nd4, lane, ds, fsum, ahead, behind);
                    else
                        bwd_products<CAP, 0>(dp, keep, pw, nd4, lane, ds, fsum, ahead, behind);
                    if constexpr (BIAS == kBiasTable) {
                        if (grad && side == 0) {
                            // block (query block, key block) of 32: lane m holds distance m, and m - 32
                            const long long at = (static_cast<long long>(bh) * p.n_kv + ikv) * p.near_n + (first + t - ikv - p.near_lo);
                            float* dst = p.near_part + at * kNearFloats + (hw * 4 + (warp & 3)) * 64;
                            dst[lane] = ahead;
                            dst[32 + lane] = behind;
                        }
                    }
                    tmem_st16(tS + kQC / 2, ds);
#pragma unroll
                    for (int q4 = 0; q4 < 4; ++q4) {
                        const int chunk = ds_chunk0 + q4;
                        *reinterpret_cast<uint4*>(ds_row + ((chunk ^ (r & 7)) << 4)) =
                            make_uint4(ds[4 * q4], ds[4 * q4 + 1], ds[4 * q4 + 2], ds[4 * q4 + 3]);
                    }
                    fence_async_shared();
                    tmem_st_wait();
                    tc_fence_before();
                }
                mbar_arrive(bar_ds);

                // dQ drain: this warpgroup's columns -> fp32 tiles -> bulk reduce-add
                if (ok) ok = __all_sync(FULL, mbar_wait_sleep(bar_dq, s & 1, wd, kSiteDrain));
                uint8_t* stage = smem + L::kStage0 + st * L::kStageBytes;
                uint32_t acc[kDrainChunks][16];
                if (ok) {
                    tc_fence_after();
#pragma unroll
                    for (int x = 0; x < kDrainChunks; ++x) tmem_ld16(tDQ + 16 * x, acc[x]);
#pragma unroll
                    for (int x = 0; x < kDrainChunks; ++x) tmem_ld_wait(acc[x]);
                    tc_fence_before();
                    mbar_arrive(bar_dr);
                    // staged over dO (free: dV and dP^T come before dQ) and over Q (free once dK is done)
                    if (hw < kNWG / 2) ok = __all_sync(FULL, mbar_wait_sleep(bar_dk, s & 1, wd, kSiteDrain));
                } else {
                    mbar_arrive(bar_dr);
                }
                if (ok) {
#pragma unroll
                    for (int x = 0; x < kDrainChunks; ++x) {
                        const int col = hw * kDC + 16 * x;
                        uint8_t* box = stage + (col / 32) * L::kBox + r * 128;
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            *reinterpret_cast<uint4*>(box + ((((col % 32) / 4 + j) ^ (r & 7)) << 4)) =
                                make_uint4(acc[x][4 * j], acc[x][4 * j + 1], acc[x][4 * j + 2], acc[x][4 * j + 3]);
                    }
                    fence_async_shared();
                }
                mbar_arrive(hw >= kNWG / 2 ? bar_sgd : bar_sgq);
            }
            if (grad && fside != 0) flush(bh);
        }
        // dK = tau * dK_acc and dV, staged over the K and V tiles once the last dK is done (its commit
        // covers every MMA of this CTA)
        if (ok) ok = __all_sync(FULL, mbar_wait_sleep(bar_dk, (steps - 1) & 1, wd, kSiteDrain));
        if (ok) {
            tc_fence_after();
#pragma unroll
            for (int which = 0; which < 2; ++which) {
                uint8_t* dst = smem + (which ? L::kK : L::kV);
                const float scale = (which ? (CAP ? -p.tau : p.tau) : 1.f) * kUnliftP;
                const uint32_t src = tmem + lane_off + (which ? L::kTmDK : L::kTmDV);
#pragma unroll
                for (int cc = 0; cc < kDC; cc += 16) {
                    const int c0 = hw * kDC + cc;
                    uint32_t o[16];
                    tmem_ld16(src + c0, o);
                    tmem_ld_wait(o);
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const int chunk = (c0 % 64) / 8 + q;
                        uint4 v;
                        v.x = pack_bf16(u2f(o[8 * q + 0]) * scale, u2f(o[8 * q + 1]) * scale);
                        v.y = pack_bf16(u2f(o[8 * q + 2]) * scale, u2f(o[8 * q + 3]) * scale);
                        v.z = pack_bf16(u2f(o[8 * q + 4]) * scale, u2f(o[8 * q + 5]) * scale);
                        v.w = pack_bf16(u2f(o[8 * q + 6]) * scale, u2f(o[8 * q + 7]) * scale);
                        *reinterpret_cast<uint4*>(dst + (c0 / 64) * L::kBox + r * 128 + ((chunk ^ (r & 7)) << 4)) = v;
                    }
                }
            }
            fence_async_shared();
        }
        // (all warps reach this barrier, also after a failed wait, and agree)
        if (!named_bar_or(4, kEW, !ok) && threadIdx.x == 0) {
            for (int x = 0; x < L::kBoxes; ++x) {
                tma_store_3d(&tmdV, sbase + L::kV + x * L::kBox, x * 64, kvs, bkv);
                tma_store_3d(&tmdK, sbase + L::kK + x * L::kBox, x * 64, kvs, bkv);
            }
            bulk_commit();
            bulk_wait_read<0>();
        }
    }

    // -------------------------------------------------------------- teardown --
    if (sh.abort_flag) drain_after_abort();
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// The table's biases by distance, [H][2 far + 1] in log2 units.
__global__ void __launch_bounds__(256) fa_score_expand_kernel(const void* table, int f32, const int* buckets, int num_buckets, int H,
                                                              int far, float* bias2) {
    griddep_launch_dependents();
    griddep_wait();
    const int n = 2 * far + 1, h = static_cast<int>(blockIdx.x), i = static_cast<int>(blockIdx.y) * 256 + threadIdx.x;
    if (i < n) bias2[static_cast<long long>(h) * n + i] = kLog2e * table_bias(table, f32, buckets, num_buckets, H, h, i);
}

// dQ = bf16(scale * acc), 8 elements per thread, grid-stride.
__global__ void __launch_bounds__(256) fa_score_post_kernel(const float* acc, __nv_bfloat16* dQ, float scale, int64_t n8) {
    griddep_launch_dependents();
    griddep_wait();
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n8; i += static_cast<int64_t>(gridDim.x) * 256) {
        const float4 a = reinterpret_cast<const float4*>(acc)[2 * i];
        const float4 b = reinterpret_cast<const float4*>(acc)[2 * i + 1];
        uint4 o;
        o.x = pack_bf16(a.x * scale, a.y * scale);
        o.y = pack_bf16(a.z * scale, a.w * scale);
        o.z = pack_bf16(b.x * scale, b.y * scale);
        o.w = pack_bf16(b.z * scale, b.w * scale);
        reinterpret_cast<uint4*>(dQ)[i] = o;
    }
}

struct TableGradParams {
    const float* near_part;
    const float* far_part;
    float* red;       // [near_n kParts][H][num_buckets] sums per bucket; then [H][2] of the far parts
    const int* buckets;
    void* out;        // [num_buckets][H]
    int B, H, n_kv, near_lo, near_n, far_warps, far, num_buckets, out_f32;
};

// Block (head, x): x < near_n kParts adds the diagonals of the tile pairs at offset near_lo + x / kParts, of a part of
// the batch and the key tiles, in order, and then, bucket by bucket, the diagonals of each; the last
// block adds the far parts.  (One block for all of an offset's tiles read 256 KB by itself, 24 us.)
constexpr int kParts = 8;
__global__ void __launch_bounds__(1024) fa_score_buckets_kernel(const TableGradParams p) {
    __shared__ float val[kNearFloats];
    __shared__ int of[kNearFloats];
    griddep_launch_dependents();
    griddep_wait();
    const int x = static_cast<int>(blockIdx.y), h = static_cast<int>(blockIdx.x);
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
    if (x == p.near_n * kParts) {
        const long long parts = static_cast<long long>(p.n_kv) * p.far_warps;
        float sum = 0.f;
        for (int b = 0; b < p.B; ++b) {
            const float* src = p.far_part + (static_cast<long long>(b) * p.H + h) * parts * kFarFloats;
            for (long long i = t >> 1; i < parts; i += 512) sum += src[i * kFarFloats + (t & 1)];
        }
        val[t] = sum;
        __syncthreads();
        if (warp < 2) {
            float s = 0.f;
            for (int i = lane; i < 512; i += 32) s += val[2 * i + warp];
            s = warp_sum(s);
            if (lane == 0) p.red[static_cast<long long>(p.near_n) * kParts * p.H * p.num_buckets + h * 2 + warp] = s;
        }
        return;
    }
    const int off = p.near_lo + x / kParts;  // query tile - key tile
    const int k0 = max(0, -off), nk = min(p.n_kv, p.n_kv - off) - k0;  // key tiles of each sequence
    const long long all = static_cast<long long>(p.B) * nk;
    const int i0 = static_cast<int>(all * (x % kParts) / kParts), i1 = static_cast<int>(all * (x % kParts + 1) / kParts);
    float sum = 0.f;
    int b = nk > 0 ? i0 / nk : 0, k = i0 - b * nk;
#pragma unroll 8
    for (int i = i0; i < i1; ++i) {
        sum += p.near_part[(((static_cast<long long>(b) * p.H + h) * p.n_kv + k + k0) * p.near_n + x / kParts) * kNearFloats + t];
        if (++k == nk) {
            k = 0;
            ++b;
        }
    }
    const int blk = t >> 6, m = t & 63;
    const int dist = off * 128 + 32 * (blk / 4 - blk % 4) + (m < 32 ? m : m - 64);
    val[t] = sum;
    of[t] = p.buckets[max(0, min(2 * p.far, dist + p.far))];
    __syncthreads();
    float* dst = p.red + (static_cast<long long>(x) * p.H + h) * p.num_buckets;
    for (int e = warp; e < p.num_buckets; e += 32) {
        float s = 0.f;
        for (int i = lane; i < kNearFloats; i += 32)
            if (of[i] == e) s += val[i];
        s = warp_sum(s);
        if (lane == 0) dst[e] = s;
    }
}

// Block h: the gradient of head h's biases.
__global__ void __launch_bounds__(256) fa_score_table_kernel(const TableGradParams p) {
    griddep_launch_dependents();
    griddep_wait();
    const int h = static_cast<int>(blockIdx.x), nb = p.num_buckets;
    const long long step = static_cast<long long>(p.H) * nb;
    const float* red = p.red + static_cast<long long>(h) * nb;
    const int parts = p.near_n * kParts;
    const float* far = p.red + parts * step + h * 2;  // far keys behind the query's tiles, and before
    const int low = p.buckets[0], high = p.buckets[2 * p.far];
    for (int e = threadIdx.x; e < nb; e += 256) {
        float s = 0.f;
#pragma unroll 8
        for (int x = 0; x < parts; ++x) s += red[x * step + e];
        if (e == low) s += far[0];
        if (e == high) s += far[1];
        s *= kUnliftP;
        if (p.out_f32) static_cast<float*>(p.out)[static_cast<long long>(e) * p.H + h] = s;
        else static_cast<__nv_bfloat16*>(p.out)[static_cast<long long>(e) * p.H + h] = __float2bfloat16_rn(s);
    }
}

size_t up(size_t x) { return (x + 255) / 256 * 256; }

// grad: with the parts of the table's gradient (4 KB per near tile pair and head, most of what such a call takes).
BwdPlan plan_of(const ScoreArgs& a, bool grad) {
    BwdPlan pl;
    const size_t rows = static_cast<size_t>(a.B) * a.H * a.N;
    const int n_kv = (a.N + kBK - 1) / kBK;
    pl.acc = up(rows * sizeof(float));
    pl.next = pl.acc + up(rows * a.d * sizeof(float));
    pl.spans = pl.next + up(sizeof(int));
    pl.order = pl.spans + (a.mod.docs ? score_spans_bytes(a.B, a.N) : 0);  // of pairs, then of key tiles
    pl.bias2 = pl.order + (a.mod.docs ? up(static_cast<size_t>(a.B) * (n_kv + (n_kv + 1) / 2) * sizeof(int)) : 0);
    pl.near = pl.far = pl.red = pl.bytes = pl.bias2;
    if (!a.mod.table) return pl;
    pl.near = pl.bias2 + up(static_cast<size_t>(a.H) * (2 * a.mod.far + 1) * sizeof(float));
    pl.far = pl.red = pl.bytes = pl.near;
    if (!grad) return pl;
    // (offsets that tiles have; behind the query only where a prefix, or no mask, shows such keys)
    const int n = std::min(near_tiles(a.mod.far, kBQ), n_kv - 1);
    pl.near_lo = a.causal && !a.mod.prefix ? 0 : -n;
    pl.near_n = n - pl.near_lo + 1;
    pl.warps = 4 * kNWG;
    const size_t tiles = static_cast<size_t>(a.B) * a.H * n_kv;
    pl.far = pl.near + tiles * pl.near_n * kNearFloats * sizeof(float);
    pl.red = pl.far + up(tiles * pl.warps * kFarFloats * sizeof(float));
    pl.bytes = pl.red + up((static_cast<size_t>(pl.near_n) * kParts * a.H * a.mod.num_buckets + a.H * 2) * sizeof(float));
    return pl;
}

// Key heads per launch-order group: what the resident CTAs read (K, V, and of each query head of the
// group Q, dO and the accumulator) within L2, as the backward without biases was measured.
int head_group(const ScoreArgs& a) {
    const double budget = (a.causal ? 128.0 : 48.0) * 1024 * 1024;
    const double per_head = static_cast<double>(a.N) * a.d * (4.0 + 8.0 * a.H / a.H_kv);
    int g = 1;
    while (g < 16 && 2.0 * g * per_head <= budget) g *= 2;
    return std::max(1, std::min(a.B * a.H_kv, g));
}

ScoreBwdParams params_of(const ScoreArgs& a, const BwdPlan& pl) {
    const bool cap = a.mod.softcap > 0.f;
    ScoreBwdParams p;
    p.LSE = a.LSE;
    p.Dvec = reinterpret_cast<const float*>(a.workspace + pl.dvec);
    p.H = a.H;
    p.H_kv = a.H_kv;
    p.BHkv = a.B * a.H_kv;
    p.G = a.H / a.H_kv;
    p.n_kv = (a.N + kBK - 1) / kBK;
    p.head_group = head_group(a);
    p.order = a.mod.docs ? reinterpret_cast<const int*>(a.workspace + pl.order) + static_cast<size_t>(a.B) * ((p.n_kv + 1) / 2) : nullptr;
    p.mask.spans = a.mod.docs ? reinterpret_cast<const int2*>(a.workspace + pl.spans) : nullptr;
    p.mask.prefix = a.mod.prefix;
    p.mask.N = a.N;
    p.mask.window = a.mod.window;
    p.mask.causal = a.causal;
    p.scale_log2 = a.tau * kLog2e;
    p.tau = a.tau;
    p.x_scale = cap ? a.tau / a.mod.softcap : 0.f;
    p.cap_log2 = a.mod.softcap * kLog2e;
    p.slopes = a.mod.slopes;
    p.bias2 = reinterpret_cast<const float*>(a.workspace + pl.bias2);
    p.far = a.mod.far;
    p.near_part = a.dTable ? reinterpret_cast<float*>(a.workspace + pl.near) : nullptr;
    p.far_part = reinterpret_cast<float*>(a.workspace + pl.far);
    p.near_lo = pl.near_lo;
    p.near_n = pl.near_n;
    p.next = reinterpret_cast<unsigned*>(a.workspace + pl.next);
    p.err = a.err;
    p.wait_limit_ns = a.wait_limit_ns;
    return p;
}

template <int CAP, int BIAS>
cudaError_t launch_main(const ScoreArgs& a, const ScoreBwdParams& p, float* acc, cudaStream_t stream) {
    using L = ScoreBwdLayout;
    CUtensorMap tq, tk, tv, tdo, tacc, tdk, tdv;
    const auto BF = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const int BH = a.B * a.H, BHkv = p.BHkv;
    if (!make_tile_map(&tq, a.Q, BF, 2, D, a.N, BH, 64, kBQ) || !make_tile_map(&tk, a.K, BF, 2, D, a.N, BHkv, 64, kBK) ||
        !make_tile_map(&tv, a.V, BF, 2, D, a.N, BHkv, 64, kBK) || !make_tile_map(&tdo, a.dO, BF, 2, D, a.N, BH, 64, kBQ) ||
        !make_tile_map(&tacc, acc, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, D, a.N, BH, 32, kBQ) ||
        !make_tile_map(&tdk, a.dK, BF, 2, D, a.N, BHkv, 64, kBK) || !make_tile_map(&tdv, a.dV, BF, 2, D, a.N, BHkv, 64, kBK))
        return cudaErrorInvalidValue;
    constexpr auto kern = &fa_score_bwd_kernel<CAP, BIAS>;
    cudaError_t e = set_max_dyn_smem_once<kern>(L::kBytes);
    if (e != cudaSuccess) return e;
    if (a.ev_start) cudaEventRecord(a.ev_start, stream);
    e = launch_dependent(kern, dim3(static_cast<unsigned>(BHkv) * static_cast<unsigned>(p.n_kv)),
                         dim3(kThreads), L::kBytes, stream, tq, tk, tv, tdo, tacc, tdk, tdv, p);
    if (e == cudaSuccess && a.ev_stop) e = cudaEventRecord(a.ev_stop, stream);
    return e;
}

template <int CAP>
cudaError_t launch_c(const ScoreArgs& a, const ScoreBwdParams& p, float* acc, cudaStream_t stream) {
    return a.mod.slopes  ? launch_main<CAP, kBiasSlopes>(a, p, acc, stream)
           : a.mod.table ? launch_main<CAP, kBiasTable>(a, p, acc, stream)
                         : launch_main<CAP, kBiasNone>(a, p, acc, stream);
}

cudaError_t launch_all(const ScoreArgs& a, const BwdPlan& pl, cudaStream_t stream) {
    const int64_t rows = static_cast<int64_t>(a.B) * a.H * a.N;
    const ScoreBwdParams p = params_of(a, pl);
    float* bias2 = reinterpret_cast<float*>(a.workspace + pl.bias2);
    float* acc = reinterpret_cast<float*>(a.workspace + pl.acc);
    cudaError_t e = cudaSuccess;
    if (a.mod.table) {
        const dim3 grid(static_cast<unsigned>(a.H), static_cast<unsigned>((2 * a.mod.far + 256) / 256));
        e = launch_dependent(fa_score_expand_kernel, grid, dim3(256), 0, stream, a.mod.table,
                             static_cast<int>(a.mod.table_f32), a.mod.buckets, a.mod.num_buckets, a.H, a.mod.far, bias2);
        if (e != cudaSuccess) return e;
    }
    e = launch_score_rows(a, reinterpret_cast<float*>(a.workspace + pl.dvec), acc, p.next, a.mod.docs ? a.workspace + pl.spans : nullptr,
                          a.mod.docs ? reinterpret_cast<const int*>(a.workspace + pl.order) : nullptr, bias2, stream);
    if (e != cudaSuccess) return e;
    const bool cap = a.mod.softcap > 0.f;
    if (a.d == 64) e = launch_score_bwd64(a, p, acc, stream);
    else if (cap_of(a.mod.softcap) == kCapNone) e = launch_c<kCapNone>(a, p, acc, stream);
    else if (cap_of(a.mod.softcap) == kCapCommon) e = launch_c<kCapCommon>(a, p, acc, stream);
    else e = launch_c<kCapLarge>(a, p, acc, stream);
    if (e != cudaSuccess) return e;
    const int64_t n8 = rows * a.d / 8;
    return launch_dependent(fa_score_post_kernel, dim3(static_cast<unsigned>(std::min<int64_t>((n8 + 255) / 256, 152 * 64))),
                            dim3(256), 0, stream, static_cast<const float*>(acc), static_cast<__nv_bfloat16*>(a.dQ),
                            (cap ? -a.tau : a.tau) * kUnliftP, n8);
}

}  // namespace

size_t score_bwd_workspace(const ScoreArgs& a, bool grad) { return plan_of(a, grad).bytes; }

cudaError_t launch_score_bwd(const ScoreArgs& a, cudaStream_t stream) {
    const BwdPlan pl = plan_of(a, a.dTable != nullptr);
    cudaError_t e = cudaSuccess;
    if (a.mod.docs) {
        ScoreOrder order;
        order.pairs = reinterpret_cast<int*>(a.workspace + pl.order);
        order.keys = order.pairs + static_cast<size_t>(a.B) * ((a.N + 2 * kBQ - 1) / (2 * kBQ));
        e = launch_score_spans(a, a.workspace + pl.spans, order, stream);
    }
    if (e == cudaSuccess) e = launch_all(a, pl, stream);
    if (e != cudaSuccess || !a.dTable) return e;
    TableGradParams t;
    t.near_part = reinterpret_cast<const float*>(a.workspace + pl.near);
    t.far_part = reinterpret_cast<const float*>(a.workspace + pl.far);
    t.red = reinterpret_cast<float*>(a.workspace + pl.red);
    t.buckets = a.mod.buckets;
    t.out = a.dTable;
    t.B = a.B;
    t.H = a.H;
    t.n_kv = (a.N + kBK - 1) / kBK;
    t.near_lo = pl.near_lo;
    t.near_n = pl.near_n;
    t.far_warps = pl.warps;
    t.far = a.mod.far;
    t.num_buckets = a.mod.num_buckets;
    t.out_f32 = a.mod.table_f32;
    e = launch_dependent(fa_score_buckets_kernel, dim3(static_cast<unsigned>(t.H), static_cast<unsigned>(t.near_n * kParts + 1)), dim3(1024),
                         0, stream, t);
    if (e != cudaSuccess) return e;
    return launch_dependent(fa_score_table_kernel, dim3(static_cast<unsigned>(t.H)), dim3(256), 0, stream, t);
}

}  // namespace fa
