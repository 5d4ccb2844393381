// Main kernel of the backward of attention with capped, biased or masked scores at d = 64 (the
// mathematics, and the other kernels: fa_score_bwd.cu), for sm_103a.
//
// At d = 64 a step's five products take 0.7 us and its elementwise work 1.1 to 1.8, so the
// kernel is bound by what the elementwise warps issue and wait for.  Half the columns of d = 128's accumulators leave
// room in tensor memory for the scores of two steps, and in shared memory for the keys and values of two
// tiles:
//   - one CTA per SM walks over tiles (key tile, key head), the next one's number from a counter in
//     memory, and its steps run on from tile to tile: K, V and the first S of the next tile are in
//     before the last tile's dK and dV are out.
//   - S of step s + 1 is computed while step s is worked on, and dP of s + 1 as soon as dP of s has been read.
//   - P^T lies packed over the first half of its S, so dQ of the step takes the second half, and is read
//     out in the middle of the next step.  (All four warps of a row read their scores before the first
//     writes its P: a barrier of theirs.)
//
// Measured against a CTA per tile and one step's scores in tensor memory: 96 heads of 1024 tokens with slopes
// 78 -> 60 us, 48 heads of up to 2048 with a table 221 -> 190, 16 of 8192 with window 4096 capped (with D)
// 603 -> 542.  Arrivals by one thread of a warp (551 us for 544 of the last) and dQ staged behind one fence with
// dX (452 us for 415 without a cap) are slower.
//
// A step s of tile t, in an elementwise warp: P of s; dQ of s - 1 read out; if s is the tile's first, dK and dV
// of tile t - 1; dX of s.  In the MMA warp: dV of s, S of s + 1, dQ of s, dP of s + 1, dK of s.
#include <algorithm>

#include "fa_score_bwd.cuh"

namespace fa {
namespace {

constexpr int kSms = 152;  // of a GB300
constexpr int D = 64;

struct Bwd64Layout {
    static constexpr int kTile = 128 * D * 2;  // one bf16 tile, and one [128 rows x 32] of fp32
    static constexpr int kKV = 0;                      // K and V of tile t at (t & 1) 2 kTile
    static constexpr int kQ = 4 * kTile;               // Q of step s at s % 3
    static constexpr int kDO = kQ + 3 * kTile;         // dO at s % 2
    static constexpr int kDS = kDO + 2 * kTile;        // dX^T [128 keys x 128 queries] bf16
    static constexpr int kStage = kDS + 2 * kTile;     // dQ, fp32
    static constexpr int kVec = kStage + 2 * kTile;    // 15 - LSE log2(e) [3][128], -D [3][128]
    static constexpr int kMine = kVec + 6 * 128 * 4;   // [2][128] queries that see a key
    static constexpr int kBars = kMine + 2 * 128 * 8;
    static constexpr int kBytes = kBars + 512;
    // tensor-memory columns; P^T and dQ of a step over its S
    static constexpr uint32_t kTmDV = 0, kTmDK = 64, kTmS = 128, kTmDP = 384, kTmDQ = 64;
};

struct Bwd64Tile {
    int ikv, bkv, first, per_head;  // per_head 0: no more
    int clear_lo, clear_hi;
};

struct Bwd64Shared {
    uint64_t kv_full[2];   // K, V and the tile's numbers
    uint64_t kv_empty[2];  // dK and dV, staged over them, are read
    uint64_t q_full[3];    // Q and the vectors
    uint64_t q_empty[3];
    uint64_t do_full[2];
    uint64_t do_empty[2];
    uint64_t s_full[2];
    uint64_t s_read[4];    // of 32 key rows: their warps have their scores
    uint64_t p_ready, dp_full, ds_ready, dq_full, dq_drained;
    uint64_t dk_done;      // and dP of the next step
    uint64_t acc_free;     // dK and dV of the last tile are read out
    uint64_t staged, stage_free, out;  // dQ staged, reduced; dK and dV staged
    Bwd64Tile tile[2];
    uint32_t tmem_base;
    int abort_flag;
};
static_assert(sizeof(Bwd64Shared) <= Bwd64Layout::kBytes - Bwd64Layout::kBars, "barrier block overflows its slot");

enum : uint32_t {
    kSiteProd = 101, kSiteTile = 102, kSiteMmaQ = 103, kSiteMmaP = 104, kSiteMmaDS = 105, kSiteMmaDrain = 106,
    kSiteEwS = 107, kSiteEwDP = 108, kSiteDrain = 109, kSiteReduce = 110
};

template <int CAP, int BIAS>
__global__ void __launch_bounds__(kThreads, 1)
fa_score_bwd64_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmdO,
                      const __grid_constant__ CUtensorMap tmdQacc, const __grid_constant__ CUtensorMap tmdK,
                      const __grid_constant__ CUtensorMap tmdV, const ScoreBwdParams p) {
    using L = Bwd64Layout;
    constexpr int kProducerWarp = 4 * kNWG, kMmaWarp = 4 * kNWG + 1, kReducerWarp = 4 * kNWG + 2;
    constexpr int kDC = D / kNWG;    // d-columns of dQ, dK, dV per warpgroup
    constexpr int kEW = 128 * kNWG;
    constexpr uint32_t FULL = 0xffffffffu;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sbase = smem_addr(smem);
    Bwd64Shared& sh = *reinterpret_cast<Bwd64Shared*>(smem + L::kBars);
    float* lse2_s = reinterpret_cast<float*>(smem + L::kVec);  // [3][128]
    float* dvec_s = lse2_s + 3 * 128;                          // [3][128]
    int2* mine_s = reinterpret_cast<int2*>(smem + L::kMine);   // [2][128]
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int N = p.mask.N;
    if (sbase & 1023u) {  // the swizzled tiles need 1024-byte alignment
        if (threadIdx.x == 0) atomicCAS(p.err, 0u, 1u | (0xAAu << 8));
        return;
    }

    const uint32_t bar_kvf = smem_addr(&sh.kv_full[0]), bar_kve = smem_addr(&sh.kv_empty[0]);
    const uint32_t bar_qf = smem_addr(&sh.q_full[0]), bar_qe = smem_addr(&sh.q_empty[0]);
    const uint32_t bar_df = smem_addr(&sh.do_full[0]), bar_de = smem_addr(&sh.do_empty[0]);
    const uint32_t bar_s = smem_addr(&sh.s_full[0]), bar_sr = smem_addr(&sh.s_read[0]);
    const uint32_t bar_p = smem_addr(&sh.p_ready), bar_dp = smem_addr(&sh.dp_full), bar_ds = smem_addr(&sh.ds_ready);
    const uint32_t bar_dq = smem_addr(&sh.dq_full), bar_dr = smem_addr(&sh.dq_drained), bar_dk = smem_addr(&sh.dk_done);
    const uint32_t bar_acc = smem_addr(&sh.acc_free);
    const uint32_t bar_st = smem_addr(&sh.staged), bar_sf = smem_addr(&sh.stage_free), bar_out = smem_addr(&sh.out);
    if (threadIdx.x == 0) {
        sh.abort_flag = 0;
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar_kvf + 8 * i, 32);
            mbar_init(bar_kve + 8 * i, 1);
            mbar_init(bar_df + 8 * i, 1);
            mbar_init(bar_de + 8 * i, 1);
            mbar_init(bar_s + 8 * i, 1);
        }
        for (int i = 0; i < 3; ++i) {
            mbar_init(bar_qf + 8 * i, 32);
            mbar_init(bar_qe + 8 * i, 1);
        }
        for (int i = 0; i < 4; ++i) mbar_init(bar_sr + 8 * i, kNWG);
        mbar_init(bar_p, kEW);
        mbar_init(bar_dp, 1);
        mbar_init(bar_ds, kEW);
        mbar_init(bar_dq, 1);
        mbar_init(bar_dr, kEW);
        mbar_init(bar_dk, 1);
        mbar_init(bar_acc, kEW);
        mbar_init(bar_st, kEW);
        mbar_init(bar_sf, 1);
        mbar_init(bar_out, kEW);
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
    griddep_wait();  // D, the accumulator, the counter and the spans come from the kernels before
    const uint32_t tmem = sh.tmem_base;
    const Watchdog wd{p.err, &sh.abort_flag, p.wait_limit_ns};
    // (a warp whose wait fails leaves; the others' waits then end, too, and all meet at the end)
    const auto tile_in = [&](int t) { return __all_sync(FULL, mbar_wait(bar_kvf + 8 * (t & 1), (t >> 1) & 1, wd, kSiteTile)); };

    if (warp == kProducerWarp) {
        // ------------------------------------------------------------ producer --
        const unsigned tiles = static_cast<unsigned>(p.BHkv) * p.n_kv;
        unsigned next = blockIdx.x;
        int s = 0;
        bool ok = true;
        for (int t = 0; ok; ++t) {
            const int buf = t & 1;
            const uint32_t bar = bar_kvf + 8 * buf;
            if (t >= 2 && !(ok = __all_sync(FULL, mbar_wait(bar_kve + 8 * buf, ((t >> 1) - 1) & 1, wd, kSiteProd)))) break;
            if (next >= tiles) {
                if (lane == 0) sh.tile[buf].per_head = 0;
                mbar_arrive(bar);
                break;
            }
            unsigned after = 0;
            if (lane == 0) after = gridDim.x + atomicAdd(p.next, 1u);
            // order: groups of head_group key heads, whose Q, dO and accumulator stay in L2; in a group
            // the key tiles in order (when causal the longest first), its heads interleaved
            const long long per_group = static_cast<long long>(p.head_group) * p.n_kv;
            const int g = static_cast<int>(next / per_group), j = static_cast<int>(next - g * per_group);
            const int heads = min(p.head_group, p.BHkv - g * p.head_group);
            int ikv = j / heads;
            const int bkv = g * p.head_group + (j - ikv * heads);
            const int b = bkv / p.H_kv, hkv = bkv - b * p.H_kv;
            if (p.order) ikv = p.order[static_cast<long long>(b) * p.n_kv + ikv];
            const int kvs = ikv * kBK;
            if (lane == 0) {
                const uint32_t at = sbase + L::kKV + buf * 2 * L::kTile;
                mbar_expect_tx(bar, 2 * L::kTile);
                tma_load_3d(at, &tmK, bar, 0, kvs, bkv);
                tma_load_3d(at + L::kTile, &tmV, bar, 0, kvs, bkv);
            }
            // query tiles [first, first + per_head) see this key tile, in each of the G heads; the rows in
            // [clear_lo, clear_hi) see all of its keys.  A tile of keys that nothing sees has a step all
            // the same (its sums are 0).
            const int prefix = prefix_of(p.mask, b);
            const ScoreRange left = queries_of(p.mask, b, kvs, prefix);
            const ScoreRange right = queries_of(p.mask, b, min(kvs + kBK, N) - 1, prefix);
            const ScoreRange range = blocks_of(left.lo, right.hi, kBQ);
            const int first = range.lo, per_head = range.hi - range.lo;
            if (lane == 0) sh.tile[buf] = {ikv, bkv, first, per_head, right.lo, kvs + kBK > N ? 0 : left.hi};
#pragma unroll
            for (int e = 0; e < 4; ++e) {  // (none past a ragged end)
                const int r = e * 32 + lane, kg = kvs + r;
                const ScoreRange m = kg < N ? queries_of(p.mask, b, kg, prefix) : ScoreRange{0, 0};
                mine_s[buf * 128 + r] = make_int2(m.lo, m.hi);
            }
            mbar_arrive(bar);  // 32 arrivals; the phase also waits for the copies
            int bh = b * p.H + hkv * p.G, qt = first;
            const int steps = per_head * p.G;
            for (int i = 0; i < steps; ++i, ++s) {
                const int q_start = qt * kBQ;
                const int64_t row0 = static_cast<int64_t>(bh) * N;
                // LSE and D into registers first: their latency overlaps the wait for the slot (negated,
                // for paired adds)
                float lv[4], dv[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int q = q_start + lane * 4 + e;
                    lv[e] = q < N ? kLiftP - p.LSE[row0 + q] * kLog2e : -INFINITY;
                    dv[e] = q < N ? -p.Dvec[row0 + q] : 0.f;
                }
                const int sq = s % 3, sd = s & 1;
                if (s >= 3 && !(ok = __all_sync(FULL, mbar_wait(bar_qe + 8 * sq, (s / 3 - 1) & 1, wd, kSiteProd)))) break;
                if (lane == 0) {
                    mbar_expect_tx(bar_qf + 8 * sq, L::kTile);
                    tma_load_3d(sbase + L::kQ + sq * L::kTile, &tmQ, bar_qf + 8 * sq, 0, q_start, bh);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    lse2_s[sq * 128 + lane * 4 + e] = lv[e];
                    dvec_s[sq * 128 + lane * 4 + e] = dv[e];
                }
                mbar_arrive(bar_qf + 8 * sq);
                if (s >= 2 && !(ok = __all_sync(FULL, mbar_wait(bar_de + 8 * sd, ((s >> 1) - 1) & 1, wd, kSiteProd)))) break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(bar_df + 8 * sd, L::kTile);
                    tma_load_3d(sbase + L::kDO + sd * L::kTile, &tmdO, bar_df + 8 * sd, 0, q_start, bh);
                }
                if (++qt == first + per_head) {
                    qt = first;
                    ++bh;
                }
            }
            next = __shfl_sync(FULL, after, 0);
        }
        __syncwarp();
    } else if (warp == kMmaWarp) {
        // ----------------------------------------------------------------- MMA --
        constexpr uint32_t kStep = L::kTile >> 4;
        const uint32_t k_lo = sw128_desc_lo(sbase + L::kKV, 16), k_mn = sw128_desc_lo(sbase + L::kKV, kLboMN);
        const uint32_t v_lo = sw128_desc_lo(sbase + L::kKV + L::kTile, 16);
        const uint32_t ds_mn = sw128_desc_lo(sbase + L::kDS, kLboMN), ds_lo = sw128_desc_lo(sbase + L::kDS, 16);
        const uint32_t q_lo = sw128_desc_lo(sbase + L::kQ, 16), q_mn = sw128_desc_lo(sbase + L::kQ, kLboMN);
        const uint32_t do_lo = sw128_desc_lo(sbase + L::kDO, 16), do_mn = sw128_desc_lo(sbase + L::kDO, kLboMN);
        const auto wait = [&](uint32_t bar, int parity, uint32_t site) {
            const bool in = __all_sync(FULL, mbar_wait(bar, parity & 1, wd, site));
            tc_fence_after();
            return in;
        };
        const auto issue_s = [&](int s, int t) {
            mma_rows_rows<D>(tmem + L::kTmS + 128 * (s & 1), k_lo + (t & 1) * 2 * kStep, q_lo + s % 3 * kStep);
            mma_commit_warp(bar_s + 8 * (s & 1));
        };
        const auto issue_dp = [&](int s, int t) {
            mma_rows_rows<D>(tmem + L::kTmDP, v_lo + (t & 1) * 2 * kStep, do_lo + (s & 1) * kStep);
        };
        int t = 0, left = 0;  // the tile, its steps from this one on
        bool ok = tile_in(0), first = true;
        if (ok) left = sh.tile[0].per_head * p.G;
        if (ok && (ok = wait(bar_qf, 0, kSiteMmaQ))) {
            issue_s(0, 0);
            if ((ok = wait(bar_df, 0, kSiteMmaQ))) {
                issue_dp(0, 0);
                mma_commit_warp(bar_dp);
            }
        }
        for (int s = 0; ok; ++s) {
            const uint32_t tS = tmem + L::kTmS + 128 * (s & 1);
            if (!(ok = wait(bar_p, s, kSiteMmaP))) break;
            if (first && t > 0 && !(ok = wait(bar_acc, t - 1, kSiteMmaDrain))) break;
            mma_tmem_a<D, 128>(tmem + L::kTmDV, tS, do_mn + (s & 1) * kStep, !first);  // dV
            mma_commit_warp(bar_de + 8 * (s & 1));  // the last MMA that reads this dO
            // S of the next step, over what dQ of the last has been read out of
            int t1 = t, left1 = left - 1;
            if (left1 == 0) {
                t1 = t + 1;
                if (!(ok = tile_in(t1))) break;
                left1 = sh.tile[t1 & 1].per_head * p.G;
            }
            if (s > 0 && !(ok = wait(bar_dr, s - 1, kSiteMmaDrain))) break;
            if (left1 > 0) {
                if (!(ok = wait(bar_qf + 8 * ((s + 1) % 3), (s + 1) / 3, kSiteMmaQ))) break;
                issue_s(s + 1, t1);
            }
            if (!(ok = wait(bar_ds, s, kSiteMmaDS))) break;
            mma_mn_mn<D>(tS + L::kTmDQ, ds_mn, k_mn + (t & 1) * 2 * kStep);  // dQ
            mma_commit_warp(bar_dq);
            if (left1 > 0) {
                if (!(ok = wait(bar_df + 8 * ((s + 1) & 1), (s + 1) >> 1, kSiteMmaQ))) break;
                issue_dp(s + 1, t1);
            }
            mma_rows_mn<D>(tmem + L::kTmDK, ds_lo, q_mn + s % 3 * kStep, !first);  // dK
            mma_commit_warp(bar_dk);
            mma_commit_warp(bar_qe + 8 * (s % 3));
            if (left1 == 0) break;
            first = t1 != t;
            t = t1;
            left = left1;
        }
        __syncwarp();
    } else if (warp == kReducerWarp) {
        // ------------------------------------------------------------- reducer --
        // adds each step's staged fp32 dQ to the accumulator, stores each tile's staged dK and dV
        int s = 0;
        bool ok = true;
        for (int t = 0; ok && (ok = tile_in(t)); ++t) {
            const Bwd64Tile tile = sh.tile[t & 1];
            if (tile.per_head == 0) break;
            if (lane == 0) {
                const int b = tile.bkv / p.H_kv, hkv = tile.bkv - b * p.H_kv;
                int bh = b * p.H + hkv * p.G, qt = tile.first;
                const int steps = tile.per_head * p.G;
                for (int i = 0; i < steps; ++i, ++s) {
                    if (!(ok = mbar_wait(bar_st, s & 1, wd, kSiteReduce))) break;
                    for (int x = 0; x < 2; ++x) tma_reduce_add_3d(&tmdQacc, sbase + L::kStage + x * L::kTile, x * 32, qt * kBQ, bh);
                    bulk_commit();
                    bulk_wait_read<0>();
                    mbar_arrive(bar_sf);
                    if (++qt == tile.first + tile.per_head) {
                        qt = tile.first;
                        ++bh;
                    }
                }
                if (ok && (ok = mbar_wait(bar_out, t & 1, wd, kSiteReduce))) {
                    const uint32_t at = sbase + L::kKV + (t & 1) * 2 * L::kTile;
                    tma_store_3d(&tmdK, at, 0, tile.ikv * kBK, tile.bkv);
                    tma_store_3d(&tmdV, at + L::kTile, 0, tile.ikv * kBK, tile.bkv);
                    bulk_commit();
                    bulk_wait_read<0>();
                    mbar_arrive(bar_kve + 8 * (t & 1));
                }
            }
            ok = __shfl_sync(FULL, static_cast<int>(ok), 0);
        }
        __syncwarp();
    } else {
        // ------------------------------------------ elementwise warpgroups 0 .. kNWG - 1 --
        const int hw = warp >> 2;
        const int r = threadIdx.x & 127;  // key row (P^T, dX^T, dK, dV) / query row (dQ)
        const uint32_t lanes = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        const uint32_t tDP = lanes + L::kTmDP + kQC * hw;
        uint8_t* ds_row = smem + L::kDS + (kQC * hw / 64) * (128 * 128) + r * 128;
        const int ds_chunk0 = (kQC * hw % 64) / 8;
        // of two barriers at once: a vote, and what comes with it, takes 100 cycles
        const auto wait2 = [&](uint32_t bar0, int parity0, uint32_t bar1, int parity1, uint32_t site) {
            bool in = mbar_try_wait(bar0, parity0 & 1) & mbar_try_wait(bar1, parity1 & 1);
            if (!__all_sync(FULL, in))
                in = __all_sync(FULL, mbar_wait_sleep(bar0, parity0 & 1, wd, site) && mbar_wait_sleep(bar1, parity1 & 1, wd, site));
            tc_fence_after();
            return in;
        };
        const auto wait = [&](uint32_t bar, int parity, uint32_t site) {
            const bool in = __all_sync(FULL, mbar_wait_sleep(bar, parity & 1, wd, site));
            tc_fence_after();
            return in;
        };
        // dQ of step s1 (and the wait for what follows it): this warpgroup's columns -> an fp32 tile -> bulk reduce-add
        const auto drain = [&](int s1) {
            if (!wait2(bar_dq, s1, s1 > 0 ? bar_sf : bar_dq, s1 > 0 ? s1 - 1 : s1, kSiteDrain)) return false;
            uint32_t acc[kDC];
            tmem_ld16(lanes + L::kTmS + 128 * (s1 & 1) + L::kTmDQ + hw * kDC, acc);
            tmem_ld_wait(acc);
            tc_fence_before();
            mbar_arrive(bar_dr);
            uint8_t* box = smem + L::kStage + (hw * kDC / 32) * L::kTile + r * 128;
#pragma unroll
            for (int j = 0; j < kDC / 4; ++j)
                *reinterpret_cast<uint4*>(box + (((hw * kDC % 32 / 4 + j) ^ (r & 7)) << 4)) =
                    make_uint4(acc[4 * j], acc[4 * j + 1], acc[4 * j + 2], acc[4 * j + 3]);
            fence_async_shared();
            mbar_arrive(bar_st);
            return wait(bar_dk, s1, kSiteDrain);
        };
        // dK = tau * dK_acc and dV of tile t1, whose products are done, staged over its K and V
        const auto finish = [&](int t1) {
            uint8_t* dst = smem + L::kKV + (t1 & 1) * 2 * L::kTile + r * 128;
#pragma unroll
            for (int which = 0; which < 2; ++which) {
                const float scale = (which ? 1.f : (CAP ? -p.tau : p.tau)) * kUnliftP;
                const uint32_t src = lanes + (which ? L::kTmDV : L::kTmDK) + hw * kDC;
#pragma unroll
                for (int c0 = 0; c0 < kDC; c0 += 16) {
                    uint32_t o[16];
                    tmem_ld16(src + c0, o);
                    tmem_ld_wait(o);
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        uint4 v;
                        v.x = pack_bf16(u2f(o[8 * q + 0]) * scale, u2f(o[8 * q + 1]) * scale);
                        v.y = pack_bf16(u2f(o[8 * q + 2]) * scale, u2f(o[8 * q + 3]) * scale);
                        v.z = pack_bf16(u2f(o[8 * q + 4]) * scale, u2f(o[8 * q + 5]) * scale);
                        v.w = pack_bf16(u2f(o[8 * q + 6]) * scale, u2f(o[8 * q + 7]) * scale);
                        *reinterpret_cast<uint4*>(dst + which * L::kTile + ((((hw * kDC + c0) / 8 + q) ^ (r & 7)) << 4)) = v;
                    }
                }
            }
            tc_fence_before();
            mbar_arrive(bar_acc);
        };
        // the table gradient's sums of far pairs, kept while steps stay on one side
        [[maybe_unused]] uint64_t fsum = 0;
        [[maybe_unused]] int fside = 0;
        const bool grad = BIAS == kBiasTable && p.near_part != nullptr;
        int s = 0;  // of all tiles
        const auto walk = [&]() {
            for (int t = 0;; ++t) {
                if (!tile_in(t)) return;
                const Bwd64Tile tile = sh.tile[t & 1];
                if (tile.per_head == 0) {
                    if (t > 0 && drain(s - 1)) {
                        finish(t - 1);
                        fence_async_shared();
                        mbar_arrive(bar_out);
                    }
                    return;
                }
                const int2 mine = mine_s[(t & 1) * 128 + r];
                const int b = tile.bkv / p.H_kv, hkv = tile.bkv - b * p.H_kv;
                const int kvs = tile.ikv * kBK, kg = kvs + r;
                for (int g = 0; g < p.G; ++g) {
                    const int h = hkv * p.G + g;
                    [[maybe_unused]] const long long at = static_cast<long long>(b * p.H + h) * p.n_kv + tile.ikv;
                    [[maybe_unused]] const auto flush = [&]() {
                        const float2 f = f2_unpack(fsum);
                        const float fs = warp_sum(f.x + f.y);
                        if (lane == 0) p.far_part[(at * (4 * kNWG) + warp) * kFarFloats + (fside > 0)] = fs;
                        fsum = 0;
                    };
                    BwdRow row{kg, mine.x, static_cast<uint32_t>(mine.y - mine.x), false, 0, 0.f, nullptr, 0};
                    if constexpr (BIAS == kBiasSlopes) row.slope2 = p.slopes[h] * kLog2e;
                    if constexpr (BIAS == kBiasTable) row.bias2 = p.bias2 + static_cast<long long>(h) * (2 * p.far + 1);
                    if (grad) {
                        // what no step of this head writes is zero
                        if (lane < kFarFloats) p.far_part[(at * (4 * kNWG) + warp) * kFarFloats + lane] = 0.f;
                        __syncwarp();
                        for (int x = 0; x < p.near_n; ++x) {
                            const int qt = tile.ikv + p.near_lo + x;
                            if (qt >= 0 && qt < p.n_kv && (qt < tile.first || qt >= tile.first + tile.per_head))
                                for (int i = threadIdx.x; i < kNearFloats; i += kEW) p.near_part[(at * p.near_n + x) * kNearFloats + i] = 0.f;
                        }
                        fside = 0;
                    }
                    for (int i = 0; i < tile.per_head; ++i, ++s) {
                        const int q_start = (tile.first + i) * kBQ, qh = q_start + kQC * hw;
                        const uint32_t tS = lanes + L::kTmS + 128 * (s & 1);
                        [[maybe_unused]] const uint32_t tPW = tS + L::kTmDQ + kQC / 2 * hw;  // (until dQ takes its columns)
                        uint32_t keep[keep_regs(CAP, BIAS)];  // P (1 - tanh^2)
                        row.side = far_side(q_start, kvs, kBQ, BIAS == kBiasTable ? p.far : 0);
                        row.general = q_start < tile.clear_lo || q_start + kBQ > tile.clear_hi || (BIAS != kBiasNone && row.side == 0);
                        if constexpr (BIAS == kBiasTable) {
                            if (row.side != 0) {
                                const float v = row.bias2[row.side > 0 ? 2 * p.far : 0];
                                row.far_bias = f2_pack(v, v);
                            }
                        }
                        if (!wait2(bar_qf + 8 * (s % 3), s / 3, bar_s + 8 * (s & 1), s >> 1, kSiteEwS)) return;
                        {
                            uint32_t sv[32];
                            tmem_ld32(tS + kQC * hw, sv);
                            tmem_ld_wait(sv);
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(bar_sr + 8 * (warp & 3));
                            const ulonglong2* nl4 = reinterpret_cast<const ulonglong2*>(lse2_s + s % 3 * 128 + kQC * hw);
                            uint32_t pk[16], pw[16];
                            bwd_weights<CAP, BIAS>(p, row, sv, nl4, qh, pk, keep, pw);
                            if (!wait(bar_sr + 8 * (warp & 3), s, kSiteEwS)) return;
                            tmem_st16(tS + kQC / 2 * hw, pk);
                            if constexpr (CAP && BIAS == kBiasTable) tmem_st16(tPW, pw);
                            tmem_st_wait();
                            tc_fence_before();
                            mbar_arrive(bar_p);
                        }

                        const bool last = s > 0 && g == 0 && i == 0;  // of the tile before: its dK and dV
                        if (s == 0) {
                            if (!wait(bar_dp, 0, kSiteEwDP)) return;
                        } else if (!drain(s - 1)) {  // (dP is in, and dX^T's tile is free again, too)
                            return;
                        }
                        if (last) finish(t - 1);

                        const ulonglong2* nd4 = reinterpret_cast<const ulonglong2*>(dvec_s + s % 3 * 128 + kQC * hw);
                        if (grad && row.side != fside) {
                            if (fside != 0) flush();
                            fside = row.side;
                        }
                        uint32_t dp[32], ds[16];
                        tmem_ld32(tDP, dp);
                        [[maybe_unused]] uint32_t pw[16];  // CAP: P itself, fp16
                        if constexpr (CAP && BIAS == kBiasTable) {
                            tmem_ld16(tPW, pw);
                            tmem_ld_wait(pw);
                        }
                        tmem_ld_wait(dp);
                        [[maybe_unused]] float ahead = 0.f, behind = 0.f;
                        if (BIAS == kBiasTable && grad && row.side != 0)
                            bwd_products<CAP, BIAS == kBiasTable>(dp, keep, pw, nd4, lane, ds, fsum, ahead, behind);
                        else if (BIAS == kBiasTable && grad)
                            bwd_products<CAP, BIAS == kBiasTable ? 2 : 0>(dp, keep, pw, nd4, lane, ds, fsum, ahead, behind);
                        else
                            bwd_products<CAP, 0>(dp, keep, pw, nd4, lane, ds, fsum, ahead, behind);
                        if constexpr (BIAS == kBiasTable) {
                            if (grad && row.side == 0) {
                                // block (query block, key block) of 32: lane m holds distance m, and m - 32
                                float* dst = p.near_part + (at * p.near_n + (tile.first + i - tile.ikv - p.near_lo)) * kNearFloats +
                                             (hw * 4 + (warp & 3)) * 64;
                                dst[lane] = ahead;
                                dst[32 + lane] = behind;
                            }
                        }
#pragma unroll
                        for (int q4 = 0; q4 < 4; ++q4)
                            *reinterpret_cast<uint4*>(ds_row + (((ds_chunk0 + q4) ^ (r & 7)) << 4)) =
                                make_uint4(ds[4 * q4], ds[4 * q4 + 1], ds[4 * q4 + 2], ds[4 * q4 + 3]);
                        fence_async_shared();
                        tc_fence_before();
                        mbar_arrive(bar_ds);
                        if (last) mbar_arrive(bar_out);
                    }
                    if (grad && fside != 0) flush();
                }
            }
        };
        walk();
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

template <int CAP, int BIAS>
cudaError_t launch_t(const ScoreArgs& a, const ScoreBwdParams& p, float* acc, cudaStream_t stream) {
    CUtensorMap tq, tk, tv, tdo, tacc, tdk, tdv;
    const auto BF = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const int BH = a.B * a.H, BHkv = p.BHkv;
    if (!make_tile_map(&tq, a.Q, BF, 2, D, a.N, BH, 64, kBQ) || !make_tile_map(&tk, a.K, BF, 2, D, a.N, BHkv, 64, kBK) ||
        !make_tile_map(&tv, a.V, BF, 2, D, a.N, BHkv, 64, kBK) || !make_tile_map(&tdo, a.dO, BF, 2, D, a.N, BH, 64, kBQ) ||
        !make_tile_map(&tacc, acc, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, D, a.N, BH, 32, kBQ) ||
        !make_tile_map(&tdk, a.dK, BF, 2, D, a.N, BHkv, 64, kBK) || !make_tile_map(&tdv, a.dV, BF, 2, D, a.N, BHkv, 64, kBK))
        return cudaErrorInvalidValue;
    constexpr auto kern = &fa_score_bwd64_kernel<CAP, BIAS>;
    cudaError_t e = set_max_dyn_smem_once<kern>(Bwd64Layout::kBytes);
    if (e != cudaSuccess) return e;
    const long long tiles = static_cast<long long>(BHkv) * p.n_kv;
    if (a.ev_start) cudaEventRecord(a.ev_start, stream);
    e = launch_dependent(kern, dim3(static_cast<unsigned>(std::min<long long>(tiles, kSms))), dim3(kThreads),
                         Bwd64Layout::kBytes, stream, tq, tk, tv, tdo, tacc, tdk, tdv, p);
    if (e == cudaSuccess && a.ev_stop) e = cudaEventRecord(a.ev_stop, stream);
    return e;
}

template <int CAP>
cudaError_t launch_c(const ScoreArgs& a, const ScoreBwdParams& p, float* acc, cudaStream_t stream) {
    return a.mod.slopes  ? launch_t<CAP, kBiasSlopes>(a, p, acc, stream)
           : a.mod.table ? launch_t<CAP, kBiasTable>(a, p, acc, stream)
                         : launch_t<CAP, kBiasNone>(a, p, acc, stream);
}

}  // namespace

cudaError_t launch_score_bwd64(const ScoreArgs& a, const ScoreBwdParams& p, float* acc, cudaStream_t stream) {
    switch (cap_of(a.mod.softcap)) {
        case kCapNone: return launch_c<kCapNone>(a, p, acc, stream);
        case kCapCommon: return launch_c<kCapCommon>(a, p, acc, stream);
        default: return launch_c<kCapLarge>(a, p, acc, stream);
    }
}

}  // namespace fa
