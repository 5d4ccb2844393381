// Forward of attention whose scores are capped by a tanh, biased by distance or masked by
// documents, a prefix or a window, with grouped heads, for sm_103a.
//
// Mathematics: with x = tau q_i.k_j, the score of a visible pair is
//   y = cap tanh(x / cap) (or x) + b(h, i - j),
// b a slope times the distance or an entry of a learned table by bucket of distance;
// O = sum_j softmax_j(y) v_j by the online recurrence, LSE = ln sum_j exp(y_ij).  Which keys
// a query sees is one range of positions (fa_score.h), so a tile's mask is one unsigned
// compare per score, and needed only where a tile is not wholly visible.
//
// Design: one CTA per 128-row query tile and query head, two CTAs to an SM (256 of its 512
// tensor-memory columns each), so that one's loads, S and P V products and epilogue run
// beside the other's softmax: per score the mask, the cap (6 to 8 operations on the fp32 pipe; see
// tanh2), the bias, one exponential and two sums, against the 2 x 128 x 128 x d products of a tile pair.
// What bounds it is each CTA's chain S -> softmax -> P V -> S at d = 128 (16 heads of 16384 tokens, window 4096:
// 367 us without a cap, 535 with, and no less where a sum or the exponential is left out), a score's
// instructions at d = 64 (half of the issue slots, with the waits of the same chain).
//   - Softmax warpgroups (WGS): one, a row per thread; or two, half of a row's keys each, with one CTA to an
//     SM, where tiles are few (launch_t).  The next warp streams Q, K_j and V_j by TMA through a ring of
//     slots, the last issues S = Q K_j^T and O += P V_j (tcgen05, P read from tensor memory).  At d = 64,
//     P has columns of its own and the next S is issued as soon as the softmax has read the last; at d = 128
//     it is written over S.
//   - The query heads that share a key head are neighbours in launch order, so that its
//     keys are read from L2; longest tiles first when causal.
//   - Capped scores without a bias: the maximum is found before the cap, which keeps the order,
//     and the cap's last multiply-add takes the reference off.
//   - Slopes: a tile on one side of its queries adds slope * column, the same for all rows, from
//     shared memory; what is left, slope times the distance of the first column, goes into
//     the row's reference.
//   - Table: the head's biases by distance, 2 far + 1 of them, lie in shared memory; a
//     tile all of whose pairs are at `far` or more has one bias.
//   - A row that sees nothing keeps its reference at -inf: its weights and its sum stay 0,
//     O = 0 and LSE = -inf.
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>

#include "fa_score.cuh"

namespace fa {
namespace {

constexpr int kSms = 152;  // of a GB300
constexpr int kBM = 128, kBN = 128;
constexpr int threads_for(int wgs) { return 128 * wgs + 64; }
constexpr float kLn2 = 0.69314718055994531f;
constexpr float kLog2e = 1.44269504088896341f;
constexpr float kRescaleThreshold = 8.0f;  // log2 units: P stays <= 2^8

template <int D>
struct ScoreFwdLayout {
    static constexpr int kTile = kBM * D * 2;    // one bf16 tile
    static constexpr int kBox = 128 * 128;       // one [128 rows x 64 columns] TMA box
    static constexpr int kBoxes = D / 64;
    static constexpr int kStages = D == 64 ? 4 : 2;
    static constexpr int kRing = kTile;
    static constexpr int kTable = kRing + kStages * kTile;
    static constexpr int kDynSmem = kTable + 1024;  // + alignment slack; + the table's biases
    static constexpr uint32_t kTmS = 0, kTmO = 128, kTmCols = 256;
    static constexpr bool kPipe = D == 64;       // P in columns of its own
    static constexpr uint32_t kTmP = kPipe ? 192 : 0;
};

struct ScoreFwdParams {
    float* LSE;
    int H, G, n_q;  // query heads, those to a key head, query tiles
    const int* order;  // [B][n_q], or null: from the last
    ScoreMask mask;
    float scale_log2;  // tau * log2(e)
    CapScale cap;
    const float* slopes;
    const void* table;
    const int* buckets;
    int table_f32, num_buckets, far;
    unsigned int* err;
    unsigned long long wait_limit_ns;
};

struct ScoreFwdShared {
    uint64_t q_full;
    uint64_t kv_full[4];
    uint64_t kv_empty[4];
    uint64_t s_full, s_free, p_ready, o_done;
    __align__(16) float ramp[2][128];  // slopes: +-slope log2(e) times the column
    float top[2][2][128];  // two warpgroups: [block's parity][warpgroup][row], largest score
    float sum[2][2][128];  // [l, l_mma][warpgroup][row], at the end
    uint32_t tmem_base;
    int abort_flag;
};

enum : uint32_t {
    kSiteProd = 61, kSiteMmaQ = 62, kSiteMmaKV = 63, kSiteMmaS = 64, kSiteMmaP = 65,
    kSiteSoftS = 66, kSiteSoftO = 67, kSiteEpi = 68
};

__device__ __forceinline__ float u2f(uint32_t x) { return __uint_as_float(x); }
__device__ __forceinline__ uint32_t f2u(float x) { return __float_as_uint(x); }

constexpr uint32_t kDescHi = sw128_desc_hi(1024);

// (volatile: loads of the whole ramp ahead of its use would take the scores' registers)
__device__ __forceinline__ ulonglong2 lds_2x64(uint32_t a) {
    ulonglong2 v;
    asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(v.x), "=l"(v.y) : "r"(a));
    return v;
}

// A thread's scores, in registers, two at a time: f(column, pair) -> pair.
template <int N, typename F>
__device__ __forceinline__ void each_pair(uint32_t (&s)[N][32], F&& f) {
#pragma unroll
    for (int c = 0; c < 32 * N; c += 2) {
        uint32_t &a = s[c >> 5][c & 31], &b = s[c >> 5][(c & 31) + 1];
        const float2 y = f2_unpack(f(c, f2_pack(u2f(a), u2f(b))));
        a = f2u(y.x);
        b = f2u(y.y);
    }
}

template <int D, int CAP, int BIAS, int WGS>
__global__ void __launch_bounds__(threads_for(WGS), WGS == 1 ? 2 : 1)
fa_score_fwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                    const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmO,
                    const ScoreFwdParams p) {
    using L = ScoreFwdLayout<D>;
    [[maybe_unused]] constexpr int kFar = far_form(CAP);
    constexpr bool PIPE = L::kPipe;
    constexpr int kProducerWarp = 4 * WGS, kMmaWarp = 4 * WGS + 1;
    constexpr int kSoftmax = 128 * WGS, kCols = 128 / WGS, kParts = kCols / 32;  // threads; keys of a block per thread
    extern __shared__ uint8_t smem_raw[];
    __shared__ ScoreFwdShared sh;
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t pad = ((raw + 1023u) & ~1023u) - raw;
    uint8_t* smem = smem_raw + pad;
    const uint32_t sbase = raw + pad;
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int N = p.mask.N;
    const int bh = static_cast<int>(blockIdx.x);
    const int b = bh / p.H, h = bh - b * p.H;
    const int bkv = b * (p.H / p.G) + h / p.G;

    const uint32_t bar_q = smem_addr(&sh.q_full);
    const uint32_t bar_kvf = smem_addr(&sh.kv_full[0]);
    const uint32_t bar_kve = smem_addr(&sh.kv_empty[0]);
    const uint32_t bar_s = smem_addr(&sh.s_full);
    const uint32_t bar_sf = smem_addr(&sh.s_free);
    const uint32_t bar_p = smem_addr(&sh.p_ready);
    const uint32_t bar_o = smem_addr(&sh.o_done);
    if (threadIdx.x == 0) {
        sh.abort_flag = 0;
        mbar_init(bar_q, 1);
        for (int s = 0; s < L::kStages; ++s) {
            mbar_init(bar_kvf + 8 * s, 1);
            mbar_init(bar_kve + 8 * s, 1);
        }
        mbar_init(bar_s, 1);
        mbar_init(bar_sf, kSoftmax);
        mbar_init(bar_p, kSoftmax);
        mbar_init(bar_o, 1);
        mbar_init_fence();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(smem_addr(&sh.tmem_base), L::kTmCols);
        tmem_relinquish();
    }
    if (warp == kProducerWarp && lane == 0) {
        tma_prefetch_map(&tmQ);
        tma_prefetch_map(&tmK);
        tma_prefetch_map(&tmV);
        tma_prefetch_map(&tmO);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // launched as a dependent of the kernel before it: its start-up overlaps that kernel's end
    griddep_launch_dependents();
    griddep_wait();
    const uint32_t tmem = sh.tmem_base;
    const Watchdog wd{p.err, &sh.abort_flag, p.wait_limit_ns};
    const int rank = static_cast<int>(blockIdx.y);
    const int q_start = (p.order ? p.order[static_cast<long long>(b) * p.n_q + rank] : p.n_q - 1 - rank) * kBM;

    // key blocks [jlo, jlo + nb); those within [clear_lo, clear_hi) every row sees
    const int prefix = prefix_of(p.mask, b);
    const ScoreRange top = keys_of(p.mask, b, q_start, prefix);
    const ScoreRange bottom = keys_of(p.mask, b, min(q_start + kBM, N) - 1, prefix);
    const ScoreRange blocks = blocks_of(top.lo, bottom.hi, kBN);
    const int clear_lo = bottom.lo, clear_hi = top.hi;
    const int jlo = blocks.lo, nb = blocks.hi - blocks.lo;

    if (warp == kProducerWarp) {
        // ------------------------------------------------------------ producer --
        if (lane == 0) {
            mbar_arrive_expect_tx(bar_q, L::kTile);
            for (int x = 0; x < L::kBoxes; ++x) tma_load_3d(sbase + x * L::kBox, &tmQ, bar_q, x * 64, q_start, bh);
            for (int ld = 0; ld < 2 * nb; ++ld) {
                const int slot = ld % L::kStages;
                if (ld >= L::kStages && !mbar_wait(bar_kve + 8 * slot, ((ld / L::kStages) - 1) & 1, wd, kSiteProd)) break;
                bool is_k = (ld & 1) == 0;
                int blk = ld >> 1;
                if constexpr (PIPE) {  // the MMA warp's order: K0 K1 V0 K2 V1 ... K(nb-1) V(nb-2) V(nb-1)
                    is_k = ld == 0 || ((ld & 1) && ld < 2 * nb - 1);
                    blk = is_k ? (ld + 1) / 2 : (ld == 2 * nb - 1 ? nb - 1 : ld / 2 - 1);
                }
                mbar_arrive_expect_tx(bar_kvf + 8 * slot, L::kTile);
                for (int x = 0; x < L::kBoxes; ++x)
                    tma_load_3d(sbase + L::kRing + slot * L::kTile + x * L::kBox, is_k ? &tmK : &tmV, bar_kvf + 8 * slot,
                                x * 64, (jlo + blk) * kBN, bkv);
            }
        }
        __syncwarp();
    } else if (warp == kMmaWarp) {
        // ----------------------------------------------------------------- MMA --
        const uint32_t tS = tmem + L::kTmS, tO = tmem + L::kTmO, tP = tmem + L::kTmP;
        const uint32_t qlo = sw128_desc_lo(sbase, 16);
        const uint32_t klo0 = sw128_desc_lo(sbase + L::kRing, 16);          // K: K-major
        const uint32_t vlo0 = sw128_desc_lo(sbase + L::kRing, 128 * 128);   // V: MN-major
        constexpr uint32_t kSlot = L::kTile >> 4;
        constexpr uint32_t id_s = idesc_bf16(128, 128, false, false);
        constexpr uint32_t id_pv = idesc_bf16(128, D, false, true);
        const auto issue_s = [&](int slot) {
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                const uint32_t off = ((k / 4) * (128 * 128) + (k % 4) * 32) >> 4;
                if (k == 0) mma_ss_warp<0>(tS, qlo + off, klo0 + slot * kSlot + off, kDescHi, id_s);
                else mma_ss_warp<1>(tS, qlo + off, klo0 + slot * kSlot + off, kDescHi, id_s);
            }
            mma_commit_warp(bar_s);
            mma_commit_warp(bar_kve + 8 * slot);
        };
        const auto issue_pv = [&](int slot, bool accumulate) {
            if (accumulate) mma_ts_warp<1>(tO, tP, vlo0 + slot * kSlot, kDescHi, id_pv);
            else mma_ts_warp<0>(tO, tP, vlo0 + slot * kSlot, kDescHi, id_pv);
#pragma unroll
            for (int k = 1; k < kBN / 16; ++k)
                mma_ts_warp<1>(tO, tP + (PIPE || WGS == 1 ? k * 8 : (k / 4) * kCols + (k % 4) * 8), vlo0 + slot * kSlot + ((k * 2048) >> 4), kDescHi, id_pv);
            mma_commit_warp(bar_o);
            mma_commit_warp(bar_kve + 8 * slot);
        };
        const auto kv_in = [&](int ld) { return mbar_wait(bar_kvf + 8 * (ld % L::kStages), (ld / L::kStages) & 1, wd, kSiteMmaKV); };
        bool ok = __all_sync(0xffffffffu, mbar_wait(bar_q, 0, wd, kSiteMmaQ));
        for (int j = 0; ok && j <= nb; ++j) {
            if (PIPE && j < nb) {  // S of block j, once the softmax has read S of j - 1
                const int ld = j == 0 ? 0 : 2 * j - 1;
                ok = __all_sync(0xffffffffu, kv_in(ld) && (j == 0 || mbar_wait(bar_sf, (j - 1) & 1, wd, kSiteMmaS)));
                if (!ok) break;
                tc_fence_after();
                issue_s(ld % L::kStages);
            }
            if (j > 0) {  // P V of block j - 1
                const int ld = !PIPE ? 2 * j - 1 : min(2 * j, 2 * nb - 1);
                ok = __all_sync(0xffffffffu, kv_in(ld) && mbar_wait(bar_p, (j - 1) & 1, wd, kSiteMmaP));
                if (!ok) break;
                tc_fence_after();
                issue_pv(ld % L::kStages, j > 1);
            }
            if (!PIPE && j < nb) {  // S of block j, over P, which the P V just issued reads first: they run in order
                ok = __all_sync(0xffffffffu, kv_in(2 * j));
                if (!ok) break;
                tc_fence_after();
                issue_s((2 * j) % L::kStages);
            }
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------- softmax --
        // A failed wait poisons the rest (ok = false); two warpgroups agree on it at the block's barrier, which every
        // warp reaches.
        const int wg = WGS == 1 ? 0 : warp >> 2, r = threadIdx.x & 127;
        const int row = q_start + r;
        const uint32_t lanes = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        const uint32_t tS = lanes + L::kTmS + kCols * wg, tO = lanes + L::kTmO + D / WGS * wg;
        const uint32_t tP = lanes + L::kTmP + (PIPE ? kCols / 2 : kCols) * wg;  // (d = 128: over this thread's S)
        const float sl2 = p.scale_log2;
        const uint64_t c2 = f2_pack(sl2, sl2);
        const ScoreRange mine = keys_of(p.mask, b, min(row, N - 1), prefix);
        [[maybe_unused]] float* bias_s = reinterpret_cast<float*>(smem + L::kTable);
        [[maybe_unused]] float slope2 = 0.f;
        if constexpr (BIAS == kBiasSlopes) {
            slope2 = p.slopes[h] * kLog2e;
            sh.ramp[0][r] = slope2 * r;
            sh.ramp[1][r] = -slope2 * r;
            named_bar_sync(1, kSoftmax);
        }
        if constexpr (BIAS == kBiasTable) {
            for (int i = threadIdx.x; i <= 2 * p.far; i += kSoftmax)
                bias_s[i] = kLog2e * table_bias(p.table, p.table_f32, p.buckets, p.num_buckets, p.H, h, i);
            named_bar_sync(1, kSoftmax);
        }
        constexpr bool SCALED = CAP || BIAS != kBiasNone;  // y in log2 units before the max is taken
        float m_used = -INFINITY;
        float l = 0.f, l_mma = 0.f;
        [[maybe_unused]] int most = kTanhPoly3;  // CAP: the farthest form of the tanh so far
        bool ok = true;
        for (int j = 0; j < nb; ++j) {
            if (ok) ok = __all_sync(0xffffffffu, mbar_wait(bar_s, j & 1, wd, kSiteSoftS));
            if (WGS == 1 && !ok) break;
            uint32_t s[kParts][32];
            const int kb0 = (jlo + j) * kBN, kbase = kb0 + kCols * wg;
            const bool masked = kb0 < clear_lo || kb0 + kBN > clear_hi;
            [[maybe_unused]] int how = kTanhExp;  // CAP: form of the tanh
            [[maybe_unused]] bool late = false;   // CAP: the cap is yet to come
            [[maybe_unused]] float base = 0.f;    // slopes: what the scores below lack, the same for the row
            float m_cand = -INFINITY;
            if (ok) {
                tc_fence_after();
#pragma unroll
                for (int g = 0; g < kParts; ++g) tmem_ld32(tS + 32 * g, s[g]);
#pragma unroll
                for (int g = 0; g < kParts; ++g) tmem_ld_wait(s[g]);
                if constexpr (PIPE) {
                    tc_fence_before();
                    mbar_arrive(bar_sf);  // S's columns may take the next block's scores now
                }
                if constexpr (CAP) {
                    float hi0 = -INFINITY, hi1 = -INFINITY, lo0 = INFINITY, lo1 = INFINITY;
#pragma unroll
                    for (int g = 0; g < kParts; ++g)
#pragma unroll
                        for (int c = 0; c < 32; c += 4) {
                            hi0 = fmax3(hi0, u2f(s[g][c]), u2f(s[g][c + 1]));
                            hi1 = fmax3(hi1, u2f(s[g][c + 2]), u2f(s[g][c + 3]));
                            lo0 = fmin3(lo0, u2f(s[g][c]), u2f(s[g][c + 1]));
                            lo1 = fmin3(lo1, u2f(s[g][c + 2]), u2f(s[g][c + 3]));
                        }
                    const float hi = fmaxf(hi0, hi1);
                    const float mx = fmaxf(hi, -fminf(lo0, lo1)) * p.cap.k;  // of the warp's rows: the tanh's form
                    how = !__any_sync(0xffffffffu, !(mx <= kTanhNear))  ? kTanhPoly3
                          : !__any_sync(0xffffffffu, !(mx <= kTanhMid)) ? kTanhPoly4
                                                                        : kTanhExp;
                    // (once one of a warp's blocks has needed a farther form, those behind it take it, too: warps that go
                    // to and fro between the forms wait for instructions, 292 -> 351 us where a third of the blocks
                    // passed a bound.  The last form is off by a part of the cap, whatever the score (fa_score.cuh): not
                    // where caps are in the thousands.)
                    if (how > most) most = how;
                    else if (most == kTanhPoly4 || CAP == kCapCommon) how = most;
                    if (BIAS == kBiasNone && !masked) {
                        late = true;
                        const uint64_t v = f2_pack(hi, hi);
                        m_cand = f2_unpack(how == kTanhPoly3   ? cap_score2<kTanhPoly3>(p.cap, v, 0)
                                           : how == kTanhPoly4 ? cap_score2<kTanhPoly4>(p.cap, v, 0)
                                                               : cap_score2<kFar>(p.cap, v, 0)).x;
                    } else if (how == kTanhPoly3) {
                        each_pair(s, [&](int, uint64_t v) { return cap_score2<kTanhPoly3>(p.cap, v, 0); });
                    } else if (how == kTanhPoly4) {
                        each_pair(s, [&](int, uint64_t v) { return cap_score2<kTanhPoly4>(p.cap, v, 0); });
                    } else {
                        each_pair(s, [&](int, uint64_t v) { return cap_score2<kFar>(p.cap, v, 0); });
                    }
                }
                if constexpr (BIAS == kBiasSlopes) {
                    const float d0 = static_cast<float>(kbase - row);  // j - i at column 0, exact below 2^24
                    const int side = far_side(q_start, kb0, kBM, 0);
                    if (side != 0) {
                        // all keys before (or behind) all queries: y - slope |i - j| with the sign in the slope
                        base = side * slope2 * d0;
                        const uint32_t ramp = smem_addr(sh.ramp[side < 0]);
#pragma unroll
                        for (int c = 0; c < kCols; c += 4) {
                            const ulonglong2 w = lds_2x64(ramp + 4 * c);
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                uint32_t &a = s[c >> 5][(c & 31) + 2 * e], &bb = s[c >> 5][(c & 31) + 2 * e + 1];
                                const uint64_t v = f2_pack(u2f(a), u2f(bb)), add = e ? w.y : w.x;
                                const float2 y = f2_unpack(CAP ? fadd2(v, add) : ffma2(v, c2, add));
                                a = f2u(y.x);
                                bb = f2u(y.y);
                            }
                        }
                    } else {
                        each_pair(s, [&](int c, uint64_t v) {
                            float2 y = f2_unpack(CAP ? v : fmul2(v, c2));
                            y.x = fmaf(-slope2, fabsf(d0 + c), y.x);
                            y.y = fmaf(-slope2, fabsf(d0 + c + 1), y.y);
                            return f2_pack(y.x, y.y);
                        });
                    }
                }
                if constexpr (BIAS == kBiasTable) {
                    const int side = far_side(q_start, kb0, kBM, p.far);
                    if (side != 0) {
                        const float bf = bias_s[side > 0 ? 2 * p.far : 0];
                        const uint64_t b2 = f2_pack(bf, bf);
                        each_pair(s, [&](int, uint64_t v) { return CAP ? fadd2(v, b2) : ffma2(v, c2, b2); });
                    } else {
                        const int i0 = row - kbase + p.far, top_i = 2 * p.far;
                        each_pair(s, [&](int c, uint64_t v) {
                            const uint64_t b2 = f2_pack(bias_s[max(0, min(top_i, i0 - c))], bias_s[max(0, min(top_i, i0 - c - 1))]);
                            return CAP ? fadd2(v, b2) : ffma2(v, c2, b2);
                        });
                    }
                }
                if (masked) {
                    const int from = mine.lo - kbase;
                    const uint32_t n = static_cast<uint32_t>(mine.hi - mine.lo);
#pragma unroll
                    for (int c = 0; c < kCols; ++c)
                        if (static_cast<uint32_t>(c - from) >= n) s[c >> 5][c & 31] = f2u(-INFINITY);
                }
                if (!late) {
                    float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
                    for (int g = 0; g < kParts; ++g)
#pragma unroll
                        for (int c = 0; c < 32; c += 4) {
                            mx0 = fmax3(mx0, u2f(s[g][c]), u2f(s[g][c + 1]));
                            mx1 = fmax3(mx1, u2f(s[g][c + 2]), u2f(s[g][c + 3]));
                        }
                    m_cand = fmaxf(mx0, mx1);
                    if constexpr (!SCALED) m_cand *= sl2;
                    if constexpr (BIAS == kBiasSlopes) m_cand += base;
                }
            }
            if constexpr (WGS == 2) {
                sh.top[j & 1][wg][r] = m_cand;
                if (named_bar_or(1, kSoftmax, !ok)) {
                    ok = false;
                    break;
                }
                m_cand = fmaxf(m_cand, sh.top[j & 1][wg ^ 1][r]);
            }
            const bool grow = m_cand > m_used + kRescaleThreshold;
            float alpha = 1.f;
            if (grow) {
                alpha = ex2(m_used - m_cand);  // 0 on the first block (m_used = -inf)
                m_used = m_cand;
            }
            l *= alpha;
            l_mma *= alpha;
            const float neg_m = (m_used == -INFINITY ? 0.f : -m_used) + base;
            // l_mma sums the bf16 weights that the P V product takes (it normalises O), l the
            // fp32 ones (it gives LSE)
            const uint64_t nm2 = f2_pack(neg_m, neg_m);
            uint64_t ls2 = 0;
            float lr0 = 0.f, lr1 = 0.f;
            constexpr int kPC = D == 128 || WGS == 2 ? 16 : 32;  // packed columns per tensor-memory store
            if (PIPE && j > 0) {
                // P's columns are free once the previous P V has read them
                ok = __all_sync(0xffffffffu, mbar_wait(bar_o, (j - 1) & 1, wd, kSiteSoftO));
                if (!ok && WGS == 1) break;
                tc_fence_after();
            }
            const auto weights = [&](auto&& exponent) {  // of a pair
#pragma unroll
                for (int hh = 0; hh < kCols / 2 / kPC; ++hh) {
                    uint32_t pk[kPC];
#pragma unroll
                    for (int i = 0; i < kPC; ++i) {
                        const int c = hh * 2 * kPC + 2 * i;
                        const float2 x = f2_unpack(exponent(f2_pack(u2f(s[c >> 5][c & 31]), u2f(s[c >> 5][(c & 31) + 1]))));
                        const float p0 = ex2(x.x), p1 = ex2(x.y);
                        pk[i] = pack_bf16(p0, p1);
                        ls2 = fadd2(ls2, f2_pack(p0, p1));
                        add_bf16x2_f32(pk[i], lr0, lr1);
                    }
                    if constexpr (kPC == 16) tmem_st16(tP + hh * 16, pk);
                    else tmem_st32(tP + hh * 32, pk);
                }
            };
            if (!ok) {
            } else if (CAP && late) {
                if (how == kTanhPoly3) weights([&](uint64_t v) { return cap_score2<kTanhPoly3>(p.cap, v, nm2); });
                else if (how == kTanhPoly4) weights([&](uint64_t v) { return cap_score2<kTanhPoly4>(p.cap, v, nm2); });
                else weights([&](uint64_t v) { return cap_score2<kFar>(p.cap, v, nm2); });
            } else {
                weights([&](uint64_t v) { return SCALED ? fadd2(v, nm2) : ffma2(v, c2, nm2); });
            }
            const float2 a2 = f2_unpack(ls2);
            l += a2.x + a2.y;
            l_mma += lr0 + lr1;
            if (ok && j > 0 && __any_sync(0xffffffffu, grow)) {
                // rescale this thread's part of O once the previous P V has landed
                ok = __all_sync(0xffffffffu, mbar_wait(bar_o, (j - 1) & 1, wd, kSiteSoftO));
                if (!ok && WGS == 1) break;
                tc_fence_after();
                if (ok) {
#pragma unroll
                    for (int c0 = 0; c0 < D / WGS; c0 += 32) {
                        uint32_t o[32];
                        tmem_ld32(tO + c0, o);
                        tmem_ld_wait(o);
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = f2u(u2f(o[i]) * alpha);
                        tmem_st32(tO + c0, o);
                    }
                }
            }
            if (ok) {
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(bar_p);
            }
        }
        // ----------------------------------------------------------- epilogue --
        // O / l_mma -> bf16, staged over Q (every S has read it), one TMA store
        if (ok) ok = __all_sync(0xffffffffu, mbar_wait(bar_o, (nb - 1) & 1, wd, kSiteEpi));
        if constexpr (WGS == 2) {
            sh.sum[0][wg][r] = l;
            sh.sum[1][wg][r] = l_mma;
            ok = !named_bar_or(1, kSoftmax, !ok);
            l += sh.sum[0][wg ^ 1][r];
            l_mma += sh.sum[1][wg ^ 1][r];
        }
        if (ok) {
            tc_fence_after();
            const float inv_l = l_mma > 0.f ? 1.f / l_mma : 0.f;
#pragma unroll
            for (int c0 = 0; c0 < D / WGS; c0 += 32) {
                uint32_t o[32];
                tmem_ld32(tO + c0, o);
                tmem_ld_wait(o);
                const int col = D / WGS * wg + c0;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int chunk = (col % 64) / 8 + q;
                    uint4 v;
                    v.x = pack_bf16(u2f(o[8 * q + 0]) * inv_l, u2f(o[8 * q + 1]) * inv_l);
                    v.y = pack_bf16(u2f(o[8 * q + 2]) * inv_l, u2f(o[8 * q + 3]) * inv_l);
                    v.z = pack_bf16(u2f(o[8 * q + 4]) * inv_l, u2f(o[8 * q + 5]) * inv_l);
                    v.w = pack_bf16(u2f(o[8 * q + 6]) * inv_l, u2f(o[8 * q + 7]) * inv_l);
                    *reinterpret_cast<uint4*>(smem + (col / 64) * L::kBox + r * 128 + ((chunk ^ (r & 7)) << 4)) = v;
                }
            }
            fence_async_shared();
            if (wg == 0 && row < N) p.LSE[static_cast<int64_t>(bh) * N + row] = (m_used + __log2f(l)) * kLn2;
        }
        // (every warp reaches this barrier, also after a failed wait, and all agree)
        if (!named_bar_or(1, kSoftmax, !ok) && threadIdx.x == 0) {
            for (int x = 0; x < L::kBoxes; ++x) tma_store_3d(&tmO, sbase + x * L::kBox, x * 64, q_start, bh);
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
        tmem_dealloc(tmem, L::kTmCols);
    }
}

template <int D, int CAP, int BIAS, int WGS>
cudaError_t launch_w(const ScoreArgs& a, cudaStream_t stream) {
    using L = ScoreFwdLayout<D>;
    CUtensorMap tq, tk, tv, to;
    const auto BF = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const int BH = a.B * a.H, BHkv = a.B * a.H_kv;
    if (!make_tile_map(&tq, a.Q, BF, 2, D, a.N, BH, 64, kBM) || !make_tile_map(&tk, a.K, BF, 2, D, a.N, BHkv, 64, kBN) ||
        !make_tile_map(&tv, a.V, BF, 2, D, a.N, BHkv, 64, kBN) || !make_tile_map(&to, a.O, BF, 2, D, a.N, BH, 64, kBM))
        return cudaErrorInvalidValue;
    constexpr auto kern = &fa_score_fwd_kernel<D, CAP, BIAS, WGS>;
    // (the limit is set for the largest table, so that it is set once)
    constexpr int kTableMax = BIAS == kBiasTable ? (2 * kScoreMaxFar + 1) * 4 : 0;
    cudaError_t e = set_max_dyn_smem_once<kern>(L::kDynSmem + kTableMax);
    if (e != cudaSuccess) return e;
    const int bytes = L::kDynSmem + (BIAS == kBiasTable ? (2 * a.mod.far + 1) * 4 : 0);
    ScoreFwdParams p;
    p.LSE = a.LSE;
    p.H = a.H;
    p.G = a.H / a.H_kv;
    p.n_q = (a.N + kBM - 1) / kBM;
    p.mask.spans = a.mod.docs ? reinterpret_cast<const int2*>(a.workspace) : nullptr;
    p.order = a.mod.docs ? reinterpret_cast<const int*>(a.workspace + score_spans_bytes(a.B, a.N)) : nullptr;
    p.mask.prefix = a.mod.prefix;
    p.mask.N = a.N;
    p.mask.window = a.mod.window;
    p.mask.causal = a.causal;
    p.scale_log2 = a.tau * kLog2e;
    if (CAP) p.cap = CapScale(a.tau, a.mod.softcap);
    p.slopes = a.mod.slopes;
    p.table = a.mod.table;
    p.buckets = a.mod.buckets;
    p.table_f32 = a.mod.table_f32;
    p.num_buckets = a.mod.num_buckets;
    p.far = a.mod.far;
    p.err = a.err;
    p.wait_limit_ns = a.wait_limit_ns;
    if (a.ev_start) cudaEventRecord(a.ev_start, stream);
    e = launch_dependent(kern, dim3(static_cast<unsigned>(BH), static_cast<unsigned>(p.n_q)), dim3(threads_for(WGS)),
                         static_cast<size_t>(bytes), stream, tq, tk, tv, to, p);
    if (e == cudaSuccess && a.ev_stop) e = cudaEventRecord(a.ev_stop, stream);
    return e;
}

// Two softmax warpgroups where there are at most two tiles for each SM, and the chain of steps of the longest sets the
// time (16 heads, d = 64: 901 tokens with slopes 15.0 us by one and 12.6 by two, 2000 capped 41.3 and 30.9, 4096
// capped 84 and 108).
template <int D, int CAP, int BIAS>
cudaError_t launch_t(const ScoreArgs& a, cudaStream_t stream) {
    const long long ctas = static_cast<long long>(a.B) * a.H * ((a.N + kBM - 1) / kBM);
    if constexpr (CAP == kCapLarge) return launch_w<D, CAP, BIAS, 1>(a, stream);  // (rare: one form)
    else return ctas <= 2 * kSms ? launch_w<D, CAP, BIAS, 2>(a, stream) : launch_w<D, CAP, BIAS, 1>(a, stream);
}

template <int D, int CAP>
cudaError_t launch_c(const ScoreArgs& a, cudaStream_t stream) {
    return a.mod.slopes  ? launch_t<D, CAP, kBiasSlopes>(a, stream)
           : a.mod.table ? launch_t<D, CAP, kBiasTable>(a, stream)
                         : launch_t<D, CAP, kBiasNone>(a, stream);
}

template <int D>
cudaError_t launch_d(const ScoreArgs& a, cudaStream_t stream) {
    switch (cap_of(a.mod.softcap)) {
        case kCapNone: return launch_c<D, kCapNone>(a, stream);
        case kCapCommon: return launch_c<D, kCapCommon>(a, stream);
        default: return launch_c<D, kCapLarge>(a, stream);
    }
}

}  // namespace

size_t score_fwd_workspace(int B, int N, bool docs) {
    return docs ? score_spans_bytes(B, N) + static_cast<size_t>(B) * ((static_cast<size_t>(N) + kBM - 1) / kBM) * sizeof(int) : 0;
}

cudaError_t launch_score_fwd(const ScoreArgs& a, cudaStream_t stream) {
    if (a.mod.docs) {
        ScoreOrder order;
        order.queries = reinterpret_cast<int*>(a.workspace + score_spans_bytes(a.B, a.N));
        const cudaError_t e = launch_score_spans(a, a.workspace, order, stream);
        if (e != cudaSuccess) return e;
    }
    return a.d == 64 ? launch_d<64>(a, stream) : launch_d<128>(a, stream);
}

}  // namespace fa
