// Row sums of the backward of attention with capped, biased or masked scores, for sm_103a:
// D_i = sum_j P_ij dP_ij, and a zeroed fp32 dQ accumulator and tile counter.
//
// Mathematics: D_i = dO_i . O_i as well, which costs nothing but reads O as the forward rounded it, from
// weights that it rounded too: off by 2^-8 of |dO| |O|, while dY = P (dP - D) is a small
// difference wherever a row's weight lies on few keys.  Capped and biased scores are often of that
// kind: dQ and dK were off by 3.1e-3 (16 heads of 8192 tokens, scores of deviation 4, capped
// at 50; their other two roundings alone give 2.3e-3), and the bias's gradient of a far bucket, which
// sums D's error over almost all of a row's weight, by 1e-2 at 4096 tokens.  Summed from fp32 weights
// the error is fp32's.
//
// Design: one CTA per pair of 128-row query tiles of a head.  Warp 16 streams K_j and V_j by TMA,
// warp 17 (d = 128: 17 for one tile, 18 for the other) issues S_t = Q_t K_j^T and dP_t = dO_t V_j^T (tcgen05; all 512
// tensor-memory columns), and four warpgroups, two to a tile with half of its columns each, add
// p * dP, a row per thread: no maximum, no second product, LSE being known.  One tile's
// elementwise work runs beside the other's products: 16 heads of 8192 tokens, window 4096 and 8 key heads at d = 128, capped, 185 us (tensor
// pipe 51%); 96 heads of 1024 tokens with slopes, d = 64, 33.
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "fa_score.cuh"

namespace fa {
namespace {

constexpr int kBM = 128, kBN = 128;
constexpr int kProducerWarp = 16, kMmaWarp = 17;
constexpr float kLog2e = 1.44269504088896341f;

// Warps that issue products: at d = 128 one for each tile, since one's issue (16 in each block and tile, at 110 cycles
// each beside busy warps) bounds the kernel (16 heads of 16384 tokens, window 4096: 389 us by one, 325 by two); at
// d = 64, where it does not, the second costs more (129 us, 148).
constexpr int mma_warps(int D) { return D == 128 ? 2 : 1; }
constexpr int threads_for(int D) { return 32 * (kMmaWarp + mma_warps(D)); }

template <int D>
struct RowsLayout {
    static constexpr int kTile = kBM * D * 2;
    static constexpr int kBox = 128 * 128;
    static constexpr int kBoxes = D / 64;
    static constexpr int kStages = D == 64 ? 6 : 3;
    // tile t: Q at 2 t kTile, dO behind it
    static constexpr int kRing = 4 * kTile;
    static constexpr int kDynSmem = kRing + kStages * kTile + 1024;  // + alignment slack
};

struct RowsParams {
    const float* LSE;
    float* Dvec;
    float* dQacc;
    unsigned* next;  // zeroed, too
    int H, G, n_pairs;
    const int* order;  // [B][n_pairs], or null: from the last
    ScoreMask mask;
    float scale_log2;
    CapScale cap;
    const float* slopes;
    const float* bias2;  // [H][2 far + 1], log2 units
    int far;
    unsigned int* err;
    unsigned long long wait_limit_ns;
};

struct RowsShared {
    uint64_t q_full;
    uint64_t kv_full[6];
    uint64_t kv_empty[6];
    uint64_t full[2];   // S_t and dP_t are in
    uint64_t free_[2];  // both have been read
    float half[2][128];  // the sums of a tile's second columns
    uint32_t tmem_base;
    int abort_flag;
};

enum : uint32_t { kSiteProd = 91, kSiteMmaQ = 92, kSiteMmaKV = 93, kSiteMmaFree = 94, kSiteSum = 95 };

__device__ __forceinline__ float u2f(uint32_t x) { return __uint_as_float(x); }

constexpr uint32_t kDescHi = sw128_desc_hi(1024);

template <int D, int CAP, int BIAS>
__global__ void __launch_bounds__(threads_for(D), 1)
fa_score_rows_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmdO, const RowsParams p) {
    using L = RowsLayout<D>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ RowsShared sh;
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t sbase = (raw + 1023u) & ~1023u;
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int N = p.mask.N;
    const int bh = static_cast<int>(blockIdx.x);
    const int b = bh / p.H, h = bh - b * p.H;
    const int bkv = b * (p.H / p.G) + h / p.G;

    const uint32_t bar_q = smem_addr(&sh.q_full);
    const uint32_t bar_kvf = smem_addr(&sh.kv_full[0]);
    const uint32_t bar_kve = smem_addr(&sh.kv_empty[0]);
    const uint32_t bar_full = smem_addr(&sh.full[0]);
    const uint32_t bar_free = smem_addr(&sh.free_[0]);
    if (threadIdx.x == 0) {
        sh.abort_flag = 0;
        mbar_init(bar_q, 1);
        for (int s = 0; s < L::kStages; ++s) {
            mbar_init(bar_kvf + 8 * s, 1);
            mbar_init(bar_kve + 8 * s, mma_warps(D));
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(bar_full + 8 * t, 1);
            mbar_init(bar_free + 8 * t, 256);
        }
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
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    griddep_launch_dependents();
    griddep_wait();
    if (threadIdx.x == 0 && blockIdx.x == 0 && blockIdx.y == 0) *p.next = 0;
    const uint32_t tmem = sh.tmem_base;
    const Watchdog wd{p.err, &sh.abort_flag, p.wait_limit_ns};
    const int rank = static_cast<int>(blockIdx.y);
    const int q0 = (p.order ? p.order[static_cast<long long>(b) * p.n_pairs + rank] : p.n_pairs - 1 - rank) * 2 * kBM;
    const bool two = q0 + kBM < N;

    // tile t takes key blocks [lo[t], hi[t]); the two ranges overlap or touch (a tile's own block is
    // in its range or beside it), so the loaders walk [jlo, jhi)
    const int prefix = prefix_of(p.mask, b);
    int lo[2], hi[2], clear_lo[2], clear_hi[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        lo[t] = hi[t] = clear_lo[t] = clear_hi[t] = 0;
        if (t == 1 && !two) continue;
        const int q = q0 + t * kBM;
        const ScoreRange top = keys_of(p.mask, b, q, prefix);
        const ScoreRange bottom = keys_of(p.mask, b, min(q + kBM, N) - 1, prefix);
        const ScoreRange blocks = blocks_of(top.lo, bottom.hi, kBN);
        lo[t] = blocks.lo;
        hi[t] = blocks.hi;
        clear_lo[t] = bottom.lo;
        clear_hi[t] = top.hi;
    }
    const int jlo = lo[0], jhi = max(hi[0], hi[1]);

    if (warp == kProducerWarp) {
        // ------------------------------------------------------------ producer --
        if (lane == 0) {
            mbar_arrive_expect_tx(bar_q, (two ? 4 : 2) * L::kTile);
            for (int t = 0; t < (two ? 2 : 1); ++t)
                for (int x = 0; x < L::kBoxes; ++x) {
                    const uint32_t dst = sbase + 2 * t * L::kTile + x * L::kBox;
                    tma_load_3d(dst, &tmQ, bar_q, x * 64, q0 + t * kBM, bh);
                    tma_load_3d(dst + L::kTile, &tmdO, bar_q, x * 64, q0 + t * kBM, bh);
                }
            for (int ld = 0; ld < 2 * (jhi - jlo); ++ld) {
                const int slot = ld % L::kStages;
                if (ld >= L::kStages && !mbar_wait(bar_kve + 8 * slot, ((ld / L::kStages) - 1) & 1, wd, kSiteProd)) break;
                mbar_arrive_expect_tx(bar_kvf + 8 * slot, L::kTile);
                for (int x = 0; x < L::kBoxes; ++x)
                    tma_load_3d(sbase + L::kRing + slot * L::kTile + x * L::kBox, (ld & 1) ? &tmV : &tmK, bar_kvf + 8 * slot,
                                x * 64, (jlo + (ld >> 1)) * kBN, bkv);
            }
        }
        __syncwarp();
    } else if (warp >= kMmaWarp) {
        // ----------------------------------------------------------------- MMA --
        constexpr uint32_t id = idesc_bf16(128, 128, false, false);
        constexpr uint32_t kStep = L::kTile >> 4;
        const uint32_t a0 = sw128_desc_lo(sbase, 16), ring0 = sw128_desc_lo(sbase + L::kRing, 16);
        const auto product = [&](uint32_t d, uint32_t a, uint32_t bb) {  // both K-major
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                const uint32_t off = ((k / 4) * (128 * 128) + (k % 4) * 32) >> 4;
                if (k == 0) mma_ss_warp<0>(d, a + off, bb + off, kDescHi, id);
                else mma_ss_warp<1>(d, a + off, bb + off, kDescHi, id);
            }
        };
        const auto kv_in = [&](int ld) { return mbar_wait(bar_kvf + 8 * (ld % L::kStages), (ld / L::kStages) & 1, wd, kSiteMmaKV); };
        bool ok = __all_sync(0xffffffffu, mbar_wait(bar_q, 0, wd, kSiteMmaQ));
        if constexpr (mma_warps(D) == 2) {
            const int t = warp - kMmaWarp;
            const int j0 = t ? lo[1] : lo[0], j1 = t ? hi[1] : hi[0];
            for (int j = jlo; ok && j < jhi; ++j) {
                const int lk = 2 * (j - jlo), lv = lk + 1, sk = lk % L::kStages, sv = lv % L::kStages;
                ok = __all_sync(0xffffffffu, kv_in(lk));
                if (!ok) break;
                if (j < j0 || j >= j1) {  // not of this tile
                    ok = __all_sync(0xffffffffu, kv_in(lv));
                    if (ok && lane == 0) {
                        mbar_arrive(bar_kve + 8 * sk);
                        mbar_arrive(bar_kve + 8 * sv);
                    }
                    continue;
                }
                if (j > j0) ok = __all_sync(0xffffffffu, mbar_wait(bar_free + 8 * t, (j - j0 - 1) & 1, wd, kSiteMmaFree));
                if (!ok) break;
                tc_fence_after();
                product(tmem + 256 * t, a0 + 2 * t * kStep, ring0 + sk * kStep);                 // S
                mma_commit_warp(bar_kve + 8 * sk);  // (its slot is the next V's, wanted a tile's products later)
                ok = __all_sync(0xffffffffu, kv_in(lv));
                if (!ok) break;
                tc_fence_after();
                product(tmem + 256 * t + 128, a0 + (2 * t + 1) * kStep, ring0 + sv * kStep);     // dP
                mma_commit_warp(bar_full + 8 * t);
                mma_commit_warp(bar_kve + 8 * sv);
            }
        } else {
            for (int j = jlo; ok && j < jhi; ++j) {
                const int lk = 2 * (j - jlo), lv = lk + 1, sk = lk % L::kStages, sv = lv % L::kStages;
                ok = __all_sync(0xffffffffu, kv_in(lk) && kv_in(lv));
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    if (!ok || j < lo[t] || j >= hi[t]) continue;
                    if (j > lo[t]) ok = __all_sync(0xffffffffu, mbar_wait(bar_free + 8 * t, (j - lo[t] - 1) & 1, wd, kSiteMmaFree));
                    if (!ok) continue;
                    tc_fence_after();
                    product(tmem + 256 * t, a0 + 2 * t * kStep, ring0 + sk * kStep);                 // S
                    // (K goes back as soon as both tiles' S have read it: its slot is the next V's, wanted a tile's products later)
                    if (t == 1 || j >= hi[1] || j < lo[1]) mma_commit_warp(bar_kve + 8 * sk);
                    product(tmem + 256 * t + 128, a0 + (2 * t + 1) * kStep, ring0 + sv * kStep);     // dP
                    mma_commit_warp(bar_full + 8 * t);
                }
                if (!ok) break;
                mma_commit_warp(bar_kve + 8 * sv);
            }
        }
        __syncwarp();
    } else {
        // ---------------------------------------------------------------- sums --
        const int t = warp >> 3, side_half = (warp >> 2) & 1;
        const int r = threadIdx.x & 127;
        const int q_start = q0 + t * kBM, row = q_start + r;
        const int64_t at = static_cast<int64_t>(bh) * N + row;
        const uint32_t tS = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + 256 * t + 64 * side_half;
        // zero the accumulator's rows (256 threads per tile, a row's D floats in a row)
        {
            float4* z = reinterpret_cast<float4*>(p.dQacc + (static_cast<int64_t>(bh) * N + q_start) * D);
            const int n = max(0, min(kBM, N - q_start)) * (D / 4);
            for (int i = side_half * 128 + r; i < n; i += 256) z[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        const ScoreRange mine = keys_of(p.mask, b, min(row, N - 1), prefix);
        // (a row that sees nothing: LSE = -inf, every weight masked to 0)
        const float nl = row < N ? -p.LSE[at] * kLog2e : -INFINITY;
        const uint64_t c2 = f2_pack(p.scale_log2, p.scale_log2), nl2 = f2_pack(nl, nl);
        [[maybe_unused]] float slope2 = 0.f;
        [[maybe_unused]] const float* bias2 = nullptr;
        if constexpr (BIAS == kBiasSlopes) slope2 = p.slopes[h] * kLog2e;
        if constexpr (BIAS == kBiasTable) bias2 = p.bias2 + static_cast<long long>(h) * (2 * p.far + 1);
        uint64_t sum[2] = {0, 0};
        bool ok = true;
        const int nb = t ? hi[1] - lo[1] : hi[0] - lo[0], jt = t ? lo[1] : lo[0];
        const int c_lo = t ? clear_lo[1] : clear_lo[0], c_hi = t ? clear_hi[1] : clear_hi[0];
        for (int jj = 0; jj < nb; ++jj) {
            if (!__all_sync(0xffffffffu, mbar_wait(bar_full + 8 * t, jj & 1, wd, kSiteSum))) {
                ok = false;
                break;
            }
            tc_fence_after();
            const int kbase = (jt + jj) * kBN;
            const int side = far_side(q_start, kbase, kBM, BIAS == kBiasTable ? p.far : 0);
            const bool general = kbase < c_lo || kbase + kBN > c_hi || (BIAS != kBiasNone && side == 0);
            [[maybe_unused]] const uint64_t sl = f2_pack(side * slope2, side * slope2);  // (of j - i)
            [[maybe_unused]] uint64_t add0 = nl2;
            if constexpr (BIAS == kBiasTable) {
                if (side != 0) {
                    const float v = bias2[side > 0 ? 2 * p.far : 0];
                    add0 = fadd2(nl2, f2_pack(v, v));
                }
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                uint32_t s[32], dp[32];
                tmem_ld32(tS + 32 * c, s);
                tmem_ld32(tS + 128 + 32 * c, dp);
                tmem_ld_wait(s);
                tmem_ld_wait(dp);
                if (c == 1) {
                    tc_fence_before();
                    mbar_arrive(bar_free + 8 * t);
                }
                const int col0 = kbase + 64 * side_half + 32 * c;  // the chunk's first key
                const int from = mine.lo - col0;
                const uint32_t n = static_cast<uint32_t>(mine.hi - mine.lo);
                // a pair of keys, s as it comes.  GENERAL: any mask, any bias; else all are visible and the
                // bias is the same or, of slopes, on one side.
                [[maybe_unused]] uint64_t dist = f2_pack(static_cast<float>(col0 - row), static_cast<float>(col0 - row + 1));
                const auto one = [&](auto how, auto general, int i) {
                    constexpr bool GENERAL = decltype(general)::value;
                    uint64_t add = add0;
                    if constexpr (BIAS == kBiasSlopes) {
                        if constexpr (GENERAL) {
                            const float2 y = f2_unpack(dist);
                            add = f2_pack(fmaf(-slope2, fabsf(y.x), nl), fmaf(-slope2, fabsf(y.y), nl));
                        } else {
                            add = ffma2(dist, sl, add0);
                        }
                        dist = fadd2(dist, f2_pack(2.f, 2.f));
                    }
                    if constexpr (BIAS == kBiasTable && GENERAL) {
                        const int x = row - col0 - 2 * i + p.far, top = 2 * p.far;
                        add = fadd2(nl2, f2_pack(bias2[max(0, min(top, x))], bias2[max(0, min(top, x - 1))]));
                    }
                    const uint64_t v = f2_pack(u2f(s[2 * i]), u2f(s[2 * i + 1]));
                    float2 x;
                    if constexpr (CAP) x = f2_unpack(cap_score2<decltype(how)::value>(p.cap, v, add));
                    else x = f2_unpack(ffma2(v, c2, add));
                    float p0 = ex2(x.x), p1 = ex2(x.y);
                    if constexpr (GENERAL) {
                        if (static_cast<uint32_t>(2 * i - from) >= n) p0 = 0.f;
                        if (static_cast<uint32_t>(2 * i + 1 - from) >= n) p1 = 0.f;
                    }
                    sum[i & 1] = ffma2(f2_pack(p0, p1), f2_pack(u2f(dp[2 * i]), u2f(dp[2 * i + 1])), sum[i & 1]);
                };
                const auto all = [&](auto how, auto general_) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) one(how, general_, i);
                };
                using Poly4 = std::integral_constant<int, kTanhPoly4>;
                using Exp = std::integral_constant<int, far_form(CAP)>;
                if constexpr (CAP) {
                    float mx0 = 0.f, mx1 = 0.f;
#pragma unroll
                    for (int i = 0; i < 32; i += 4) {
                        mx0 = fmax3(mx0, fabsf(u2f(s[i])), fabsf(u2f(s[i + 1])));
                        mx1 = fmax3(mx1, fabsf(u2f(s[i + 2])), fabsf(u2f(s[i + 3])));
                    }
                    // (the few tiles at the edges: two forms)
                    const float mx = fmaxf(mx0, mx1) * p.cap.k;
                    const bool near = !__any_sync(0xffffffffu, !(mx <= kTanhNear)), mid = !__any_sync(0xffffffffu, !(mx <= kTanhMid));
                    if (general && mid) all(Poly4{}, std::true_type{});
                    else if (general) all(Exp{}, std::true_type{});
                    else if (near) all(std::integral_constant<int, kTanhPoly3>{}, std::false_type{});
                    else if (mid) all(Poly4{}, std::false_type{});
                    else all(Exp{}, std::false_type{});
                } else if (general) {
                    all(Exp{}, std::true_type{});
                } else {
                    all(Exp{}, std::false_type{});
                }
            }
        }
        const float2 a = f2_unpack(fadd2(sum[0], sum[1]));
        if (side_half == 1) sh.half[t][r] = a.x + a.y;
        named_bar_sync(1 + t, 256);
        if (side_half == 0 && ok && row < N) p.Dvec[at] = a.x + a.y + sh.half[t][r];
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

template <int D, int CAP, int BIAS>
cudaError_t launch_t(const ScoreArgs& a, float* dvec, float* acc, unsigned* next, const void* spans, const int* order,
                     const float* bias2, cudaStream_t stream) {
    using L = RowsLayout<D>;
    CUtensorMap tq, tk, tv, tdo;
    const auto BF = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const int BH = a.B * a.H, BHkv = a.B * a.H_kv;
    if (!make_tile_map(&tq, a.Q, BF, 2, D, a.N, BH, 64, kBM) || !make_tile_map(&tk, a.K, BF, 2, D, a.N, BHkv, 64, kBN) ||
        !make_tile_map(&tv, a.V, BF, 2, D, a.N, BHkv, 64, kBN) || !make_tile_map(&tdo, a.dO, BF, 2, D, a.N, BH, 64, kBM))
        return cudaErrorInvalidValue;
    constexpr auto kern = &fa_score_rows_kernel<D, CAP, BIAS>;
    cudaError_t e = set_max_dyn_smem_once<kern>(L::kDynSmem);
    if (e != cudaSuccess) return e;
    RowsParams p;
    p.LSE = a.LSE;
    p.Dvec = dvec;
    p.dQacc = acc;
    p.next = next;
    p.H = a.H;
    p.G = a.H / a.H_kv;
    p.n_pairs = (a.N + 2 * kBM - 1) / (2 * kBM);
    p.mask.spans = static_cast<const int2*>(spans);
    p.order = order;
    p.mask.prefix = a.mod.prefix;
    p.mask.N = a.N;
    p.mask.window = a.mod.window;
    p.mask.causal = a.causal;
    p.scale_log2 = a.tau * kLog2e;
    if (CAP) p.cap = CapScale(a.tau, a.mod.softcap);
    p.slopes = a.mod.slopes;
    p.bias2 = bias2;
    p.far = a.mod.far;
    p.err = a.err;
    p.wait_limit_ns = a.wait_limit_ns;
    return launch_dependent(kern, dim3(static_cast<unsigned>(BH), static_cast<unsigned>(p.n_pairs)), dim3(threads_for(D)), L::kDynSmem,
                            stream, tq, tk, tv, tdo, p);
}

template <int D, int CAP>
cudaError_t launch_c(const ScoreArgs& a, float* dvec, float* acc, unsigned* next, const void* spans, const int* order,
                     const float* bias2, cudaStream_t stream) {
    return a.mod.slopes  ? launch_t<D, CAP, kBiasSlopes>(a, dvec, acc, next, spans, order, bias2, stream)
           : a.mod.table ? launch_t<D, CAP, kBiasTable>(a, dvec, acc, next, spans, order, bias2, stream)
                         : launch_t<D, CAP, kBiasNone>(a, dvec, acc, next, spans, order, bias2, stream);
}

template <int D>
cudaError_t launch_d(const ScoreArgs& a, float* dvec, float* acc, unsigned* next, const void* spans, const int* order,
                     const float* bias2, cudaStream_t stream) {
    switch (cap_of(a.mod.softcap)) {
        case kCapNone: return launch_c<D, kCapNone>(a, dvec, acc, next, spans, order, bias2, stream);
        case kCapCommon: return launch_c<D, kCapCommon>(a, dvec, acc, next, spans, order, bias2, stream);
        default: return launch_c<D, kCapLarge>(a, dvec, acc, next, spans, order, bias2, stream);
    }
}

}  // namespace

cudaError_t launch_score_rows(const ScoreArgs& a, float* dvec, float* acc, unsigned* next, const void* spans, const int* order,
                              const float* bias2, cudaStream_t stream) {
    return a.d == 64 ? launch_d<64>(a, dvec, acc, next, spans, order, bias2, stream)
                     : launch_d<128>(a, dvec, acc, next, spans, order, bias2, stream);
}

}  // namespace fa
