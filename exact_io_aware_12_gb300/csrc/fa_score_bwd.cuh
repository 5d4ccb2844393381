// Parts of the backward of attention with capped, biased or masked scores that its two main kernels
// share (fa_score_bwd.cu: d = 128, fa_score_bwd64.cu: d = 64): a thread's elementwise work on 32 scores of
// its key row, the products' forms, and the workspace's layout.
#pragma once

#include <cuda_bf16.h>

#include <type_traits>

#include "fa_score.cuh"

namespace fa {

struct ScoreBwdParams {
    const float* LSE;
    const float* Dvec;
    int H, H_kv, BHkv, G, n_kv, head_group;
    const int* order;  // [B][n_kv], or null: as they come
    ScoreMask mask;
    float scale_log2, tau;
    float x_scale, cap_log2;
    const float* slopes;
    const float* bias2;  // [H][2 far + 1], log2 units
    int far;
    float* near_part;    // [B H][n_kv][near_n][kNearFloats], or null
    float* far_part;     // [B H][n_kv][4 NWG][kFarFloats]
    int near_lo, near_n;  // near tile pairs: query tile - key tile from near_lo on
    unsigned* next;  // d = 64: tiles taken, behind the first of every CTA
    unsigned int* err;
    unsigned long long wait_limit_ns;
};

namespace {

constexpr int kBQ = 128, kBK = 128;
constexpr float kLog2e = 1.44269504088896341f;
constexpr float kLiftP = 15.f, kUnliftP = 0x1p-15f;

// The table gradient's partial sums, in the workspace.
constexpr int kNearFloats = 1024;  // of a near tile pair: 16 blocks of 64
constexpr int kFarFloats = 2;      // of a warp: the sum over far keys behind the query, and before it

__device__ __forceinline__ float u2f(uint32_t x) { return __uint_as_float(x); }

constexpr uint32_t kDescHi = sw128_desc_hi(1024);
constexpr uint32_t kLboMN = 128 * 128;

// D = A B^T, both K-major tiles of 128 rows x Dk.
template <int Dk>
__device__ __forceinline__ void mma_rows_rows(uint32_t tmem_d, uint32_t a_lo, uint32_t b_lo) {
    constexpr uint32_t id = idesc_bf16(128, 128, false, false);
#pragma unroll
    for (int k = 0; k < Dk / 16; ++k) {
        const uint32_t off = ((k / 4) * (128 * 128) + (k % 4) * 32) >> 4;
        if (k == 0) mma_ss_warp<0>(tmem_d, a_lo + off, b_lo + off, kDescHi, id);
        else mma_ss_warp<1>(tmem_d, a_lo + off, b_lo + off, kDescHi, id);
    }
}
// D (+)= A_tmem[128 x 128] B, B an MN-major tile; each warpgroup's QC columns of A lie packed over
// the first half of its QC fp32 columns.
template <int Dn, int QC>
__device__ __forceinline__ void mma_tmem_a(uint32_t tmem_d, uint32_t tmem_a, uint32_t b_lo, bool accumulate) {
    constexpr uint32_t id = idesc_bf16(128, Dn, false, true);
    if (accumulate) mma_ts_warp<1>(tmem_d, tmem_a, b_lo, kDescHi, id);
    else mma_ts_warp<0>(tmem_d, tmem_a, b_lo, kDescHi, id);
#pragma unroll
    for (int k = 1; k < 128 / 16; ++k)
        mma_ts_warp<1>(tmem_d, tmem_a + (16 * k / QC) * QC + (16 * k % QC) / 2, b_lo + ((k * 2048) >> 4), kDescHi, id);
}
// D (+)= A B, A a K-major tile [128 x 128], B MN-major.
template <int Dn>
__device__ __forceinline__ void mma_rows_mn(uint32_t tmem_d, uint32_t a_lo, uint32_t b_lo, bool accumulate) {
    constexpr uint32_t id = idesc_bf16(128, Dn, false, true);
    if (accumulate) mma_ss_warp<1>(tmem_d, a_lo, b_lo, kDescHi, id);
    else mma_ss_warp<0>(tmem_d, a_lo, b_lo, kDescHi, id);
#pragma unroll
    for (int k = 1; k < 128 / 16; ++k)
        mma_ss_warp<1>(tmem_d, a_lo + (((k / 4) * (128 * 128) + (k % 4) * 32) >> 4), b_lo + ((k * 2048) >> 4), kDescHi, id);
}
// D = A B, both MN-major.
template <int Dn>
__device__ __forceinline__ void mma_mn_mn(uint32_t tmem_d, uint32_t a_lo, uint32_t b_lo) {
    constexpr uint32_t id = idesc_bf16(128, Dn, true, true);
    mma_ss_warp<0>(tmem_d, a_lo, b_lo, kDescHi, id);
#pragma unroll
    for (int k = 1; k < 128 / 16; ++k) mma_ss_warp<1>(tmem_d, a_lo + ((k * 2048) >> 4), b_lo + ((k * 2048) >> 4), kDescHi, id);
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// Elementwise warpgroups: 32 query columns of a step each.  (Two at d = 64: 16 heads of 8192 tokens, window 4096, 483 us
// for 418.)
constexpr int kNWG = 4;
constexpr int kQC = 128 / kNWG;
constexpr int kThreads = 32 * (4 * kNWG + 3);

// P (1 - tanh^2) waits for dP as fp32, or as fp16 (off by 2^-11 of it down to 2^-29, being lifted by 2^15) where a cap and
// a bias leave no registers: 16 of 96 a thread.  (Cut to fp16's largest, a P of 2: beside scores of 2^21, which fp32 holds to
// 2^-3, P comes out above 1, and infinite it made dQ and dK NaN.)  (fp32 saves the conversions: 16 heads of 8192 tokens, window 4096, d = 128
// 636 -> 628 us, slopes at d = 64 448 -> 427.)
constexpr int keep_regs(int cap, int bias) { return cap != kCapNone && bias != kBiasNone ? 16 : 32; }

// What a thread knows of a step: its key, the side of the pair of tiles, its bias there.
struct BwdRow {
    int kg;        // the key
    int lo;        // the queries that see it: [lo, lo + seen)
    uint32_t seen;
    bool general;  // any mask, any bias; else all pairs are visible and the bias is the same or, of slopes, on one side
    int side;      // far_side of the tiles
    float slope2;
    const float* bias2;
    uint64_t far_bias;
};

// Of one row's scores with queries [q0, q0 + 32): P as bf16 pairs (pk), and P (1 - tanh^2), what dP is to
// be multiplied by, as fp32 or, where keep_regs gives half the registers, as fp16 pairs (keep).  With a cap and a table, whose gradient takes P itself, P as fp16 pairs, too
// (pw).  nl4: the queries' 15 - LSE log2(e).
template <int CAP, int BIAS>
__device__ __forceinline__ void bwd_weights(const ScoreBwdParams& p, const BwdRow& r, const uint32_t (&sv)[32], const ulonglong2* nl4,
                                            int q0, uint32_t (&pk)[16], uint32_t (&keep)[keep_regs(CAP, BIAS)],
                                            [[maybe_unused]] uint32_t (&pw)[16]) {
    constexpr uint32_t FULL = 0xffffffffu;
    const uint64_t c2 = f2_pack(p.scale_log2, p.scale_log2);
    [[maybe_unused]] const uint64_t k2 = f2_pack(p.x_scale, p.x_scale), cap2 = f2_pack(p.cap_log2, p.cap_log2);
    [[maybe_unused]] const uint64_t sl = f2_pack(-r.side * r.slope2, -r.side * r.slope2);  // (of i - j)
    const int from = r.lo - q0;
    const float d0 = static_cast<float>(q0 - r.kg);  // i - j at the first query
    [[maybe_unused]] uint64_t dist = f2_pack(d0, d0 + 1.f);
    const auto weights = [&](auto how, auto general_, int i) {  // of a pair of queries
        constexpr bool GENERAL = decltype(general_)::value;
        const int q = 2 * i;
        const ulonglong2 nl = nl4[i >> 1];
        uint64_t add = (i & 1) ? nl.y : nl.x;
        if constexpr (BIAS == kBiasSlopes) {
            if constexpr (GENERAL) {
                const float2 a = f2_unpack(add), y = f2_unpack(dist);
                add = f2_pack(fmaf(-r.slope2, fabsf(y.x), a.x), fmaf(-r.slope2, fabsf(y.y), a.y));
            } else {
                add = ffma2(dist, sl, add);
            }
            dist = fadd2(dist, f2_pack(2.f, 2.f));
        }
        if constexpr (BIAS == kBiasTable) {
            if constexpr (GENERAL) {
                const int at = q0 - r.kg + q + p.far, top = 2 * p.far;
                add = fadd2(add, f2_pack(r.bias2[max(0, min(top, at))], r.bias2[max(0, min(top, at + 1))]));
            } else {
                add = fadd2(add, r.far_bias);
            }
        }
        const uint64_t v = f2_pack(u2f(sv[2 * i]), u2f(sv[2 * i + 1]));
        [[maybe_unused]] uint64_t th = 0;
        float2 x;
        if constexpr (CAP) {
            th = tanh2<decltype(how)::value>(fmul2(v, k2));
            x = f2_unpack(ffma2(th, cap2, add));
        } else {
            x = f2_unpack(ffma2(v, c2, add));
        }
        float p0 = ex2(x.x), p1 = ex2(x.y);
        if constexpr (GENERAL) {
            if (static_cast<uint32_t>(q - from) >= r.seen) p0 = 0.f;
            if (static_cast<uint32_t>(q + 1 - from) >= r.seen) p1 = 0.f;
        }
        pk[i] = pack_bf16(p0, p1);
        if constexpr (CAP && BIAS == kBiasTable) pw[i] = pack_f16_sat(p0, p1);
        if constexpr (CAP) {  // (tanh^2 - 1: dX, dK and dQ come with their sign turned)
            const float2 k = f2_unpack(fmul2(f2_pack(p0, p1), ffma2(th, th, f2_pack(-1.f, -1.f))));
            p0 = k.x;
            p1 = k.y;
        }
        if constexpr (keep_regs(CAP, BIAS) == 32) {
            keep[2 * i] = __float_as_uint(p0);
            keep[2 * i + 1] = __float_as_uint(p1);
        } else {
            keep[i] = pack_f16_sat(p0, p1);
        }
    };
    const auto all = [&](auto how, auto general_) {
#pragma unroll
        for (int i = 0; i < 16; ++i) weights(how, general_, i);
    };
    using Poly4 = std::integral_constant<int, kTanhPoly4>;
    using Exp = std::integral_constant<int, far_form(CAP)>;
    if constexpr (CAP) {
        float mx0 = 0.f, mx1 = 0.f;
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
            mx0 = fmax3(mx0, fabsf(u2f(sv[i])), fabsf(u2f(sv[i + 1])));
            mx1 = fmax3(mx1, fabsf(u2f(sv[i + 2])), fabsf(u2f(sv[i + 3])));
        }
        // (the few tiles at the edges: two forms)
        const float mx = fmaxf(mx0, mx1) * p.x_scale;
        const bool near = !__any_sync(FULL, !(mx <= kTanhNear)), mid = !__any_sync(FULL, !(mx <= kTanhMid));
        if (r.general && mid) all(Poly4{}, std::true_type{});
        else if (r.general) all(Exp{}, std::true_type{});
        else if (near) all(std::integral_constant<int, kTanhPoly3>{}, std::false_type{});
        else if (mid) all(Poly4{}, std::false_type{});
        else all(Exp{}, std::false_type{});
    } else if (r.general) {
        all(Exp{}, std::true_type{});
    } else {
        all(Exp{}, std::false_type{});
    }
}

// Of the same pairs: dX as bf16 pairs (ds) from dP.  nd4: the queries' -D.  pw: with a cap and SUMS, P.  SUMS: of
// the table's gradient, for far (1) or near (2) pairs: sums of dY = P (dP - D), in which a far bucket's pairs, almost
// all of a row's weight, nearly cancel.  So P is not the product's bf16 one there: 32 buckets, cap 50, 2500 tokens, an fp32
// gradient off by 1.7e-3 to 2.7e-3 with that, by 1.5e-4 to 3.9e-4 with fp16 of 2^15 times it (backward of 16 heads of 4096
// tokens at d = 128 328 -> 335 us, 48 of 2048 both ways at d = 64 417 -> 436; packed only where the gradient is wanted, by a
// branch, 395 and 500).
template <int CAP, int SUMS, int KEEP>
__device__ __forceinline__ void bwd_products(const uint32_t (&dp)[32], const uint32_t (&keep)[KEEP], [[maybe_unused]] const uint32_t (&pw)[16],
                                             const ulonglong2* nd4, [[maybe_unused]] int lane, uint32_t (&ds)[16],
                                             [[maybe_unused]] uint64_t& fsum, [[maybe_unused]] float& ahead,
                                             [[maybe_unused]] float& behind) {
    constexpr uint32_t FULL = 0xffffffffu;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const ulonglong2 nd = nd4[i >> 1];
        const uint64_t t2 = fadd2(f2_pack(u2f(dp[2 * i]), u2f(dp[2 * i + 1])), (i & 1) ? nd.y : nd.x);
        const float2 kk = KEEP == 32 ? make_float2(u2f(keep[2 * i % KEEP]), u2f(keep[(2 * i + 1) % KEEP])) : unpack_f16(keep[i]);
        const uint64_t d2 = fmul2(f2_pack(kk.x, kk.y), t2);
        const float2 dx = f2_unpack(d2);
        ds[i] = pack_bf16(dx.x, dx.y);
        if constexpr (SUMS != 0) {
            uint64_t dy = d2;
            if constexpr (CAP) {
                const float2 w = unpack_f16(pw[i]);
                dy = fmul2(f2_pack(w.x, w.y), t2);
            }
            if constexpr (SUMS == 1) {
                fsum = fadd2(fsum, dy);
            } else {
                // column q's value of key row l to lane (q - l) mod 32
                const float2 y = f2_unpack(dy);
                const float y0 = __shfl_sync(FULL, y.x, 2 * i - lane);
                const float y1 = __shfl_sync(FULL, y.y, 2 * i + 1 - lane);
                if (lane <= 2 * i) ahead += y0;
                else behind += y0;
                if (lane <= 2 * i + 1) ahead += y1;
                else behind += y1;
            }
        }
    }
}

// The workspace's parts, each 256-aligned.
struct BwdPlan {
    int near_lo = 0, near_n = 0, warps = 0;
    size_t dvec = 0, acc = 0, next = 0, spans = 0, order = 0, bias2 = 0, near = 0, far = 0, red = 0, bytes = 0;
};

}  // namespace

// The main kernel at d = 64.
cudaError_t launch_score_bwd64(const ScoreArgs& a, const ScoreBwdParams& p, float* acc, cudaStream_t stream);

}  // namespace fa
