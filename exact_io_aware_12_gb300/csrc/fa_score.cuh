// Device parts that the kernels of attention with capped, biased or masked scores share.
#pragma once

#include <cstring>

#include "fa_internal.h"
#include "fa_score.h"
#include "ptx.cuh"

namespace fa {

enum : int { kBiasNone = 0, kBiasSlopes = 1, kBiasTable = 2 };

struct ScoreMask {
    const int2* spans;  // [B][N], or null: one document
    const int* prefix;  // [B], or null
    int N, window;
    bool causal;
};

__device__ __forceinline__ int prefix_of(const ScoreMask& m, int b) {
    return m.causal && m.prefix ? max(0, min(m.N, m.prefix[b])) : 0;
}
__device__ __forceinline__ int2 span_of(const ScoreMask& m, int b, int pos) {
    return m.spans ? m.spans[static_cast<long long>(b) * m.N + pos] : make_int2(0, m.N);
}
__device__ __forceinline__ ScoreRange keys_of(const ScoreMask& m, int b, int i, int prefix) {
    const int2 s = span_of(m, b, i);
    return keys_of(i, s.x, s.y, m.causal, prefix, m.window);
}
__device__ __forceinline__ ScoreRange queries_of(const ScoreMask& m, int b, int j, int prefix) {
    const int2 s = span_of(m, b, j);
    return queries_of(j, s.x, s.y, m.causal, prefix, m.window);
}

// The bias of head h at entry i of the buckets' map: 0 where the map names no bucket.
__device__ __forceinline__ float table_bias(const void* table, bool f32, const int* buckets, int num_buckets, int H, int h,
                                            int i) {
    const int e = buckets[i];
    if (static_cast<unsigned>(e) >= static_cast<unsigned>(num_buckets)) return 0.f;
    const long long at = static_cast<long long>(e) * H + h;
    if (f32) return static_cast<const float*>(table)[at];
    return __uint_as_float(static_cast<uint32_t>(static_cast<const unsigned short*>(table)[at]) << 16);
}

__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// tanh(x) for |x| <= kTanhNear, by x p(x^2): p of degree 3 fitted to least largest error
// (6e-9), degree 4 up to kTanhMid (1.4e-8); beyond, 1 - 2 / (1 + e^2x) with the
// hardware's exponential and reciprocal (two of them per score, which a polynomial on the
// fp32 pipe beats while it is short: forward of 16 heads of 8192 tokens, window 4096, 229 us by
// the first, 294 by the last).  tanh.approx is off by 2^-11 of its value: 0.02 of a score
// capped at 50.
//
// The last form is off by an absolute error, whatever x, and so by that part of the cap: with the exponential off by
// d = 2^-22.7 of its value and the reciprocal by 2^-23.2 (the largest of all fp32 arguments here), and each rounding by
// 2^-24, (1 - t^2)/2 (d + 2^-22 |x|) + (1 - t)(2^-23.2 + 2^-24) + 2^-25 <= 3.3 2^-23 = 3.9e-7; the largest measured, over all
// fp32 |x| from 2^-14 to 16, is 2.4e-7 (x > 0: 1.8e-7).  That is 1.7e-4 of a score where the cap is kCapExact, 710, but for
// larger ones too much beside small scores.  There kTanhSafe takes, score by score, the polynomial up to kTanhMid, and is
// off by 5e-7 of its own value at most (measured; 8e-7 by the bound).
constexpr float kTanhNear = 0.3f, kTanhMid = 0.5f;
constexpr float kCapExact = 1024.f;  // log2 units
enum : int { kTanhPoly3 = 0, kTanhPoly4 = 1, kTanhExp = 2, kTanhSafe = 3 };
// A kernel's cap: none, one up to kCapExact, a larger one (kernels of their own: another form in the same ones cost
// 5 to 10% of those with a common cap).
enum : int { kCapNone = 0, kCapCommon = 1, kCapLarge = 2 };
__host__ __device__ constexpr int far_form(int cap) { return cap == kCapLarge ? kTanhSafe : kTanhExp; }
inline int cap_of(float softcap) {
    return softcap <= 0.f ? kCapNone : softcap * 1.44269504088896341f > kCapExact ? kCapLarge : kCapCommon;
}
// Two values of tanh(x) at once, |x| within the bound of HOW.
template <int HOW>
__device__ __forceinline__ uint64_t tanh2(uint64_t x) {
    if constexpr (HOW == kTanhSafe) {
        const float2 v = f2_unpack(x), p = f2_unpack(tanh2<kTanhPoly4>(x)), e = f2_unpack(tanh2<kTanhExp>(x));
        return f2_pack(fabsf(v.x) <= kTanhMid ? p.x : e.x, fabsf(v.y) <= kTanhMid ? p.y : e.y);
    } else if constexpr (HOW == kTanhExp) {
        constexpr float k = 2.f * 1.44269504088896341f;
        const float2 v = f2_unpack(x);
        return f2_pack(fmaf(-2.f, rcp(1.f + ex2(k * v.x)), 1.f), fmaf(-2.f, rcp(1.f + ex2(k * v.y)), 1.f));
    } else {
        const uint64_t u = fmul2(x, x);
        const auto c = [](float v) { return f2_pack(v, v); };
        uint64_t p;
        if constexpr (HOW == kTanhPoly3) {
            p = ffma2(u, c(-0.05022904649376869f), c(0.1331268697977066f));
            p = ffma2(u, p, c(-0.3333296477794647f));
        } else {
            p = ffma2(u, c(0.017151299864053726f), c(-0.05299423262476921f));
            p = ffma2(u, p, c(0.13324907422065735f));
            p = ffma2(u, p, c(-0.33333075046539307f));
        }
        p = ffma2(u, p, c(1.f));
        return fmul2(x, p);
    }
}

// Scores capped, in log2 units: what cap log2(e) tanh(s tau / cap) takes.
struct CapScale {
    float k, k_exp, cap2;
    uint64_t k_2, cap_2, cap_m2, near[4], mid[5];  // pairs: a paired instruction takes them as they come
    __host__ __device__ CapScale() {}
    static uint64_t pair(float v) {
        uint32_t x;
        std::memcpy(&x, &v, 4);
        return static_cast<uint64_t>(x) << 32 | x;
    }
    CapScale(float tau, float cap) {
        const float log2e = 1.44269504088896341f, lin = tau * log2e;
        k = tau / cap;
        k_exp = 2.f * log2e * k;
        cap2 = cap * log2e;
        k_2 = pair(k);
        cap_2 = pair(cap2);
        cap_m2 = pair(-2.f * cap2);
        // the fits of tanh2, times tau log2(e): y = s p((k s)^2) needs no products beside p's
        const float n[4] = {1.f, -0.3333296477794647f, 0.1331268697977066f, -0.05022904649376869f};
        const float m[5] = {1.f, -0.33333075046539307f, 0.13324907422065735f, -0.05299423262476921f, 0.017151299864053726f};
        for (int i = 0; i < 4; ++i) near[i] = pair(lin * n[i]);
        for (int i = 0; i < 5; ++i) mid[i] = pair(lin * m[i]);
    }
};
// Two capped scores plus `add`.
template <int HOW>
__device__ __forceinline__ uint64_t cap_score2(const CapScale& c, uint64_t s, uint64_t add) {
    if constexpr (HOW == kTanhSafe) {
        return ffma2(tanh2<kTanhSafe>(fmul2(s, c.k_2)), c.cap_2, add);
    } else if constexpr (HOW == kTanhExp) {
        const float2 v = f2_unpack(s);
        const uint64_t r = f2_pack(rcp(1.f + ex2(c.k_exp * v.x)), rcp(1.f + ex2(c.k_exp * v.y)));
        return ffma2(c.cap_m2, r, fadd2(c.cap_2, add));
    } else {
        constexpr int n = HOW == kTanhPoly3 ? 4 : 5;
        const uint64_t* q = HOW == kTanhPoly3 ? c.near : c.mid;
        const uint64_t t = fmul2(s, c.k_2), u = fmul2(t, t);
        uint64_t p = q[n - 1];
#pragma unroll
        for (int i = n - 2; i >= 0; --i) p = ffma2(u, p, q[i]);
        return ffma2(s, p, add);
    }
}

}  // namespace fa
