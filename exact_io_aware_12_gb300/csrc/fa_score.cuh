// Device parts that the kernels of attention with capped, biased or masked scores share.
#pragma once

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
// (6e-9), degree 5 up to kTanhMid (4e-8); beyond, 1 - 2 / (1 + e^2x) with the
// hardware's exponential and reciprocal (two of them per score, which a polynomial on the
// fp32 pipe beats while it is short).  tanh.approx is off by 2^-11 of its value: 0.02 of a
// score capped at 50.
constexpr float kTanhNear = 0.3f, kTanhMid = 0.75f;
enum : int { kTanhPoly3 = 0, kTanhPoly5 = 1, kTanhExp = 2 };
// Two values of tanh(x) at once, |x| within the bound of HOW.
template <int HOW>
__device__ __forceinline__ uint64_t tanh2(uint64_t x) {
    if constexpr (HOW == kTanhExp) {
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
            p = ffma2(u, c(-0.004736414644867182f), c(0.019611310213804245f));
            p = ffma2(u, p, c(-0.053358446806669235f));
            p = ffma2(u, p, c(0.13325688242912292f));
            p = ffma2(u, p, c(-0.33332979679107666f));
        }
        p = ffma2(u, p, c(1.f));
        return fmul2(x, p);
    }
}

}  // namespace fa
