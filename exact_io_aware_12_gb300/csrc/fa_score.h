// Arithmetic of attention with capped, biased or masked scores, shared by its kernels:
// which keys a query sees and which queries see a key, from the run of tokens (the
// document) that a token lies in; and the tiles these give.  Plain C++: every function
// also runs on the host, where the tests call it.
#pragma once

#include <cstdint>

#if defined(__CUDACC__)
#define FA_SCORE_HD __host__ __device__ __forceinline__
#else
#define FA_SCORE_HD inline
#endif

namespace fa {

// Farthest distance whose bias has an entry of its own, and most buckets.
constexpr int kScoreMaxFar = 1024, kScoreMaxBuckets = 1024;

// Positions [lo, hi).
struct ScoreRange {
    int lo, hi;
};

// Query i and key j of one sequence see one another iff both lie in one document [s, e) and,
// causal, j <= i or j < prefix, and with a window (0: none) j > i - window.  Without
// documents [s, e) is [0, N); a token in no document has s = e, its own position.
// Documents lie in order, so both ends of both ranges ascend (weakly) with the position: the
// ranges of a tile's first and last position bound those of all between.  A token in a
// document is in its own range; the others' are empty.
FA_SCORE_HD ScoreRange keys_of(int i, int s, int e, bool causal, int prefix, int window) {
    ScoreRange r{s, e};
    if (causal) {
        const int to = i + 1 > prefix ? i + 1 : prefix;
        r.hi = to < e ? to : e;
        if (window > 0 && i - window + 1 > s) r.lo = i - window + 1;
        if (s == e) r.lo = r.hi = i;
    }
    return r;
}
FA_SCORE_HD ScoreRange queries_of(int j, int s, int e, bool causal, int prefix, int window) {
    ScoreRange r{s, e};
    if (causal) {
        if (j >= prefix && j > s) r.lo = j;
        // (window <= N: no sum passes an int)
        if (window > 0 && j + window < e) r.hi = j + window;
        if (s == e) r.lo = r.hi = j;
    }
    return r;
}

// Blocks of `block` positions that hold [lo, hi), at least one.
FA_SCORE_HD ScoreRange blocks_of(int lo, int hi, int block) {
    const int a = lo / block, b = (hi + block - 1) / block;
    return {a, b > a ? b : a + 1};
}

// Whether every pair of a query in [q, q + n) and a key in [k, k + n) is at a distance
// q - k of `far` or more (1), -far or less (-1), or neither (0).
FA_SCORE_HD int far_side(int q, int k, int n, int far) {
    if (q - (k + n - 1) >= far) return 1;
    if (k - (q + n - 1) >= far) return -1;
    return 0;
}

// Offsets (query tile - key tile, of `block` positions) at which some pair is nearer than
// `far`: [-n, n] with this n.
FA_SCORE_HD int near_tiles(int far, int block) { return (far + block - 2) / block; }

}  // namespace fa
