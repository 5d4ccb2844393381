// Documents of a batch as ranges of tokens, for attention with masked scores.
//
// A document is a run of equal ids; ids below 0 are tokens of none.  One block per sequence
// takes 32768 tokens at a time: where a run starts is a bit per token (a ballot per 32), two scans over
// the block's words give the last start before each and the first behind it, and a second walk writes
// [first token, end) of every token's run.  Longer sequences are walked backwards for the ends and then
// forwards for the starts.  (A thread per stretch of tokens, walked one by one, took 48 us for
// 16384 tokens.)
//
// Documents of uneven length give tiles of uneven work, which left the SMs waiting for the last
// long ones: the same block then sorts its sequence's tiles by the blocks that they visit, most
// first, into the order in which the kernels behind it take them.
#include <algorithm>

#include "fa_score.cuh"

namespace fa {
namespace {

constexpr int kSpanThreads = 1024;
constexpr int kChunk = 32 * kSpanThreads;  // tokens
constexpr int kBins = 1024;  // of work: blocks visited, up to this many

// The n tiles of `rows` positions, in the order of the blocks that they visit, most first (among those of
// equal work in any order).  KEYS: tiles of keys, else of queries.
template <bool KEYS>
__device__ void sort_tiles(const ScoreMask& m, int b, int prefix, int rows, int n, int* order, int* bins, int* sums) {
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
    const auto bin_of = [&](int i) {
        const int first = i * rows, last = min(m.N, first + rows) - 1;
        const ScoreRange a = KEYS ? queries_of(m, b, first, prefix) : keys_of(m, b, first, prefix);
        const ScoreRange z = KEYS ? queries_of(m, b, last, prefix) : keys_of(m, b, last, prefix);
        const ScoreRange r = blocks_of(a.lo, z.hi, 128);
        return kBins - min(kBins, r.hi - r.lo);
    };
    bins[t] = 0;
    const int own = t < n ? bin_of(t) : 0;  // of a thread's first tile, mostly its only one
    __syncthreads();
    for (int i = t; i < n; i += kSpanThreads) atomicAdd(&bins[i == t ? own : bin_of(i)], 1);
    __syncthreads();
    const int mine = bins[t];
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) sums[warp] = incl;
    __syncthreads();
    int at = incl - mine;
    for (int w = 0; w < warp; ++w) at += sums[w];
    bins[t] = at;
    __syncthreads();
    for (int i = t; i < n; i += kSpanThreads) order[static_cast<long long>(b) * n + atomicAdd(&bins[i == t ? own : bin_of(i)], 1)] = i;
    __syncthreads();
}

__global__ void __launch_bounds__(kSpanThreads) fa_score_spans_kernel(const int* docs, int2* spans, ScoreMask mask, ScoreOrder order) {
    __shared__ int before[kSpanThreads / 32], behind[kSpanThreads / 32];
    __shared__ int bins[kBins];
    __shared__ uint32_t start_bits[kChunk / 32], none_bits[kChunk / 32];
    __shared__ int word_first[kChunk / 32], word_end[kChunk / 32];
    static_assert(kChunk / 32 == kSpanThreads, "a word per thread");
    static_assert(kBins == kSpanThreads, "a bin per thread");
    griddep_launch_dependents();
    griddep_wait();
    const int N = mask.N;
    const int* id = docs + static_cast<long long>(blockIdx.x) * N;
    int2* out = spans + static_cast<long long>(blockIdx.x) * N;
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
    // tokens [c0, c0 + kChunk): starts (given the last start before them) and ends (the first behind them); returns
    // the last start (or first) of all up to (from) these
    const auto chunk = [&](int c0, bool starts, bool ends, int& carry_start, int& carry_end) {
        const int words = (min(kChunk, N - c0) + 31) / 32;
#pragma unroll 8
        for (int k = 0; k < (words + 31) / 32; ++k) {
            const int w = k * 32 + warp, i = c0 + 32 * w + lane;
            int v = 0, prev = 0;
            if (i < N) {
                v = id[i];
                prev = i > 0 ? id[i - 1] : 0;
            }
            const uint32_t start = __ballot_sync(0xffffffffu, i < N && (i == 0 || v != prev));
            const uint32_t none = __ballot_sync(0xffffffffu, v < 0);
            if (lane == 0) {
                start_bits[w] = start;
                none_bits[w] = none;
            }
        }
        __syncthreads();
        // word t: the last start before it, the first behind it
        const uint32_t mine = t < words ? start_bits[t] : 0u;
        int mx = mine ? c0 + 32 * t + 31 - __clz(mine) : -1, mn = mine ? c0 + 32 * t + __ffs(mine) - 1 : N;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, mx, o), y = __shfl_down_sync(0xffffffffu, mn, o);
            if (lane >= o) mx = max(mx, x);
            if (lane + o < 32) mn = min(mn, y);
        }
        if (lane == 31) before[warp] = mx;
        if (lane == 0) behind[warp] = mn;
        int first = __shfl_up_sync(0xffffffffu, mx, 1), end = __shfl_down_sync(0xffffffffu, mn, 1);
        if (lane == 0) first = -1;
        if (lane == 31) end = N;
        __syncthreads();
        int all_first = carry_start, all_end = carry_end;
        for (int w = 0; w < 32; ++w) {
            if (w < warp) first = max(first, before[w]);
            if (w > warp) end = min(end, behind[w]);
            all_first = max(all_first, before[w]);
            all_end = min(all_end, behind[w]);
        }
        word_first[t] = max(first, carry_start);
        word_end[t] = min(end, carry_end);
        __syncthreads();
#pragma unroll 4
        for (int k = 0; k < (words + 31) / 32; ++k) {
            const int w = k * 32 + warp, i = c0 + 32 * w + lane;
            if (i >= N) break;
            const uint32_t upto = (2u << lane) - 1u, b = start_bits[w];
            const int x = b & upto ? c0 + 32 * w + 31 - __clz(b & upto) : word_first[w];
            const int y = b & ~upto ? c0 + 32 * w + __ffs(b & ~upto) - 1 : word_end[w];
            if (none_bits[w] >> lane & 1u) out[i] = make_int2(i, i);
            else if (starts && ends) out[i] = make_int2(x, y);
            else if (starts) out[i].x = x;
            else out[i].y = y;
        }
        carry_start = all_first;
        carry_end = all_end;
        __syncthreads();
    };
    int none = N, first = -1, end = N;
    if (N <= kChunk) {
        chunk(0, true, true, first, end);
    } else {
        for (int c = (N - 1) / kChunk; c >= 0; --c) {
            none = -1;
            chunk(c * kChunk, false, true, none, end);
        }
        for (int c0 = 0; c0 < N; c0 += kChunk) {
            none = N;
            chunk(c0, true, false, first, none);
        }
    }
    __syncthreads();
    mask.spans = spans;
    const int b = static_cast<int>(blockIdx.x), prefix = prefix_of(mask, b);
    if (order.queries) sort_tiles<false>(mask, b, prefix, 128, (N + 127) / 128, order.queries, bins, before);
    if (order.pairs) sort_tiles<false>(mask, b, prefix, 256, (N + 255) / 256, order.pairs, bins, before);
    if (order.keys) sort_tiles<true>(mask, b, prefix, 128, (N + 127) / 128, order.keys, bins, before);
}

}  // namespace

size_t score_spans_bytes(int B, int N) { return (static_cast<size_t>(B) * N * sizeof(int2) + 255) / 256 * 256; }

cudaError_t launch_score_spans(const ScoreArgs& a, void* spans, const ScoreOrder& order, cudaStream_t stream) {
    ScoreMask m;
    m.spans = nullptr;
    m.prefix = a.mod.prefix;
    m.N = a.N;
    m.window = a.mod.window;
    m.causal = a.causal;
    return launch_dependent(fa_score_spans_kernel, dim3(static_cast<unsigned>(a.B)), dim3(kSpanThreads), 0, stream, a.mod.docs,
                            static_cast<int2*>(spans), m, order);
}

}  // namespace fa
