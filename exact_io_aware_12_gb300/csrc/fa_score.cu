// Documents of a batch as ranges of tokens, for attention with masked scores.
//
// A document is a run of equal ids; ids below 0 are tokens of none.  One block per sequence:
// each thread takes a stretch of tokens and looks for the first and the last start of a run
// in it, two scans over the block give what lies before and behind, and a second walk writes
// [first token, end) of every token's run.  Bound by the ids' and ranges' latency: 16384
// tokens take about 5 us, once per call, beside kernels of hundreds.
#include <algorithm>

#include "fa_score.cuh"

namespace fa {
namespace {

constexpr int kSpanThreads = 1024;

__global__ void __launch_bounds__(kSpanThreads) fa_score_spans_kernel(const int* docs, int2* spans, int N) {
    __shared__ int before[kSpanThreads / 32], behind[kSpanThreads / 32];
    griddep_launch_dependents();
    griddep_wait();
    const int* id = docs + static_cast<long long>(blockIdx.x) * N;
    int2* out = spans + static_cast<long long>(blockIdx.x) * N;
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
    const int per = (N + kSpanThreads - 1) / kSpanThreads;
    const int i0 = min(N, t * per), i1 = min(N, i0 + per);
    int first = N, last = 0;  // starts of runs in this stretch (position 0 starts one)
    int prev = i0 > 0 && i0 < N ? id[i0 - 1] : 0;
    for (int i = i0; i < i1; ++i) {
        const int v = id[i];
        if (i == 0 || v != prev) {
            first = min(first, i);
            last = i;
        }
        prev = v;
    }
    // the last start before the stretch, the first behind it
    int mx = last, mn = first;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int a = __shfl_up_sync(0xffffffffu, mx, o), b = __shfl_down_sync(0xffffffffu, mn, o);
        if (lane >= o) mx = max(mx, a);
        if (lane + o < 32) mn = min(mn, b);
    }
    if (lane == 31) before[warp] = mx;
    if (lane == 0) behind[warp] = mn;
    int start = __shfl_up_sync(0xffffffffu, mx, 1), end = __shfl_down_sync(0xffffffffu, mn, 1);
    if (lane == 0) start = 0;
    if (lane == 31) end = N;
    __syncthreads();
    for (int w = 0; w < warp; ++w) start = max(start, before[w]);
    for (int w = warp + 1; w < kSpanThreads / 32; ++w) end = min(end, behind[w]);
    // backwards for the ends, then forwards for the starts
    for (int i = i1 - 1; i >= i0; --i) {
        out[i].y = end;
        if (i == 0 || id[i] != id[i - 1]) end = i;
    }
    for (int i = i0; i < i1; ++i) {
        if (i == 0 || id[i] != id[i - 1]) start = i;
        if (id[i] < 0) out[i] = make_int2(i, i);
        else out[i].x = start;
    }
}

}  // namespace

cudaError_t launch_score_spans(const int* docs, void* spans, int B, int N, cudaStream_t stream) {
    return launch_dependent(fa_score_spans_kernel, dim3(static_cast<unsigned>(B)), dim3(kSpanThreads), 0, stream, docs,
                            static_cast<int2*>(spans), N);
}

}  // namespace fa
