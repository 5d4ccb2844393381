// Arithmetic of the causal window beside sinks (key j is visible from query i iff j <= i
// and (j > i - window or j < sinks)), shared by its kernels.  Plain C++: every function
// also runs on the host, where the tests call it.
#pragma once

#include <cstdint>

#if defined(__CUDACC__)
#define FA_WIN_HD __host__ __device__ __forceinline__
#else
#define FA_WIN_HD inline
#endif

namespace fa {

// Whether a causal window of `window` keys (0: none) beside `sinks` first keys hides
// anything that the causal mask shows: the last query, N - 1, sees neither the keys
// from `sinks` on nor those within its window.  Where it hides nothing the forward
// kernels without a window run.
FA_WIN_HD bool window_hides(int N, int window, int sinks) {
    return window > 0 && static_cast<long long>(window) + sinks < N;
}

// A window (0: none) and a number of sinks, each up to the largest int, cut to the N keys
// that there are: the same keys are visible, and the kernels' sums of them with a block's
// size stay within an int.
struct WindowCut {
    int window, sinks;
};
FA_WIN_HD WindowCut cut_window(int N, int window, int sinks) {
    return {window < N ? window : N, sinks < N ? sinks : N};
}

// Key blocks of `block` keys that hold sinks and lie before block `win`.
FA_WIN_HD int sink_blocks(int sinks, int win, int block) {
    const int n = (sinks + block - 1) / block;
    return n < win ? n : win;
}

// Numbers x with lo <= x < hi, for bounds up to 2^30 either side of 0: one unsigned compare,
// x - lo < span, tells whether x is among them.  (2^30 - -2^30 passes an int.)
FA_WIN_HD uint32_t span(int lo, int hi) {
    return hi > lo ? static_cast<uint32_t>(hi) - static_cast<uint32_t>(lo) : 0u;
}

}  // namespace fa
