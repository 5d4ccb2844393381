// Appending new keys and values to a paged cache, with the rotation of keys (and of the
// same tokens' queries) by their position on the way.
//
// Mathematics: token i of sequence b stands at position p = lens[b] + i.  Each pair
// (x, y) of the first `rot` columns, paired as (c, c + rot / 2) or, interleaved, as
// (2c, 2c + 1), turns by p * inv_freq[c]: (x cos - y sin, y cos + x sin), in fp32 from
// the bf16 inputs and rounded once.  The angle is kept as a 64-bit fraction of a turn
// (turn_fraction), so position 2^20 is as exact as position 1.
//
// An e4m3 page holds codes and one scale per head for K and one for V, a power of two
// (page_scale_exp).  The scale follows from the values before the rotation - 1.5 times
// their largest magnitude for rotated keys, since a turned pair is at most sqrt(2) times
// its larger half, and that magnitude itself for values and unrotated keys - so it
// depends neither on positions nor on rounding.  A page begun by an earlier call keeps
// the larger of its scale and the new one; where that grows, its codes are rescaled
// (exactly, but for values that fall among the subnormals, which round to nearest even).
//
// Both kernels only move bytes: each input is read and each output written once (the
// 8-bit kernel reads its rows twice, the second time from L1/L2).  A thread owns 16
// columns of a token (two 16-byte pieces that rotate into each other) and one token's
// eight (cos, sin) stay in registers while it walks heads.
#include <cuda_bf16.h>

#include <algorithm>

#include "fa_internal.h"
#include "fa_paged.h"
#include "ptx.cuh"

namespace fa {
namespace {

struct AppendParams {
    const __nv_bfloat16* q;   // [T][H][d] by strides, or null
    const __nv_bfloat16* k;   // [T][H_kv][d] by strides
    const __nv_bfloat16* v;
    __nv_bfloat16* q_out;
    uint8_t* kc;              // cache [num_pages][H_kv][page_size][d]
    uint8_t* vc;
    float* k_scale;           // 8-bit: [num_pages][H_kv]
    float* v_scale;
    const int* table;
    const int* lens;
    const int* cu;            // [B + 1], or null: T / B tokens each
    const uint64_t* inv_freq; // [rot / 2] (the bits of doubles)
    long long q_st, q_sh, k_st, k_sh, v_st, v_sh, o_st, o_sh;  // elements
    int T, B, H, H_kv, rot, interleaved, num_pages, max_pages, shift;
    int groups;               // head groups (grid.y)
    int kv_blocks;            // 8-bit: blocks (x) of the pages, the rest rotate queries
    unsigned int* err;
};

__device__ __forceinline__ float lo_f(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float hi_f(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }

// Records a length, token count or page number out of bounds.
__device__ __forceinline__ void page_error(unsigned int* err) { atomicCAS(err, 0u, kErrPage); }

__device__ __forceinline__ int cu_of(const AppendParams& p, int b) {
    return p.cu ? __ldg(p.cu + b) : b * (p.T / p.B);
}

// The largest b in [0, B) with key(b) <= x (0 if none), key non-decreasing: 32 probes at a
// time, so a warp needs two rounds of loads for 1024 sequences.  All lanes take part.
template <typename Key>
__device__ __forceinline__ int last_not_above(int B, long long x, Key key) {
    const int lane = static_cast<int>(lane_id());
    int lo = 0, n = B;  // the answer lies in [lo, lo + n)
    while (n > 1) {
        const int step = (n + 31) / 32;
        const int at = lo + lane * step;
        const bool le = lane * step < n && key(at) <= x;
        const uint32_t m = __ballot_sync(0xffffffffu, le);
        const int j = m ? 31 - __clz(m) : 0;
        lo += j * step;
        n = min(step, n - j * step);
    }
    return lo;
}

// One token's eight (cos, sin): pairs [8 u, 8 u + 8).
struct Turn {
    float c[8], s[8];
};
__device__ __forceinline__ void turn_at(const AppendParams& p, int u, int pos, Turn& t) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint64_t turns = turn_fraction(__ldg(p.inv_freq + 8 * u + i)) * static_cast<uint64_t>(pos);
        // half turns in [-1, 1): the top 32 bits
        const float half = static_cast<float>(static_cast<int32_t>(turns >> 32)) * 0x1p-31f;
        sincospif(half, &t.s[i], &t.c[i]);
    }
}

// The two 16-byte pieces of 8 columns that unit u of a row owns.
__device__ __forceinline__ void pieces(const AppendParams& p, int u, int& a, int& b) {
    const int ru = p.rot / 16;  // units that rotate
    if (!p.interleaved && u < ru) {
        a = u;
        b = u + ru;
    } else {
        a = 2 * u;  // (past the rotated columns, too: 2 ru pieces lie before them)
        b = 2 * u + 1;
    }
}

// Rotates 16 columns (two pieces) into fp32.
__device__ __forceinline__ void rotate(const AppendParams& p, const uint4& wa, const uint4& wb, const Turn& t,
                                       float (&x)[16]) {
    const uint32_t a[4] = {wa.x, wa.y, wa.z, wa.w}, b[4] = {wb.x, wb.y, wb.z, wb.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = lo_f(a[i]);
        x[2 * i + 1] = hi_f(a[i]);
        x[8 + 2 * i] = lo_f(b[i]);
        x[8 + 2 * i + 1] = hi_f(b[i]);
    }
    if (p.interleaved) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float e = x[2 * i], o = x[2 * i + 1];
            x[2 * i] = e * t.c[i] - o * t.s[i];
            x[2 * i + 1] = o * t.c[i] + e * t.s[i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float e = x[i], o = x[8 + i];
            x[i] = e * t.c[i] - o * t.s[i];
            x[8 + i] = o * t.c[i] + e * t.s[i];
        }
    }
}

__device__ __forceinline__ uint4 pack8(const float* x) {
    return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}

// Rows (tokens) of a block are consecutive; heads [h0, h1) of the list [Q heads | K
// heads | V heads] are walked by every row.  Used by both kernels (the 8-bit kernel
// sends its queries here).  Measured: see fa_kv_append_kernel.
template <int D>
__device__ __forceinline__ void append_rows(const AppendParams& p, int t_first, int h0, int h1) {
    constexpr int U = D / 16;  // units per row
    const int u = threadIdx.x % U;
    const int warp_t = t_first + static_cast<int>(threadIdx.x & ~31u) / U;  // the warp's first token
    if (warp_t >= p.T) return;  // warp-uniform
    const int t = t_first + static_cast<int>(threadIdx.x) / U;
    int b = last_not_above(p.B, warp_t, [&](int i) { return static_cast<long long>(cu_of(p, i)); });
    if (t >= p.T) return;
    while (b + 1 < p.B && cu_of(p, b + 1) <= t) ++b;
    const int c0 = cu_of(p, b), c1 = cu_of(p, b + 1);
    if (t < c0 || t >= c1) return;  // a row behind the last sequence: left as it is
    const int past = __ldg(p.lens + b);
    const long long pos = static_cast<long long>(past) + (t - c0);
    const int pg = past < 0 ? -1 : page_of(p.table + static_cast<long long>(b) * p.max_pages, p.max_pages,
                                           p.num_pages, p.shift, pos);
    if (pg < 0 && h1 > p.H) page_error(p.err);
    const bool turns = u < p.rot / 16;
    Turn tr;
    if (turns && h0 < p.H + p.H_kv) turn_at(p, u, static_cast<int>(pos), tr);
    int a, c;
    pieces(p, u, a, c);
    const int off = static_cast<int>(pos) & ((1 << p.shift) - 1);
    constexpr int kBatch = 4;  // heads whose loads are in flight together
    for (int hb = h0; hb < h1; hb += kBatch) {
        uint4 wa[kBatch], wb[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int h = hb + i;
            if (h >= h1) break;
            const __nv_bfloat16* src =
                h < p.H            ? p.q + t * p.q_st + h * p.q_sh
                : h < p.H + p.H_kv ? p.k + t * p.k_st + (h - p.H) * p.k_sh
                                   : p.v + t * p.v_st + (h - p.H - p.H_kv) * p.v_sh;
            wa[i] = __ldg(reinterpret_cast<const uint4*>(src) + a);
            wb[i] = __ldg(reinterpret_cast<const uint4*>(src) + c);
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int h = hb + i;
            if (h >= h1) break;
            if (turns && h < p.H + p.H_kv) {
                float x[16];
                rotate(p, wa[i], wb[i], tr, x);
                wa[i] = pack8(x);
                wb[i] = pack8(x + 8);
            }
            __nv_bfloat16* dst;
            if (h < p.H) {
                dst = p.q_out + t * p.o_st + h * p.o_sh;
            } else {
                if (pg < 0) continue;
                const bool is_k = h < p.H + p.H_kv;
                const int hk = h - p.H - (is_k ? 0 : p.H_kv);
                dst = reinterpret_cast<__nv_bfloat16*>(is_k ? p.kc : p.vc) +
                      (((static_cast<long long>(pg) * p.H_kv + hk) << p.shift) + off) * D;
            }
            reinterpret_cast<uint4*>(dst)[a] = wa[i];
            reinterpret_cast<uint4*>(dst)[c] = wb[i];
        }
    }
}

constexpr int kAppendThreads = 256;

template <int D>
__global__ void __launch_bounds__(kAppendThreads) fa_kv_append_kernel(const AppendParams p) {
    const int n = p.H + 2 * p.H_kv;
    const int per = (n + p.groups - 1) / p.groups;
    const int h0 = static_cast<int>(blockIdx.y) * per;
    append_rows<D>(p, static_cast<int>(blockIdx.x) * (kAppendThreads / (D / 16)), h0, min(n, h0 + per));
}

__device__ __forceinline__ float amax8(const uint4& w, float m) {
    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) m = fmaxf(m, fmaxf(fabsf(lo_f(x[i])), fabsf(hi_f(x[i]))));  // (NaN is passed over)
    return m;
}

// Four e4m3 codes rescaled by r (rounded to nearest even).
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float r) {
    uint32_t lo, hi;
    widen_e4m3x4(w, lo, hi);
    const float2 a = unpack_f16(lo), b = unpack_f16(hi);
    return pack_e4m3x4(a.x * r, a.y * r, b.x * r, b.y * r);
}

constexpr int kMaxGroupHeads = 64;  // heads (of the list [K | V]) that one block walks

// One block per (sequence, page reached, head group): it alone writes that page's heads,
// so the scale needs no communication.  Two passes over the page's new rows, the second
// from L1/L2: the largest magnitude per head, then rotate, scale, round and store.
template <int D>
__global__ void __launch_bounds__(256) fa_kv_append_fp8_kernel(const AppendParams p) {
    constexpr int U = D / 16;
    __shared__ uint32_t amax_s[kMaxGroupHeads];
    __shared__ float scale_s[kMaxGroupHeads], inv_s[kMaxGroupHeads];
    const int rows = static_cast<int>(blockDim.x) / U;
    const int bx = static_cast<int>(blockIdx.x);
    if (bx >= p.kv_blocks) {
        const int per = (p.H + p.groups - 1) / p.groups;
        const int h0 = static_cast<int>(blockIdx.y) * per;
        if (h0 < p.H) append_rows<D>(p, (bx - p.kv_blocks) * rows, h0, min(p.H, h0 + per));
        return;
    }
    const int n_list = 2 * p.H_kv;
    const int per = (n_list + p.groups - 1) / p.groups;
    const int h0 = static_cast<int>(blockIdx.y) * per, h1 = min(n_list, h0 + per);
    if (h0 >= h1) return;
    // this block's sequence and page
    const int b = last_not_above(p.B, bx, [&](int i) { return first_unit(cu_of(p, i), i, p.shift); });
    const int c0 = cu_of(p, b), c1 = cu_of(p, b + 1);
    const int i = static_cast<int>(bx - first_unit(c0, b, p.shift));
    const int past = __ldg(p.lens + b);
    if (c0 < 0 || c1 > p.T || c1 <= c0 || past < 0 || i < 0) {
        if (c1 != c0 && threadIdx.x == 0) page_error(p.err);
        return;
    }
    if (i >= pages_reached(past, c1 - c0, p.shift)) return;
    const int page = 1 << p.shift;
    const long long page0 = ((static_cast<long long>(past) >> p.shift) + i) << p.shift;  // position of the page's row 0
    const int r0 = i == 0 ? static_cast<int>(past - page0) : 0;                          // first new row
    const int r1 = static_cast<int>(min(static_cast<long long>(page), static_cast<long long>(past) + (c1 - c0) - page0));
    const int t0 = c0 + static_cast<int>(page0 + r0 - past);  // the token of row r0
    const int pg = page_of(p.table + static_cast<long long>(b) * p.max_pages, p.max_pages, p.num_pages, p.shift, page0);
    if (pg < 0) {
        if (threadIdx.x == 0) page_error(p.err);
        return;
    }
    const int u = threadIdx.x % U, tr = threadIdx.x / U;
    int a, c;
    pieces(p, u, a, c);
    for (int h = threadIdx.x; h < h1 - h0; h += blockDim.x) amax_s[h] = 0u;
    __syncthreads();
    const auto row_of = [&](int h, int r) {
        const long long t = t0 + (r - r0);
        return h < p.H_kv ? p.k + t * p.k_st + h * p.k_sh : p.v + t * p.v_st + (h - p.H_kv) * p.v_sh;
    };
    // 1. the largest magnitude of each head's new rows
    for (int h = h0; h < h1; ++h) {
        float m = 0.f;
        for (int r = r0 + tr; r < r1; r += rows) {
            const uint4* src = reinterpret_cast<const uint4*>(row_of(h, r));
            m = amax8(__ldg(src + a), m);
            m = amax8(__ldg(src + c), m);
        }
        const uint32_t mw = __reduce_max_sync(0xffffffffu, __float_as_uint(m));  // (non-negative: bits keep the order)
        if ((threadIdx.x & 31) == 0 && mw != 0u) atomicMax(&amax_s[h - h0], mw);
    }
    __syncthreads();
    // 2. the scales; a page begun earlier keeps the larger one, its codes rescaled
    for (int h = h0; h < h1; ++h) {
        const bool is_k = h < p.H_kv;
        const int hk = is_k ? h : h - p.H_kv;
        const long long ph = static_cast<long long>(pg) * p.H_kv + hk;
        float* scale = (is_k ? p.k_scale : p.v_scale) + ph;
        float bound = __uint_as_float(amax_s[h - h0]);
        if (is_k && p.rot > 0) bound *= 1.5f;
        const float need = __uint_as_float(static_cast<uint32_t>(page_scale_exp(__float_as_uint(bound)) + 127) << 23);
        float s = need;
        if (r0 > 0) {
            const float old = *scale;
            s = fmaxf(old, need);
            if (s > old) {
                const float ratio = old / s;
                uint4* codes = reinterpret_cast<uint4*>((is_k ? p.kc : p.vc) + ((ph << p.shift) * D));
                for (int e = threadIdx.x; e < r0 * (D / 16); e += blockDim.x) {
                    uint4 w = codes[e];
                    w.x = rescale4(w.x, ratio);
                    w.y = rescale4(w.y, ratio);
                    w.z = rescale4(w.z, ratio);
                    w.w = rescale4(w.w, ratio);
                    codes[e] = w;
                }
            }
        }
        if (threadIdx.x == 0) {
            scale_s[h - h0] = s;
            inv_s[h - h0] = 1.f / s;  // exact for a power of two
        }
    }
    __syncthreads();  // every thread has read the old scales
    for (int h = h0 + static_cast<int>(threadIdx.x); h < h1; h += blockDim.x) {
        const bool is_k = h < p.H_kv;
        (is_k ? p.k_scale : p.v_scale)[static_cast<long long>(pg) * p.H_kv + (is_k ? h : h - p.H_kv)] = scale_s[h - h0];
    }
    // 3. rotate, scale, round, store
    const bool turns = u < p.rot / 16;
    for (int r = r0 + tr; r < r1; r += rows) {
        Turn t;
        if (turns && h0 < p.H_kv) turn_at(p, u, static_cast<int>(page0 + r), t);
        for (int h = h0; h < h1; ++h) {
            const bool is_k = h < p.H_kv;
            const uint4* src = reinterpret_cast<const uint4*>(row_of(h, r));
            const uint4 wa = __ldg(src + a), wb = __ldg(src + c);
            float x[16];
            if (turns && is_k) {
                rotate(p, wa, wb, t, x);
            } else {
                const uint32_t w[8] = {wa.x, wa.y, wa.z, wa.w, wb.x, wb.y, wb.z, wb.w};
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    x[2 * e] = lo_f(w[e]);
                    x[2 * e + 1] = hi_f(w[e]);
                }
            }
            const float inv = inv_s[h - h0];
            uint32_t o[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                o[e] = pack_e4m3x4(x[4 * e] * inv, x[4 * e + 1] * inv, x[4 * e + 2] * inv, x[4 * e + 3] * inv);
            uint8_t* dst = (is_k ? p.kc : p.vc) +
                           (((static_cast<long long>(pg) * p.H_kv + (is_k ? h : h - p.H_kv)) << p.shift) + r) * D;
            reinterpret_cast<uint2*>(dst)[a] = make_uint2(o[0], o[1]);
            reinterpret_cast<uint2*>(dst)[c] = make_uint2(o[2], o[3]);
        }
    }
}

}  // namespace

cudaError_t launch_kv_append(const AppendArgs& a, cudaStream_t stream) {
    AppendParams p;
    p.q = static_cast<const __nv_bfloat16*>(a.q);
    p.k = static_cast<const __nv_bfloat16*>(a.k);
    p.v = static_cast<const __nv_bfloat16*>(a.v);
    p.q_out = static_cast<__nv_bfloat16*>(a.q_out);
    p.kc = static_cast<uint8_t*>(a.cache.K);
    p.vc = static_cast<uint8_t*>(a.cache.V);
    p.k_scale = a.cache.k_scale;
    p.v_scale = a.cache.v_scale;
    p.table = a.cache.page_table;
    p.lens = a.cache.lens;
    p.cu = a.cu_new;
    p.inv_freq = reinterpret_cast<const uint64_t*>(a.inv_freq);
    p.q_st = a.q_st;
    p.q_sh = a.q_sh;
    p.k_st = a.k_st;
    p.k_sh = a.k_sh;
    p.v_st = a.v_st;
    p.v_sh = a.v_sh;
    p.o_st = a.o_st;
    p.o_sh = a.o_sh;
    p.T = a.T;
    p.B = a.cache.B;
    p.H = a.q ? a.H : 0;
    p.H_kv = a.cache.H_kv;
    p.rot = a.rot;
    p.interleaved = a.interleaved;
    p.num_pages = a.cache.num_pages;
    p.max_pages = a.cache.max_pages;
    p.shift = a.cache.shift;
    p.err = a.err;
    const int d = a.cache.d, units = d / 16;
    // Heads are cut into groups so that about two full machines of threads exist: with
    // few tokens each thread takes one head (latency), with many it walks several on one
    // set of angles.
    const long long threads = static_cast<long long>(a.T) * units;
    const long long want = (2ll * 152 * 2048 + threads - 1) / threads;
    if (a.cache.k_scale == nullptr) {
        const int n = p.H + 2 * p.H_kv;
        p.groups = static_cast<int>(std::min<long long>(want, n));
        p.kv_blocks = 0;
        const int rows = kAppendThreads / units;
        const dim3 grid(static_cast<unsigned>((a.T + rows - 1) / rows), static_cast<unsigned>(p.groups));
        if (d == 64) fa_kv_append_kernel<64><<<grid, kAppendThreads, 0, stream>>>(p);
        else fa_kv_append_kernel<128><<<grid, kAppendThreads, 0, stream>>>(p);
        return cudaGetLastError();
    }
    const int n = std::max(p.H, 2 * p.H_kv);
    p.groups = static_cast<int>(std::max<long long>(std::min<long long>(want, n),
                                                    (2 * p.H_kv + kMaxGroupHeads - 1) / kMaxGroupHeads));
    // one warp per block where the sequences bring a token or a few each
    const int block = static_cast<long long>(a.T) <= 4ll * p.B ? 32 : 256;
    const int rows = block / units;
    const long long kv_blocks = (static_cast<long long>(a.T) >> p.shift) + 2ll * p.B;
    const long long q_blocks = p.H > 0 ? (a.T + rows - 1) / rows : 0;
    if (kv_blocks + q_blocks > 0x7fffffffll) return cudaErrorInvalidValue;
    p.kv_blocks = static_cast<int>(kv_blocks);
    const dim3 grid(static_cast<unsigned>(kv_blocks + q_blocks), static_cast<unsigned>(p.groups));
    if (d == 64) fa_kv_append_fp8_kernel<64><<<grid, block, 0, stream>>>(p);
    else fa_kv_append_fp8_kernel<128><<<grid, block, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace fa
