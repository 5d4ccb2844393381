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
// 8-bit kernel reads its rows twice, the second time from L1/L2).  For 21k tokens of
// prompts (32 query and 8 key heads of 128, 524 MB) the bf16 kernel takes 85 us, 6.2 TB/s
// or 91% of the copy bandwidth; into e4m3 pages (481 MB) 83 us, 5.8 TB/s: there the pages'
// blocks compute (scale, rotate, round) about as long as they load.  One token of 64
// sequences, inputs out of L2, takes 5.3 to 6.1 and 5.7 to 6.5 us, which is launch and the
// latency of four dependent loads (counts, length, page, row).  A thread owns 16 columns of
// a token (two 16-byte pieces that rotate into each other) and walks heads;
// what a token costs besides (its sequence, page, sines and cosines) is found once per
// block or held in registers over the heads.
#include <cuda_bf16.h>

#include <algorithm>
#include <climits>

#include "fa_internal.h"
#include "fa_paged.h"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr int kAppendThreads = 256;

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
    int groups;               // head groups (bf16: grid y)
    int q_groups;             // 8-bit: blocks per block of rows for the queries
    int lead, kv_blocks;      // 8-bit: blocks for the pages, in all and before the first for queries
    unsigned int* err;
};

__device__ __forceinline__ float lo_f(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float hi_f(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }

__device__ __forceinline__ int cu_of(const AppendParams& p, int b) {
    return p.cu ? p.cu[b] : b * (p.T / p.B);
}

// Reports token counts that do not ascend within [0, T], whether or not a row or page leads
// to their sequence.  For one block: its threads [from, kAppendThreads).
__device__ __forceinline__ void check_counts(const AppendParams& p, int from) {
    if (p.cu == nullptr) return;
    for (int b = static_cast<int>(threadIdx.x) - from; b < p.B; b += kAppendThreads - from) {
        const int c0 = p.cu[b], c1 = p.cu[b + 1];
        if (c0 < 0 || c1 < c0 || c1 > p.T) page_error(p.err);
    }
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

// (cos, sin) of position pos at a frequency given as a turn fraction.
__device__ __forceinline__ float2 turn_at(uint64_t freq, int pos) {
    // half turns in [-1, 1): the top 32 bits
    const uint64_t turns = freq * static_cast<uint64_t>(pos);
    float2 t;
    sincospif(static_cast<float>(static_cast<int32_t>(turns >> 32)) * 0x1p-31f, &t.y, &t.x);
    return t;
}

// A thread's eight (cos, sin), pairs [8 u, 8 u + 8) of its unit u, lie in shared memory (in
// registers they would halve the threads that an SM holds): pairs 2 i and 2 i + 1 as the
// float4 at turn[i * stride].
struct Turn {
    const float4* at;
    int stride;
};

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
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 cs = t.at[i * t.stride];  // cos, sin, cos, sin
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float c = k ? cs.z : cs.x, s = k ? cs.w : cs.y;
            const int j = 2 * i + k;
            if (p.interleaved) {
                const float e = x[2 * j], o = x[2 * j + 1];
                x[2 * j] = e * c - o * s;
                x[2 * j + 1] = o * c + e * s;
            } else {
                const float e = x[j], o = x[8 + j];
                x[j] = e * c - o * s;
                x[8 + j] = o * c + e * s;
            }
        }
    }
}

__device__ __forceinline__ uint4 pack8(const float* x) {
    return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}

constexpr int kHeadGroups = 4;  // of a block: threads that share a token's angles
constexpr int kMaxRot = 128;
constexpr long long kWantBlocks = 4 * 152;  // as many as are resident

// What the tokens of a block share.
template <int D>
struct RowShared {
    static constexpr int U = D / 16;                                   // units per row
    static constexpr int kTokens = kAppendThreads / (U * kHeadGroups);  // 8 at d = 128, 16 at 64
    float4 turn[kTokens][4][U];  // [token][pairs 2 i, 2 i + 1][unit]
    int pos[kTokens], page[kTokens];
    int live[kTokens];  // the token belongs to a sequence
};

// kTokens consecutive tokens, the heads [h0, h1) of the list [Q heads | K heads | V heads]
// in four groups of threads.  Used by both kernels (the 8-bit one sends its queries here).
template <int D>
__device__ __forceinline__ void append_rows(const AppendParams& p, RowShared<D>& sh, int t_first, int h0, int h1) {
    using S = RowShared<D>;
    constexpr int U = S::U, TOK = S::kTokens;
    const int tid = threadIdx.x, lane = tid & 31;
    const int u = tid % U, k = tid / U % TOK, hg = tid / (U * TOK);
    const int t = t_first + k;
    if (tid < 32) {
        // the sequence of each token: that of the first, and the next 32 sequences' starts
        const int b0 = last_not_above(p.B, t_first, [&](int i) { return static_cast<long long>(cu_of(p, i)); });
        const int cuv = b0 + 1 + lane < p.B ? cu_of(p, b0 + 1 + lane) : 0x7fffffff;
        int b = b0;
#pragma unroll
        for (int i = 0; i < TOK; ++i) {
            const int n = __popc(__ballot_sync(0xffffffffu, cuv <= t_first + i));
            if (lane == i) b += n;
        }
        if (lane < TOK) {
            const int tt = t_first + lane;
            if (b == b0 + 32)  // (32 sequences begin at or before the token: go on one by one)
                while (b + 1 < p.B && cu_of(p, b + 1) <= tt) ++b;
            const int c0 = cu_of(p, b), c1 = cu_of(p, b + 1), past = p.lens[b];
            const long long pos = static_cast<long long>(past) + (tt - c0);
            const bool live = tt < p.T && tt >= c0 && tt < c1;
            int pg = -1;
            if (live && h1 > p.H) {
                if (past >= 0 && c0 >= 0 && c1 <= p.T)
                    pg = page_of(p.table + static_cast<long long>(b) * p.max_pages, p.max_pages, p.num_pages, p.shift, pos);
                if (pg < 0) page_error(p.err);
            }
            sh.pos[lane] = static_cast<int>(pos);
            sh.page[lane] = pg;
            sh.live[lane] = live;
        }
    } else if (t_first == 0 && h0 == 0) {
        check_counts(p, 32);  // (while the first warp looks for the tokens' places)
    }
    __syncthreads();
    const int half = p.rot / 2;
    if (half > 0 && h0 < p.H + p.H_kv) {
        // freq ascends with idx % half, so neighbouring threads read neighbouring entries
        for (int idx = tid; idx < TOK * half; idx += kAppendThreads) {
            const int i = idx / half, c = idx - i * half;
            reinterpret_cast<float2*>(&sh.turn[i][c % 8 / 2][c / 8])[c & 1] =
                turn_at(turn_fraction(p.inv_freq[c]), sh.pos[i]);
        }
        __syncthreads();
    }
    if (!sh.live[k]) return;  // a row behind the last sequence: left as it is
    const int pg = sh.page[k], off = sh.pos[k] & ((1 << p.shift) - 1);
    const bool turns = u < p.rot / 16;
    const Turn tr{&sh.turn[k][0][u], U};
    int a, c;
    pieces(p, u, a, c);
    constexpr int kBatch = 4;  // heads whose loads are in flight together
    const __nv_bfloat16* qrow = p.q + t * p.q_st;
    const __nv_bfloat16* krow = p.k + t * p.k_st - p.H * p.k_sh;
    const __nv_bfloat16* vrow = p.v + t * p.v_st - (p.H + p.H_kv) * p.v_sh;
    for (int hb = h0 + hg; hb < h1; hb += kBatch * kHeadGroups) {
        uint4 wa[kBatch], wb[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int h = hb + i * kHeadGroups;
            if (h < h1) {
                const __nv_bfloat16* src = h < p.H            ? qrow + h * p.q_sh
                                           : h < p.H + p.H_kv ? krow + h * p.k_sh
                                                              : vrow + h * p.v_sh;
                wa[i] = reinterpret_cast<const uint4*>(src)[a];
                wb[i] = reinterpret_cast<const uint4*>(src)[c];
            }
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int h = hb + i * kHeadGroups;
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

// Both kernels are launched as dependents of the kernel before them, so that their start-up
// overlaps its end; every thread waits for it before it reads anything (by plain loads: the
// inputs may still be written while this grid is being set up).  One token of 64 sequences,
// calls in a row launched one by one (inputs in L2): 6.2 us without and 3.7 with, in 8 bits
// 8.2 and 5.6; from a captured graph, where a launch costs little, 3.7 and 3.9, 5.2 and 5.1.
template <int D>
__global__ void __launch_bounds__(kAppendThreads, 4) fa_kv_append_kernel(const AppendParams p) {
    __shared__ RowShared<D> sh;
    griddep_launch_dependents();
    griddep_wait();
    const int n = p.H + 2 * p.H_kv;
    const int per = (n + p.groups - 1) / p.groups;
    const int h0 = static_cast<int>(blockIdx.y) * per;
    append_rows<D>(p, sh, static_cast<int>(blockIdx.x) * RowShared<D>::kTokens, h0, min(n, h0 + per));
}

// The largest magnitude of 16 bf16 values, two at a time (NaN is passed over: m starts at 0).
__device__ __forceinline__ float amax16(const uint4& a, const uint4& b) {
    const uint32_t x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) asm("max.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(x[i] & 0x7fff7fffu));
    return fmaxf(lo_f(m), hi_f(m));
}

// Four e4m3 codes rescaled by r (rounded to nearest even).
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float r) {
    uint32_t lo, hi;
    widen_e4m3x4(w, lo, hi);
    const float2 a = unpack_f16(lo), b = unpack_f16(hi);
    return pack_e4m3x4(a.x * r, a.y * r, b.x * r, b.y * r);
}

constexpr int kGroupCost = 3;
constexpr int kMaxGroupHeads = 16;  // heads (of the list [K | V]) that one team walks

struct PageShared {
    float4 turn[4][kAppendThreads];  // each thread's own
    uint64_t freq[kMaxRot / 2];
    uint32_t amax[kAppendThreads / 32][kMaxGroupHeads];
    float scale[kAppendThreads / 32][kMaxGroupHeads], inv[kAppendThreads / 32][kMaxGroupHeads];
};

// One team of threads (a block, or with few new tokens per sequence a warp) per (sequence,
// page reached, head group): it alone writes that page's heads, so the scale needs no
// communication.  Two passes over the page's new rows, the second from L1/L2: the largest
// magnitude per head, then rotate, scale, round and store.
template <int D, int TEAM>
__global__ void __launch_bounds__(kAppendThreads, 4) fa_kv_append_fp8_kernel(const AppendParams p) {
    constexpr int U = D / 16, ROWS = TEAM / U, TEAMS = kAppendThreads / TEAM;
    __shared__ union {
        PageShared page;
        RowShared<D> row;
    } sh;
    griddep_launch_dependents();
    griddep_wait();
    // The blocks for the pages compute more and take longer, those for the queries wait for
    // memory: one of each in turn while there are pages, so that both share the SMs, with
    // the pages first where they are more (lead).
    int bx = static_cast<int>(blockIdx.x);
    const int turn = bx - p.lead, pairs = p.kv_blocks - p.lead;
    if (turn < 0 || (turn < 2 * pairs && (turn & 1) == 0)) {
        bx = turn < 0 ? bx : p.lead + turn / 2;
    } else {
        bx = turn < 2 * pairs ? turn / 2 : turn - pairs;
        const int rb = bx / p.q_groups, per = (p.H + p.q_groups - 1) / p.q_groups, h0 = (bx - rb * p.q_groups) * per;
        if (h0 < p.H) append_rows<D>(p, sh.row, rb * RowShared<D>::kTokens, h0, min(p.H, h0 + per));
        else if (p.H == 0) check_counts(p, 0);  // (the one block that a call without queries has here)
        return;
    }
    const int group = bx % p.groups;
    bx /= p.groups;
    const int team = static_cast<int>(threadIdx.x) / TEAM, tid = static_cast<int>(threadIdx.x) % TEAM;
    const auto sync = [] {
        if constexpr (TEAM == 32) __syncwarp();
        else __syncthreads();
    };
    if (p.rot > 0) {
        for (int i = threadIdx.x; i < p.rot / 2; i += kAppendThreads) sh.page.freq[i] = turn_fraction(p.inv_freq[i]);
        __syncthreads();
    }
    uint32_t* amax_s = sh.page.amax[team];
    float* scale_s = sh.page.scale[team];
    float* inv_s = sh.page.inv[team];
    const int n_list = 2 * p.H_kv;
    const int per = (n_list + p.groups - 1) / p.groups;
    const int h0 = group * per, h1 = min(n_list, h0 + per);
    if (h0 >= h1) return;
    // this team's sequence and page
    const int unit = bx * TEAMS + team;
    const int b = last_not_above(p.B, unit, [&](int i) { return first_unit(cu_of(p, i), i, p.shift); });
    const int c0 = cu_of(p, b), c1 = cu_of(p, b + 1), past = p.lens[b];
    const int i = static_cast<int>(unit - first_unit(c0, b, p.shift));
    // (nothing new, counts that check_counts reports, or rows before the first sequence's)
    if (c1 <= c0 || c0 < 0 || c1 > p.T || i < 0 || past < 0) {
        if (past < 0 && c1 > c0 && tid == 0) page_error(p.err);
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
        if (tid == 0) page_error(p.err);
        return;
    }
    const int u = tid % U, tr = tid / U;
    int a, c;
    pieces(p, u, a, c);
    for (int h = tid; h < h1 - h0; h += TEAM) amax_s[h] = 0u;
    sync();
    const auto row_of = [&](int h, int r) {
        const long long t = t0 + (r - r0);
        return reinterpret_cast<const uint4*>(h < p.H_kv ? p.k + t * p.k_st + h * p.k_sh
                                                         : p.v + t * p.v_st + (h - p.H_kv) * p.v_sh);
    };
    // this thread's items: (row, head), rows r0 + tr, + ROWS, ... below r1
    const int n_rows = tr < r1 - r0 ? (r1 - r0 - tr + ROWS - 1) / ROWS : 0, nh = h1 - h0;
    // 1. the largest magnitude of each head's new rows; four items' loads in flight
    const int most = (r1 - r0 + ROWS - 1) / ROWS * nh;  // (the same for the whole team)
    constexpr int kBatch = 4;
    int rr = 0, hh = 0;  // row and head of the item to load next (counted: a division per item is dear)
    for (int ib = 0; ib < most; ib += kBatch) {
        uint4 wa[kBatch], wb[kBatch];
        int head[kBatch];
        bool mine[kBatch];  // (not past this thread's rows)
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            head[k] = hh;
            mine[k] = rr < n_rows;
            if (mine[k]) {
                const uint4* src = row_of(h0 + hh, r0 + tr + rr * ROWS);
                wa[k] = src[a];
                wb[k] = src[c];
            }
            const bool wrap = hh + 1 == nh;
            hh = wrap ? 0 : hh + 1;
            rr += wrap;
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const float m = mine[k] ? amax16(wa[k], wb[k]) : 0.f;
            // (non-negative: the bits keep the order)
            const uint32_t mw = __reduce_max_sync(0xffffffffu, __float_as_uint(m));
            if ((threadIdx.x & 31) == 0 && mw != 0u) atomicMax(&amax_s[head[k]], mw);
        }
    }
    sync();
    // 2. the scales; a page begun earlier keeps the larger one, its codes rescaled
    const auto place = [&](int h, bool is_k) { return static_cast<long long>(pg) * p.H_kv + (is_k ? h : h - p.H_kv); };
    for (int h = h0 + tid; h < h1; h += TEAM) {
        const bool is_k = h < p.H_kv;
        float bound = __uint_as_float(amax_s[h - h0]);
        if (is_k && p.rot > 0) bound *= 1.5f;
        const float need = __uint_as_float(static_cast<uint32_t>(page_scale_exp(__float_as_uint(bound)) + 127) << 23);
        float* scale = (is_k ? p.k_scale : p.v_scale) + place(h, is_k);
        const float old = r0 > 0 ? *scale : need, s = fmaxf(old, need);
        scale_s[h - h0] = s > old ? old / s : 1.f;  // what held codes are multiplied by
        inv_s[h - h0] = 1.f / s;                    // (exact for a power of two)
        if (r0 == 0 || s != old) *scale = s;
    }
    sync();
    if (r0 > 0) {
        for (int h = h0; h < h1; ++h) {
            const float ratio = scale_s[h - h0];
            if (ratio == 1.f) continue;
            const bool is_k = h < p.H_kv;
            uint4* codes = reinterpret_cast<uint4*>((is_k ? p.kc : p.vc) + ((place(h, is_k) << p.shift) * D));
            for (int e = tid; e < r0 * (D / 16); e += TEAM) {
                uint4 w = codes[e];
                w.x = rescale4(w.x, ratio);
                w.y = rescale4(w.y, ratio);
                w.z = rescale4(w.z, ratio);
                w.w = rescale4(w.w, ratio);
                codes[e] = w;
            }
        }
    }
    // 3. rotate, scale, round, store; the next item's loads in flight
    const bool turns = u < p.rot / 16;
    const Turn t{&sh.page.turn[0][threadIdx.x], kAppendThreads};
    const int n_items = n_rows * nh;
    uint4 wa, wb;
    if (n_items > 0) {
        const uint4* src = row_of(h0, r0 + tr);
        wa = src[a];
        wb = src[c];
    }
    int h = h0, r = r0 + tr;
    for (int it = 0; it < n_items; ++it) {
        const uint4 xa = wa, xb = wb;
        const int hn = h + 1 < h1 ? h + 1 : h0, rn = h + 1 < h1 ? r : r + ROWS;
        if (it + 1 < n_items) {
            const uint4* src = row_of(hn, rn);
            wa = src[a];
            wb = src[c];
        }
        if (turns && h == h0 && h0 < p.H_kv) {  // a new row
#pragma unroll
            for (int e = 0; e < 8; ++e)
                reinterpret_cast<float2*>(&sh.page.turn[e / 2][threadIdx.x])[e & 1] =
                    turn_at(sh.page.freq[8 * u + e], static_cast<int>(page0 + r));
        }
        const bool is_k = h < p.H_kv;
        float x[16];
        if (turns && is_k) {
            rotate(p, xa, xb, t, x);
        } else {
            const uint32_t w[8] = {xa.x, xa.y, xa.z, xa.w, xb.x, xb.y, xb.z, xb.w};
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
        uint8_t* dst = (is_k ? p.kc : p.vc) + ((place(h, is_k) << p.shift) + r) * D;
        reinterpret_cast<uint2*>(dst)[a] = make_uint2(o[0], o[1]);
        reinterpret_cast<uint2*>(dst)[c] = make_uint2(o[2], o[3]);
        h = hn;
        r = rn;
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
    const int d = a.cache.d;
    // Heads are cut into groups (grid y) only as far as the tokens alone do not fill the
    // machine: each group finds its tokens' pages and angles again.
    const int tokens = d == 64 ? RowShared<64>::kTokens : RowShared<128>::kTokens;
    const long long row_blocks = (static_cast<long long>(a.T) + tokens - 1) / tokens;
    if (a.cache.k_scale == nullptr) {
        const int n = p.H + 2 * p.H_kv;
        p.groups = static_cast<int>(std::max(1ll, std::min<long long>((kWantBlocks + row_blocks - 1) / row_blocks,
                                                                      (n + kHeadGroups - 1) / kHeadGroups)));
        p.q_groups = p.lead = p.kv_blocks = 0;
        const dim3 grid(static_cast<unsigned>(row_blocks), static_cast<unsigned>(p.groups));
        return launch_dependent(d == 64 ? fa_kv_append_kernel<64> : fa_kv_append_kernel<128>, grid, dim3(kAppendThreads), 0,
                                stream, p);
    }
    // a warp per page where the sequences bring a token or a few each, else a block (32
    // sequences of 4 tokens: 5.8 us by warps, 6.6 by blocks; of 8: 7.7 and 6.9)
    const bool warps = static_cast<long long>(a.T) <= 4ll * p.B;
    const long long units = (static_cast<long long>(a.T) >> p.shift) + 2ll * p.B;
    long long kv_blocks = warps ? (units + kAppendThreads / 32 - 1) / (kAppendThreads / 32) : units;
    const int n = 2 * p.H_kv;
    // Heads per group: a block takes as long as its heads and kGroupCost more (angles, scales,
    // barriers); the least of the resident blocks' mean load and one block's length together
    // (21k tokens, 16 heads of K and V: four groups 40 us, two, a little over one round, 44).
    long long best = LLONG_MAX;
    for (int per = std::min(n, kMaxGroupHeads); per >= 1; --per) {
        const long long groups = (n + per - 1) / per, cost = (kv_blocks * groups + kWantBlocks) * (per + kGroupCost);
        if (cost < best) {
            best = cost;
            p.groups = static_cast<int>(groups);
        }
    }
    p.q_groups = static_cast<int>(std::max(1ll, std::min<long long>((kWantBlocks + row_blocks - 1) / row_blocks,
                                                                    (p.H + kHeadGroups - 1) / kHeadGroups)));
    const long long q_blocks = p.H > 0 ? row_blocks * p.q_groups : 1;
    kv_blocks *= p.groups;
    if (kv_blocks + q_blocks > 0x3fffffffll) return cudaErrorInvalidValue;
    p.kv_blocks = static_cast<int>(kv_blocks);
    p.lead = static_cast<int>(std::max(0ll, kv_blocks - q_blocks));
    const dim3 grid(static_cast<unsigned>(kv_blocks + q_blocks));
    return launch_dependent(d == 64 ? (warps ? fa_kv_append_fp8_kernel<64, 32> : fa_kv_append_fp8_kernel<64, 256>)
                                    : (warps ? fa_kv_append_fp8_kernel<128, 32> : fa_kv_append_fp8_kernel<128, 256>),
                            grid, dim3(kAppendThreads), 0, stream, p);
}

}  // namespace fa
