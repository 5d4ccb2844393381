// Kernels of a decode step's attention over a paged key/value cache (bf16, or e4m3 with a scale
// per page and head), for sm_103a.
//
// Mathematics: the Nq <= 8 query rows of a sequence are its last positions; row i of
// len keys sees key j iff j <= len - Nq + i and, with a window, j > len - Nq + i - window
// or j < sinks.  O = sum_j softmax_j(tau q.k_j) v_j by the online recurrence of
// fa_decode.cu, each H / H_kv query heads reading one key head.  A step reads each
// visible K and V once, so HBM bounds it.
//
// Design:
//   - Work is cut evenly whatever the lengths: the 16-key tiles of all (sequence, key
//     head) segments form one list, and every resident warp takes an equal contiguous
//     share of it, found from a prefix sum of the lengths, which stay on the device.  A
//     segment that several shares cut leaves one partial result per piece (normalised,
//     with its log-sum), which the combine kernel adds.  Shares are per warp, not per
//     CTA: warps share nothing and never wait for one another, and a warp meets fewer
//     segment borders (1 + segments / warps), where its pipeline drains.
//   - A warp holds 8 or 16 query rows.  With more rows, 2 or 4 warps of a CTA take the
//     same share for 16 rows each and read the same keys at about the same time, all but
//     one of them from L2.
//   - A warp streams its tiles through its own ring of shared memory with 16-byte
//     cp.async, written in the XOR order that makes the 16-byte fragment loads below
//     free of bank conflicts.
//   - Both products run on warp matrix instructions with the keys (and the columns of
//     V) as the 16-row operand and 8 query rows as the narrow one: S^T = K Q^T and
//     O^T = V^T P^T, so grouped heads fill a tile with little padding.  At 16 query rows
//     a step's 512 bytes per bf16 key feed 8192 multiply-adds: the tensor cores idle on
//     the memory either way, and a 128-row tcgen05 tile would be 87-94% padding.
//   - The order of the summed index is free as long as both operands agree: a thread
//     takes the 16 bytes of a key row that it can load at once, so K needs no transposing
//     load.  V^T pairs neighbouring keys with a byte permute; P^T changes from the
//     accumulator's layout to the operand's with movmatrix.
//   - Weights are taken relative to a running reference, which moves to the max (8-bit pages:
//     2^14 below it) only when some weight passes 2^8 (2^15; one vote per tile); row sums stay
//     per thread until the segment ends.
//   - Short tables (kWholeTiles) take a block, or a cluster of blocks, per segment instead:
//     its warps take the tiles in turn and join their sums in shared memory (a cluster's
//     blocks in one another's), and no second kernel runs.
//   - e4m3 keys and values are widened to fp16, which holds every code exactly; queries
//     enter as fp16 with a power of two per row, so bf16's 8 bits stay exact down to
//     2^-31 of the row's largest.  The page's K scale multiplies the scores in fp32; its
//     V scale enters the weights, which keep a reference of their own (log2 P + log2 scale).
//   - P is rounded for the second product, as O is in the end; statistics, scores and sums
//     stay in fp32.  bf16: relative error at most 2^-8 per weight.  8-bit pages, fp16: 2^-11
//     for weights (times their page's scale) down to 2^-28 of the largest of these;
//     below, fp16's subnormals, 2^-39 of the largest in all, so beside a key of value zero that
//     outweighs them by e^19 the other keys' weights still have 11 bits.
//   - Rows past a sequence's end are never read: the copy fills them with zeros, so what
//     a page holds there, NaN included, does not matter; the same goes for keys hidden
//     from all of the step's rows.
//
// Measured (d = 128, pages of 64): 48 sequences of up to 16384 keys, 8 key heads of 4
// query heads, bf16, 2.0 GB: 288 to 292 us, 6.9 TB/s, 1.02 of the copy bandwidth (which reads
// and writes; 86% of the DRAM's cycles); 96 of up to 12000, e4m3, 1.24 GB: 193 us, 6.4 TB/s, 0.95;
// 8 of up to 32768, 16 heads, e4m3, 0.53 GB: 86 us, 6.1 TB/s, 0.90.  A split call's fixed
// part is about 10 us: launch, the lengths' scan (2 us), table and first tiles (3 to 6 us,
// all rings filling at once), the slowest warp's tail, the combine kernel (3 us).  With 16
// or more query rows per key head the instructions per tile weigh as much as its bytes
// (e4m3, 32 rows: 109 us for 335 MB).
//
// MOD: scores capped by a tanh, or with a bias by distance (fa_score.cuh): applied to a
// tile's scores in fp32 before the running reference is taken off.  The kernels without it are
// those of fa_paged.cu, with it of fa_paged_score.cu.
#pragma once

#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>

#include "fa_paged.h"
#include "fa_score.cuh"

namespace fa {
namespace {

constexpr int kSms = 152;  // of a GB300
constexpr int kThreads = 32 * kPagedWarps;
constexpr float kLn2 = 0.69314718055994531f;
constexpr float kLog2e = 1.44269504088896341f;
// How far, in log2 units, scores may pass the running reference before that moves, and how
// far below the largest score it then lies: weights stay <= 2^kGrow.  8-bit pages hold
// weights in fp16, whose 11 bits reach as far down as they can when the largest lie at the
// top of its range.  (kLift8 14 and kGrow8 15 against 0 and 8: 16 sequences of 16384 keys, 32
// rows per key head 163.2 and 162.9 us; 8 of up to 32768 and 96 of up to 12000, alike.)
constexpr float kGrow = 8.0f, kLift8 = 14.0f, kGrow8 = 15.0f;
enum : uint32_t { kSitePagedSmem = 51 };

// Ring slots per warp and CTAs per SM: 130 to 200 KB of slots per SM, and as many warps as
// the registers allow, since a tile's chain of dependent instructions takes a warp as long
// as its bytes take to come (12 warps of two slots against 8 of three: 96 sequences of up to
// 12000 e4m3 keys 200 -> 193 us, 48 of up to 16384 bf16 keys 296 -> 291; 16 query rows at
// d = 128 do not fit 168 registers and keep 8: spilled, 54 -> 56 us and e4m3 41 -> 52).
template <int D, int NT, bool F8>
struct PagedLayout {
    static constexpr int kRow = D * (F8 ? 1 : 2);       // bytes of a key row
    static constexpr int kTile = kPagedTile * kRow;     // K or V of one tile
    static constexpr int TP = kTile == 4096 ? 1 : 2;    // tiles per slot and loop iteration
    static constexpr int kSlot = 2 * TP * kTile;
    static constexpr int kCtas = kSlot == 8192 ? (NT == 1 || D == 64 ? 3 : 2) : NT == 1 ? 4 : 3;
    static constexpr int kStages = kSlot == 8192 ? (kCtas == 3 ? 2 : 3) : NT == 1 ? 3 : 4;
    static constexpr int kWarpRing = kStages * kSlot;
};

struct PagedParams {
    const __nv_bfloat16* Q;
    const uint8_t* K;
    const uint8_t* V;
    const float* k_scale;
    const float* v_scale;
    const int* table;
    const int* lens;
    __nv_bfloat16* O;
    float* LSE;
    int2* seg;       // [segments]: a segment's first share and number of pieces
    float* part_o;   // [2 per warp][8 NT][D]
    float* part_l;   // [2 per warp][8 NT], log2 of the piece's sum
    long long q_sb, q_sh, q_sn, o_sb, o_sh, o_sn;
    int B, H, H_kv, G, Nq, num_pages, max_pages, shift, window, sinks;
    int rwarps;        // warps that share a share, 8 NT query rows each (1, 2 or 4)
    int shares;        // at most
    int cluster_log2;  // WW = 8: of the blocks that share a segment
    int rgroups;       // segments per (sequence, key head): rwarps * 8 NT query rows each
    float scale_log2;  // tau * log2(e)
    unsigned int* err;
    // MOD
    float cap_log2, cap_inv;  // cap * log2(e) (0: none), and 1 / that
    const float* slopes;
    const void* bias;
    const int* buckets;
    int bias_f32, num_buckets, far;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
    return v;
}

// d += A B: A 16 x 16 (rows keys or V columns), B 16 x 8 (query rows), fp32 accumulation.
template <bool F16>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    if constexpr (F16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 8 x 8 transpose of 16-bit values across the warp.
__device__ __forceinline__ uint32_t movmatrix(uint32_t x) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

__device__ __forceinline__ float lg2(float x) {  // log2, -inf at 0
    float y;
    asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A tile in shared memory: row r's 16-byte chunks in an XOR order, so that the fragment
// loads touch all 32 banks once.  K: eight threads read four chunks of two neighbouring
// rows; V: two chunks of every other row of eight.  Rows of 64 bytes lie two to a line.
//   rows >= 128 bytes:  K  r ROW + ((c ^ 4 (r & 1)) << 4)
//                       V  r ROW + ((c ^ 2 ((r >> 1) & 3)) << 4)
//   rows of 64 bytes:   K  64 r + (c << 4)
//                       V  128 (r >> 1) + 64 ((r ^ (r >> 2)) & 1) + ((c ^ 2 ((r >> 1) & 1)) << 4)
// A copy instruction j of 32 lanes fills 512 bytes, chunk idx = 32 j + lane (row idx / CH,
// chunk idx % CH).  Only the XOR terms that change with j are left for the loop; the
// lane's part is computed once.
template <int ROW>
struct Swizzle {
    static constexpr int CH = ROW / 16;
    // destination of copy j: 512 j + k_dst(lane), 512 j + (v_dst(lane) ^ v_dst_x(j))
    static __device__ __forceinline__ uint32_t k_dst(int lane) {
        const int r = lane / CH, c = lane % CH;
        return ROW >= 128 ? r * ROW + ((c ^ ((r & 1) << 2)) << 4) : lane * 16;
    }
    static __device__ __forceinline__ uint32_t v_dst(int lane) {
        const int r = lane / CH, c = lane % CH;
        return ROW >= 128 ? r * ROW + ((c ^ (((r >> 1) & 3) << 1)) << 4)
                          : ((r >> 1) << 7) + (((r ^ (r >> 2)) & 1) << 6) + ((c ^ (((r >> 1) & 1) << 1)) << 4);
    }
    static constexpr uint32_t v_dst_x(int j) { return ROW == 256 ? (j & 3) << 5 : ROW == 128 ? (j & 1) << 6 : 0; }
    // K fragment: chunk t4 + 4 c of row g at k_src ^ (c << 6), row g + 8 8 ROW further
    static __device__ __forceinline__ uint32_t k_src(int g, int t4) {
        return g * ROW + (t4 << 4) + (ROW >= 128 ? (g & 1) << 6 : 0);
    }
    // V fragment of rows 2 t4, 2 t4 + 1 (at v_row1) and these + 8 (8 ROW further)
    static __device__ __forceinline__ uint32_t v_src(int g, int t4) {
        return ROW >= 128 ? 2 * t4 * ROW + ((g ^ (t4 << 1)) << 4)
                          : (t4 << 7) + ((t4 >> 1) << 6) + (((g >> 1) ^ ((t4 & 1) << 1)) << 4) + ((g & 1) << 3);
    }
    static __device__ __forceinline__ uint32_t v_row1(uint32_t a) { return ROW >= 128 ? a + ROW : a ^ 64; }
};

// Distributed shared memory: the address of another block's copy of a place in this one's,
// loads from there, and a barrier over the cluster.
__device__ __forceinline__ uint32_t map_block(uint32_t a, int block) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(block));
    return r;
}
__device__ __forceinline__ float ld_cluster(uint32_t a) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t a) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;" ::: "memory");
}

// max over the lanes that share lane % 4
__device__ __forceinline__ float max_over_g(float x) {
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}
__device__ __forceinline__ float sum_over_g(float x) {
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

__device__ __forceinline__ int clamp_len(const PagedParams& p, int b) {
    const int len = p.lens[b];
    const long long cap = static_cast<long long>(p.max_pages) << p.shift;
    if (len < 0 || len > cap) {
        page_error(p.err);
        return len < 0 ? 0 : static_cast<int>(cap);
    }
    return len;
}

template <int WARPS, bool MOD>
struct PagedShared {
    // per ring slot: first key of the tile (a bad page: past every row); 8-bit: the page's scales
    struct __align__(16) Slot {
        int key0;
        float ks, vs, pad;
    } slot[WARPS][4][2];  // [warp][ring slot][tile]
    int scan[WARPS];
    int at_b[WARPS], at_before[WARPS];  // a share's first sequence, tiles of those before it
    float m[WARPS][16], l[WARPS][16];   // WHOLE: each warp's reference and sum
    float lse[WARPS > kPagedWarps ? 64 : 1];  // of a cluster's block: log2 of its rows' sums
    short bucket[MOD ? kScoreMaxFar + 1 : 1];  // a bias's bucket at distances 0 .. far (-1: none)
};
template <int D, int NT, bool F8, int WARPS, bool MOD>
constexpr int kPagedBytes = WARPS * PagedLayout<D, NT, F8>::kWarpRing + static_cast<int>(sizeof(PagedShared<WARPS, MOD>));

// WW > 0: a block of WW warps takes one segment, its warps the tiles in turn, and joins their
// results in shared memory: no partial results, no second kernel.  For short segments.
template <int D, int NT, bool F8, int WW, bool MOD>
__global__ void __launch_bounds__(WW > 0 ? 32 * WW : kThreads, WW > kPagedWarps ? 1 : PagedLayout<D, NT, F8>::kCtas)
fa_paged_kernel(const PagedParams p) {
    constexpr bool WHOLE = WW > 0;
    constexpr int WARPS = WHOLE ? WW : kPagedWarps;
    using L = PagedLayout<D, NT, F8>;
    constexpr int ROW = L::kRow, CH = ROW / 16, S = L::kStages, TP = L::TP;
    using W = Swizzle<ROW>;
    constexpr int R = 8 * NT;           // query rows of a segment
    constexpr int MT = D / 16;          // 16-column tiles of V^T
    constexpr int KS = D / 16;          // 16-element steps of q.k
    constexpr int kChunksK = D / (F8 ? 64 : 32);  // 16-byte pieces of a key row per thread
    constexpr float kSlack = F8 ? kGrow8 : kGrow, kLift = F8 ? kLift8 : 0.f;
    extern __shared__ __align__(1024) uint8_t smem[];
    using Shared = PagedShared<WARPS, MOD>;
    Shared& sh = *reinterpret_cast<Shared*>(smem + WARPS * L::kWarpRing);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
    // Launched as a dependent of the kernel before it: its start-up overlaps that kernel's
    // end.  Every thread waits here before it reads anything (by plain loads: the inputs may
    // still be written until then), so this grid ends after that one.
    griddep_launch_dependents();
    griddep_wait();
    const uint32_t ring = smem_addr(smem) + warp * L::kWarpRing;
    if ((smem_addr(smem) & 255u) != 0u) {  // (the XOR orders count on tiles at multiples of 256 bytes)
        if (tid == 0) atomicCAS(p.err, 0u, 1u | (kSitePagedSmem << 8));
        return;
    }
    // (the buckets' map once per block: two loads in a row for each near tile took as long as several tiles)
    [[maybe_unused]] const auto bias_at = [&](int h, int dist) {
        const int e = sh.bucket[MOD ? max(0, min(p.far, dist)) : 0];
        const long long at = static_cast<long long>(max(e, 0)) * p.H + h;  // (a load for all, no branch)
        const float y = p.bias_f32 ? static_cast<const float*>(p.bias)[at]
                                   : __uint_as_float(static_cast<uint32_t>(static_cast<const unsigned short*>(p.bias)[at]) << 16);
        return e < 0 ? 0.f : kLog2e * y;
    };
    if constexpr (MOD) {
        if (p.bias) {
            for (int i = tid; i <= p.far; i += static_cast<int>(blockDim.x)) {
                const int e = p.buckets[p.far + i];
                sh.bucket[i] = static_cast<short>(static_cast<unsigned>(e) < static_cast<unsigned>(p.num_buckets) ? e : -1);
            }
            __syncthreads();
        }
    }
    const uint32_t k_dst = W::k_dst(lane), v_dst = W::v_dst(lane), k_src = W::k_src(g, t4), v_src = W::v_src(g, t4);
    const int segs_per_b = p.H_kv * p.rgroups;
    // what this warp works on: its share of the tiles [x, x_end), from sequence b on, or (WHOLE)
    // every iw-th tile of one segment, from `turn` on; rows of row warp rw
    uint32_t share = 0, x = 0, x_end = 0, b_first = 0;
    int b = 0, rw = 0, turn = 0, iw = 1;
    [[maybe_unused]] int seg = static_cast<int>(blockIdx.x), cn = 1;  // WHOLE: the segment, and its blocks
    Shares cut(1u, 1u);
    if constexpr (WHOLE) {
        if constexpr (WW > kPagedWarps) {
            cn = 1 << p.cluster_log2;
            seg = static_cast<int>(blockIdx.x) >> p.cluster_log2;
        }
        b = seg / segs_per_b;
        iw = WARPS / p.rwarps;
        rw = warp % p.rwarps;
        turn = warp / p.rwarps + (static_cast<int>(blockIdx.x) - seg * cn) * iw;
        iw *= cn;
    } else {
        // ---- this warp's share of the tiles ----
        const int per = (p.B + kThreads - 1) / kThreads;
        int mine = 0;
        for (int i = 0; i < per; ++i) {
            const int b = tid * per + i;
            if (b < p.B) mine += paged_tiles(paged_range(clamp_len(p, b), p.Nq, p.window, p.sinks));
        }
        int incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        if (lane == 31) sh.scan[warp] = incl;
        __syncthreads();
        int total_b = 0, before = incl - mine;
#pragma unroll
        for (int w = 0; w < kPagedWarps; ++w) {
            if (w < warp) before += sh.scan[w];
            total_b += sh.scan[w];
        }
        const uint32_t total = static_cast<uint32_t>(total_b) * segs_per_b, segs = static_cast<uint32_t>(p.B) * segs_per_b;
        const int per_cta = kPagedWarps / p.rwarps;  // shares of a CTA
        // (with few tiles the last warps have none)
        const uint32_t shares = share_count(gridDim.x * per_cta, total, segs);
        cut = Shares(total, shares);
        for (int w = 0; w < per_cta; ++w) {
            const uint32_t c = blockIdx.x * per_cta + w;
            if (c >= shares) break;
            // the whole sequences' tiles before the share's first, rounded down
            const int xs = static_cast<int>(cut.start(c) / segs_per_b);
            if (xs >= before && xs < before + mine) {
                int b = tid * per, at = before;
                for (;; ++b) {
                    const int n = paged_tiles(paged_range(clamp_len(p, b), p.Nq, p.window, p.sinks));
                    if (xs < at + n) break;
                    at += n;
                }
                sh.at_b[w] = b;
                sh.at_before[w] = at;
            }
        }
        __syncthreads();
        const int wshare = warp / p.rwarps;
        rw = warp - wshare * p.rwarps;
        share = blockIdx.x * per_cta + wshare;
        if (share >= shares) return;  // (from here on the warps go their own ways)
        x = cut.start(share);
        x_end = cut.start(share + 1);
        b = sh.at_b[wshare];
        b_first = static_cast<uint32_t>(sh.at_before[wshare]) * segs_per_b;  // first tile of sequence b
    }
    PagedRange rg = paged_range(clamp_len(p, b), p.Nq, p.window, p.sinks);
    uint32_t tiles = paged_tiles(rg);

    while (true) {
        // ---- one piece: tiles [u0, u1) of segment (b, hk, rb group) ----
        const int in_b = WHOLE ? seg - b * segs_per_b : static_cast<int>((x - b_first) / tiles);
        [[maybe_unused]] const uint32_t seg_first = b_first + in_b * tiles;
        const int hk = in_b / p.rgroups;
        const int u0 = WHOLE ? 0 : static_cast<int>(x - seg_first);
        const int u1 = WHOLE ? rg.n : static_cast<int>(min(tiles, x_end - seg_first));
        [[maybe_unused]] const auto next = [&]() {  // on to the next segment; false at the share's end
            x = seg_first + u1;
            if (x >= x_end) return false;
            if (x >= b_first + tiles * segs_per_b) {
                b_first += tiles * segs_per_b;
                ++b;
                rg = paged_range(clamp_len(p, b), p.Nq, p.window, p.sinks);
                tiles = paged_tiles(rg);
            }
            return true;
        };
        if (!WHOLE && u0 > 0 && u0 >= rg.n) {  // only a segment's empty tiles
            if (!next()) return;
            continue;
        }
        const int len = rg.len;
        // row r of this warp: head hk G + (row0 + r) / Nq, position (row0 + r) % Nq
        const int row0 = ((in_b - hk * p.rgroups) * p.rwarps + rw) * R;
        const int rows = min(R, p.G * p.Nq - row0);  // (none for the last warps of a share)
        // this warp's tiles: entries entry(0) .. entry(nv - 1) of the sequence's list
        const int nv = rows <= 0 ? 0 : WHOLE ? max(0, (rg.n - turn + iw - 1) / iw) : max(0, min(u1, rg.n) - u0);
        const auto entry = [&](int i) { return WHOLE ? turn + i * iw : u0 + i; };
        const int* table = p.table + static_cast<long long>(b) * p.max_pages;

        // pages of 32 tiles at a time, one per lane; the next 32 are fetched halfway
        int pg = -1, pg_next = -1;
        float ks = 0.f, vs = 0.f, ks_next = 0.f, vs_next = 0.f;
        const auto fetch = [&](int base, int& page, float& k_s, float& v_s) {
            const int i = base + lane;
            page = -1;
            if (i < nv) {
                page = page_of(table, p.max_pages, p.num_pages, p.shift, rg.key0(entry(i)));
                if (page < 0) page_error(p.err);
                if constexpr (F8) {
                    if (page >= 0) {
                        const long long ph = static_cast<long long>(page) * p.H_kv + hk;
                        k_s = p.k_scale[ph];
                        v_s = p.v_scale[ph];
                    }
                }
            }
        };
        // first key that any row sees behind the sinks
        const int low = p.window > 0 ? max(0, len - p.Nq - p.window + 1) : 0;
        const int nu = (nv + TP - 1) / TP;  // slots' worth
        int in_slot = 0;                    // ring slot to fill next
        const auto issue = [&](int u) {
            if (u >= nu) return;
#pragma unroll
            for (int tp = 0; tp < TP; ++tp) {
                const int i = u * TP + tp;
                if ((i & 31) == 0 && i > 0) {
                    pg = pg_next;
                    ks = ks_next;
                    vs = vs_next;
                }
                if ((i & 31) == 16) fetch((i & ~31) + 32, pg_next, ks_next, vs_next);
                const int key0 = rg.key0(entry(i));
                const int page = __shfl_sync(0xffffffffu, pg, i & 31);  // (-1 behind the piece's last tile, too)
                const uint32_t dst = ring + in_slot * L::kSlot + tp * 2 * L::kTile;
                typename Shared::Slot sl;
                sl.key0 = page < 0 ? 0x7fffff00 : key0;
                if constexpr (F8) {
                    sl.ks = __shfl_sync(0xffffffffu, ks, i & 31);
                    sl.vs = __shfl_sync(0xffffffffu, vs, i & 31);
                }
                if (lane == 0) sh.slot[warp][in_slot][tp] = sl;
                // (a page is at least one tile: a tile's rows lie together)
                const long long off =
                    (((static_cast<long long>(max(page, 0)) * p.H_kv + hk) << p.shift) + (key0 & ((1 << p.shift) - 1))) * ROW +
                    lane * 16;
                const uint8_t* ksrc = p.K + off;
                const uint8_t* vsrc = p.V + off;
                if (page >= 0 && key0 + kPagedTile <= len && (key0 >= low || key0 + kPagedTile <= p.sinks)) {
#pragma unroll
                    for (int j = 0; j < CH / 2; ++j) {
                        cp_async16(dst + j * 512 + k_dst, ksrc + j * 512);
                        cp_async16(dst + L::kTile + j * 512 + (v_dst ^ W::v_dst_x(j)), vsrc + j * 512);
                    }
                } else {
                    // rows that no row of the call sees become zeros
#pragma unroll
                    for (int j = 0; j < CH / 2; ++j) {
                        const int key = key0 + (j * 32 + lane) / CH;
                        const int bytes = page >= 0 && key < len && (key >= low || key < p.sinks) ? 16 : 0;
                        cp_async16(dst + j * 512 + k_dst, ksrc + j * 512, bytes);
                        cp_async16(dst + L::kTile + j * 512 + (v_dst ^ W::v_dst_x(j)), vsrc + j * 512, bytes);
                    }
                }
            }
            in_slot = in_slot + 1 == S ? 0 : in_slot + 1;
        };
        fetch(0, pg, ks, vs);
#pragma unroll
        for (int i = 0; i < S - 1; ++i) {
            issue(i);
            cp_commit();
        }

        // ---- queries: the narrow operand, in the order of the key pieces ----
        uint32_t q[NT][KS][2];
        float rs[NT][2];  // 8-bit: 2^x that row (2 t4, 2 t4 + 1) was divided by, times tau log2 e
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int r = nt * 8 + g;
            const bool in = r < rows;
            const int rr = row0 + (in ? r : 0), hh = rr / p.Nq, qi = rr - hh * p.Nq;
            const __nv_bfloat16* src =
                p.Q + b * p.q_sb + static_cast<long long>(hk * p.G + hh) * p.q_sh + qi * p.q_sn;
            if constexpr (!F8) {
#pragma unroll
                for (int c = 0; c < kChunksK; ++c) {
                    uint4 w = make_uint4(0u, 0u, 0u, 0u);
                    if (in) w = reinterpret_cast<const uint4*>(src)[t4 + 4 * c];
                    q[nt][2 * c][0] = w.x;
                    q[nt][2 * c][1] = w.y;
                    q[nt][2 * c + 1][0] = w.z;
                    q[nt][2 * c + 1][1] = w.w;
                }
                rs[nt][0] = rs[nt][1] = p.scale_log2;
            } else {
                // key piece c of this thread holds columns 16 (t4 + 4 c) .. + 15
                uint4 w[2 * kChunksK];
                float m = 0.f;
#pragma unroll
                for (int c = 0; c < 2 * kChunksK; ++c) {
                    w[c] = make_uint4(0u, 0u, 0u, 0u);
                    if (in) w[c] = reinterpret_cast<const uint4*>(src)[2 * (t4 + 4 * (c >> 1)) + (c & 1)];
                    const uint32_t e[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        m = fmaxf(m, fmaxf(fabsf(__uint_as_float(e[i] << 16)), fabsf(__uint_as_float(e[i] & 0xffff0000u))));
                }
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
                // largest magnitude to [2^14, 2^15); a row of zeros, or with infinities, as it is
                int ex = static_cast<int>(__float_as_uint(m) >> 23) - 127 - 14;
                if (m == 0.f || m > 3.4e38f) ex = 0;
                ex = max(-126, min(112, ex));
                const float down = __uint_as_float(static_cast<uint32_t>(127 - ex) << 23);
                const float up = __uint_as_float(static_cast<uint32_t>(127 + ex) << 23);
#pragma unroll
                for (int c = 0; c < 2 * kChunksK; ++c) {
                    const uint32_t e[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        q[nt][2 * c + (i >> 1)][i & 1] =
                            pack_f16(__uint_as_float(e[i] << 16) * down, __uint_as_float(e[i] & 0xffff0000u) * down);
                }
                rs[nt][0] = p.scale_log2 * __shfl_sync(0xffffffffu, up, 8 * t4);
                rs[nt][1] = p.scale_log2 * __shfl_sync(0xffffffffu, up, 8 * t4 + 4);
            }
        }
        int last[NT][2];  // last visible key of rows 2 t4, 2 t4 + 1 of each tile (-1: no such row)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = nt * 8 + 2 * t4 + e;
                last[nt][e] = r < rows ? len - p.Nq + (row0 + r) % p.Nq : -1;
            }

        // MOD: the rows' heads, slopes and bias of far keys (log2 units)
        [[maybe_unused]] int mod_h[NT][2];
        [[maybe_unused]] float mod_f[NT][2];
        if constexpr (MOD) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = nt * 8 + 2 * t4 + e;
                    const int h = hk * p.G + (row0 + (r < rows ? r : 0)) / p.Nq;
                    mod_h[nt][e] = h;
                    mod_f[nt][e] = 0.f;
                    if (rows > 0 && p.slopes) mod_f[nt][e] = kLog2e * p.slopes[h];
                    if (rows > 0 && p.bias) mod_f[nt][e] = bias_at(h, p.far);
                }
        }

        float acc[NT][MT][4];
        float m_run[NT][2], l_run[NT][2], mv_run[NT][2], fac[NT][2];  // fac: 2^(m - mv)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int j = 0; j < MT; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[nt][j][e] = 0.f;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                m_run[nt][e] = mv_run[nt][e] = -INFINITY;
                l_run[nt][e] = 0.f;
                fac[nt][e] = 0.f;
            }
        }
        int slot_at = 0;
        for (int u = 0; u < nu; ++u) {
            cp_wait<S - 2>();
            __syncwarp();
            issue(u + S - 1);
            cp_commit();
            const uint32_t ks_at = ring + slot_at * L::kSlot + k_src, vs_at = ring + slot_at * L::kSlot + L::kTile + v_src;
            typename Shared::Slot sl[TP];
#pragma unroll
            for (int tp = 0; tp < TP; ++tp) sl[tp] = sh.slot[warp][slot_at][tp];
            slot_at = slot_at + 1 == S ? 0 : slot_at + 1;

            // a bias of near keys is fetched while the products below run (tiles all of whose keys are far from every
            // row have one bias per row)
            [[maybe_unused]] float bias_y[TP][NT][4];
            if constexpr (MOD) {
                if (p.bias) {
#pragma unroll
                    for (int tp = 0; tp < TP; ++tp) {
                        const int key0 = sl[tp].key0;
                        const bool near = len - p.Nq - (key0 + kPagedTile - 1) < p.far;
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                bias_y[tp][nt][e] = mod_f[nt][e & 1];
                                if (near)  // (keys behind the row are hidden below)
                                    bias_y[tp][nt][e] = bias_at(mod_h[nt][e & 1], last[nt][e & 1] - (key0 + g + (e & 2 ? 8 : 0)));
                            }
                    }
                }
            }

            // S^T = K Q^T
            float s[TP][NT][4];
#pragma unroll
            for (int tp = 0; tp < TP; ++tp)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[tp][nt][e] = 0.f;
#pragma unroll
            for (int c = 0; c < kChunksK; ++c) {
#pragma unroll
                for (int tp = 0; tp < TP; ++tp) {
                    const uint32_t at = (ks_at + tp * 2 * L::kTile) ^ (c << 6);
                    const uint4 ka = lds128(at), kb = lds128(at + 8 * ROW);
                    const uint32_t a[4] = {ka.x, ka.y, ka.z, ka.w}, bb[4] = {kb.x, kb.y, kb.z, kb.w};
                    if constexpr (!F8) {
#pragma unroll
                        for (int h = 0; h < 2; ++h)
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                mma16816<false>(s[tp][nt], a[2 * h], bb[2 * h], a[2 * h + 1], bb[2 * h + 1],
                                                q[nt][2 * c + h][0], q[nt][2 * c + h][1]);
                    } else {
#pragma unroll
                        for (int h = 0; h < 4; ++h) {
                            uint32_t a0, a2, a1, a3;
                            widen_e4m3x4(a[h], a0, a2);
                            widen_e4m3x4(bb[h], a1, a3);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                mma16816<true>(s[tp][nt], a0, a1, a2, a3, q[nt][4 * c + h][0], q[nt][4 * c + h][1]);
                        }
                    }
                }
            }

            // scale, mask; s becomes the score less the running reference (log2 units)
            bool grow = false;
            float vsc[TP], lvs[TP];
#pragma unroll
            for (int tp = 0; tp < TP; ++tp) {
                const int key0 = sl[tp].key0;
                const float ksc = F8 ? sl[tp].ks : 1.f;
                vsc[tp] = F8 ? sl[tp].vs : 1.f;
                lvs[tp] = F8 ? lg2(vsc[tp]) : 0.f;
                const bool whole = key0 + kPagedTile <= len - p.Nq + 1 &&
                                   (p.window == 0 || key0 >= len - p.window || key0 + kPagedTile <= p.sinks);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float(&x)[4] = s[tp][nt];
                    float scale[2], ref[2], most[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float m = m_run[nt][e];  // -inf until the row has seen a key
                        scale[e] = F8 ? rs[nt][e] * ksc : rs[nt][e];
                        ref[e] = m == -INFINITY ? 0.f : m;
                        // the largest that the references allow (8-bit: that of P vs, too)
                        most[e] = F8 ? kSlack + fminf(0.f, mv_run[nt][e] - lvs[tp] - m) : kSlack;
                        if (m == -INFINITY) most[e] = -INFINITY;
                    }
                    if constexpr (!MOD) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) x[e] = fmaf(x[e], scale[e & 1], -ref[e & 1]);
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e) x[e] *= scale[e & 1];
                        if (p.cap_log2 > 0.f) {
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const uint64_t u = f2_pack(x[e] * p.cap_inv, x[e + 2] * p.cap_inv);
                                const float2 th = f2_unpack(p.cap_log2 > kCapExact ? tanh2<kTanhSafe>(u) : tanh2<kTanhExp>(u));
                                x[e] = th.x * p.cap_log2;
                                x[e + 2] = th.y * p.cap_log2;
                            }
                        }
                        if (p.slopes) {
                            // (j - i as a whole number first: positions beyond 2^24 are not exact in fp32, near distances are)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const float dist = static_cast<float>(key0 + g - last[nt][e]);
                                x[e] = fmaf(mod_f[nt][e], dist, x[e]);
                                x[e + 2] = fmaf(mod_f[nt][e], dist + 8.f, x[e + 2]);
                            }
                        } else if (p.bias) {
#pragma unroll
                            for (int e = 0; e < 4; ++e) x[e] += bias_y[tp][nt][e];
                        }
#pragma unroll
                        for (int e = 0; e < 4; ++e) x[e] -= ref[e & 1];
                    }
                    if (!whole) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int key = key0 + g + (e & 2 ? 8 : 0), la = last[nt][e & 1];
                            const bool see = key <= la && (p.window == 0 || key > la - p.window || key < p.sinks);
                            if (!see) x[e] = -INFINITY;
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) grow |= x[e] > most[e & 1];
                }
            }
            if (__any_sync(0xffffffffu, grow)) {
                // (rare: on a piece's first tiles, and where scores rise by more than the slack)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float m = m_run[nt][e], ref = m == -INFINITY ? 0.f : m;
                        float mx[TP], m_new = m;
#pragma unroll
                        for (int tp = 0; tp < TP; ++tp) {
                            mx[tp] = ref + max_over_g(fmaxf(s[tp][nt][e], s[tp][nt][e + 2]));
                            m_new = fmaxf(m_new, mx[tp] - kLift);
                        }
                        const float alpha = m == -INFINITY ? 1.f : ex2(m - m_new);
                        const float down = m_new == -INFINITY ? 0.f : m_new - ref;
                        m_run[nt][e] = m_new;
                        l_run[nt][e] *= alpha;
                        float beta = alpha;
                        if constexpr (F8) {
                            float mv_new = mv_run[nt][e];
#pragma unroll
                            for (int tp = 0; tp < TP; ++tp) mv_new = fmaxf(mv_new, mx[tp] + lvs[tp] - kLift);
                            beta = mv_new == -INFINITY ? 1.f : ex2(mv_run[nt][e] - mv_new);
                            mv_run[nt][e] = mv_new;
                            fac[nt][e] = mv_new == -INFINITY ? 0.f : ex2(fminf(m_new - mv_new, 127.f));
                        }
#pragma unroll
                        for (int tp = 0; tp < TP; ++tp) {
                            s[tp][nt][e] -= down;
                            s[tp][nt][e + 2] -= down;
                        }
#pragma unroll
                        for (int j = 0; j < MT; ++j) {
                            acc[nt][j][e] *= beta;
                            acc[nt][j][e + 2] *= beta;
                        }
                    }
            }

#pragma unroll
            for (int tp = 0; tp < TP; ++tp) {
                // P^T, from the accumulator's layout to the operand's
                uint32_t pb[NT][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) w[e] = ex2(s[tp][nt][e]);
                    l_run[nt][0] += w[0] + w[2];
                    l_run[nt][1] += w[1] + w[3];
                    if constexpr (F8) {
                        // (cut: with scales 2^100 apart the factor passes fp32, and a weight of 0 stays 0)
                        const float f0 = fminf(fac[nt][0] * vsc[tp], 0x1p112f), f1 = fminf(fac[nt][1] * vsc[tp], 0x1p112f);
                        pb[nt][0] = movmatrix(pack_f16(w[0] * f0, w[1] * f1));
                        pb[nt][1] = movmatrix(pack_f16(w[2] * f0, w[3] * f1));
                    } else {
                        pb[nt][0] = movmatrix(pack_bf16(w[0], w[1]));
                        pb[nt][1] = movmatrix(pack_bf16(w[2], w[3]));
                    }
                }

                // O^T += V^T P^T: element e of this thread's columns of rows 2 t4, 2 t4 + 1 (lo)
                // and 2 t4 + 8, 2 t4 + 9 (hi); tile j takes elements 2 j and 2 j + 1
                const uint32_t v_at = vs_at + tp * 2 * L::kTile;
                if constexpr (!F8) {
#pragma unroll
                    for (int c = 0; c < CH / 8; ++c) {
                        const uint32_t at = v_at + c * 128, at1 = W::v_row1(at);
                        const uint4 x0 = lds128(at), x1 = lds128(at1), y0 = lds128(at + 8 * ROW), y1 = lds128(at1 + 8 * ROW);
                        const uint32_t a[4] = {x0.x, x0.y, x0.z, x0.w}, a1[4] = {x1.x, x1.y, x1.z, x1.w};
                        const uint32_t bb[4] = {y0.x, y0.y, y0.z, y0.w}, b1[4] = {y1.x, y1.y, y1.z, y1.w};
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const uint32_t lo0 = __byte_perm(a[j], a1[j], 0x5410), lo1 = __byte_perm(a[j], a1[j], 0x7632);
                            const uint32_t hi0 = __byte_perm(bb[j], b1[j], 0x5410), hi1 = __byte_perm(bb[j], b1[j], 0x7632);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                mma16816<false>(acc[nt][4 * c + j], lo0, lo1, hi0, hi1, pb[nt][0], pb[nt][1]);
                        }
                    }
                } else {
                    constexpr int kWords = D / 32;  // of a row per thread (16 columns at d = 128, 8 at 64)
                    const uint32_t at = v_at, at1 = W::v_row1(at);
                    uint32_t a[4][4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t from = (k & 1 ? at1 : at) + (k >> 1) * 8 * ROW;
                        if constexpr (D == 128) {
                            const uint4 w = lds128(from);
                            a[k][0] = w.x;
                            a[k][1] = w.y;
                            a[k][2] = w.z;
                            a[k][3] = w.w;
                        } else {
                            const uint2 w = lds64(from);
                            a[k][0] = w.x;
                            a[k][1] = w.y;
                        }
                    }
#pragma unroll
                    for (int j = 0; j < kWords; ++j) {
                        uint32_t f[8];  // [lo: elements 4 j .. 4 j + 3, hi: the same]
                        widen_e4m3x4(__byte_perm(a[0][j], a[1][j], 0x5140), f[0], f[1]);
                        widen_e4m3x4(__byte_perm(a[0][j], a[1][j], 0x7362), f[2], f[3]);
                        widen_e4m3x4(__byte_perm(a[2][j], a[3][j], 0x5140), f[4], f[5]);
                        widen_e4m3x4(__byte_perm(a[2][j], a[3][j], 0x7362), f[6], f[7]);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            mma16816<true>(acc[nt][2 * j], f[0], f[1], f[4], f[5], pb[nt][0], pb[nt][1]);
                            mma16816<true>(acc[nt][2 * j + 1], f[2], f[3], f[6], f[7], pb[nt][0], pb[nt][1]);
                        }
                    }
                }
            }
        }
        cp_wait<0>();

        if constexpr (WHOLE) {
            // ---- join the warps of the same rows ----
            // factor of this warp's sums: 2^(its reference - the joint max) / the joint sum
            float f[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float l = sum_over_g(l_run[nt][e]);
                    if (g == 0) {
                        sh.m[warp][nt * 8 + 2 * t4 + e] = m_run[nt][e];
                        sh.l[warp][nt * 8 + 2 * t4 + e] = l;
                    }
                }
            __syncthreads();  // (and every warp is done with its ring)
            float* red = reinterpret_cast<float*>(smem);  // [warp][R][D]
            const int liw = WARPS / p.rwarps, lturn = warp / p.rwarps;  // of this block
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = nt * 8 + 2 * t4 + e;
                    float m = -INFINITY, l = 0.f;
                    for (int k = 0; k < liw; ++k) m = fmaxf(m, sh.m[k * p.rwarps + rw][r]);
                    const float ref = m == -INFINITY ? 0.f : m;
                    for (int k = 0; k < liw; ++k) l += sh.l[k * p.rwarps + rw][r] * ex2(sh.m[k * p.rwarps + rw][r] - ref);
                    // (a row that sees nothing: l = 0 and O = 0, LSE = -inf; NaN where a score was)
                    for (int k = 0; m == -INFINITY && k < liw; ++k) l += sh.l[k * p.rwarps + rw][r];
                    f[nt][e] = l == 0.f ? 0.f : ex2((F8 ? mv_run[nt][e] : m_run[nt][e]) - ref) / l;
                    if (WW > kPagedWarps && cn > 1) {
                        if (lturn == 0 && g == 0) sh.lse[rw * R + r] = ref + lg2(l);
                    } else if (turn == 0 && g == 0 && r < rows) {
                        const int hh = (row0 + r) / p.Nq, qi = (row0 + r) - hh * p.Nq, h = hk * p.G + hh;
                        p.LSE[(static_cast<long long>(b) * p.H + h) * p.Nq + qi] = (ref + lg2(l)) * kLn2;
                    }
                    constexpr int RUN = F8 ? D / 8 : 8;  // columns that lie together
                    float* dst = red + (warp * R + r) * D;
#pragma unroll
                    for (int j = 0; j < MT; j += 2) {
                        const int col = (2 * j / RUN) * (8 * RUN) + RUN * g + 2 * j % RUN;
                        *reinterpret_cast<float4*>(dst + col) =
                            make_float4(acc[nt][j][e] * f[nt][e], acc[nt][j][e + 2] * f[nt][e],
                                        acc[nt][j + 1][e] * f[nt][e], acc[nt][j + 1][e + 2] * f[nt][e]);
                    }
                }
            __syncthreads();
            // the iw warps of row warp rw write its rows
            for (int i = lturn * 32 + lane; i < rows * (D / 4); i += liw * 32) {
                const int r = i / (D / 4), col = i % (D / 4) * 4;
                float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
                for (int k = 0; k < liw; ++k) {
                    const float4 y = *reinterpret_cast<const float4*>(red + ((k * p.rwarps + rw) * R + r) * D + col);
                    o.x += y.x;
                    o.y += y.y;
                    o.z += y.z;
                    o.w += y.w;
                }
                if (WW > kPagedWarps && cn > 1) {  // (over row warp 0's part, which only this thread has read)
                    *reinterpret_cast<float4*>(red + (rw * R + r) * D + col) = o;
                    continue;
                }
                const int hh = (row0 + r) / p.Nq, qi = (row0 + r) - hh * p.Nq, h = hk * p.G + hh;
                *reinterpret_cast<uint2*>(p.O + b * p.o_sb + static_cast<long long>(h) * p.o_sh + qi * p.o_sn + col) =
                    make_uint2(pack_bf16(o.x, o.y), pack_bf16(o.z, o.w));
            }
            if constexpr (WW > kPagedWarps) {
                if (cn == 1) return;
                // the blocks of the cluster: O = sum_c 2^(l_c - L) O_c, each block a part of the rows
                cluster_barrier();
                for (int i = turn * 32 + lane; i < rows * (D / 4); i += iw * 32) {
                    const int r = i / (D / 4), col = i % (D / 4) * 4;
                    const uint32_t l_at = smem_addr(&sh.lse[rw * R + r]), o_at = smem_addr(red + (rw * R + r) * D + col);
                    float m = -INFINITY, sum = 0.f;
                    for (int k = 0; k < cn; ++k) m = fmaxf(m, ld_cluster(map_block(l_at, k)));
                    const float ref = m == -INFINITY ? 0.f : m;
                    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
                    for (int k = 0; k < cn; ++k) {
                        const float w = ex2(ld_cluster(map_block(l_at, k)) - ref);
                        const float4 y = ld_cluster4(map_block(o_at, k));
                        sum += w;
                        o.x = fmaf(w, y.x, o.x);
                        o.y = fmaf(w, y.y, o.y);
                        o.z = fmaf(w, y.z, o.z);
                        o.w = fmaf(w, y.w, o.w);
                    }
                    const float inv = sum == 0.f ? 0.f : 1.f / sum;  // (0: the row sees nothing)
                    const int hh = (row0 + r) / p.Nq, qi = (row0 + r) - hh * p.Nq, h = hk * p.G + hh;
                    *reinterpret_cast<uint2*>(p.O + b * p.o_sb + static_cast<long long>(h) * p.o_sh + qi * p.o_sn + col) =
                        make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
                    if (col == 0) p.LSE[(static_cast<long long>(b) * p.H + h) * p.Nq + qi] = (ref + lg2(sum)) * kLn2;
                }
                cluster_barrier();  // (no block ends while others read its memory)
            }
            return;
        }
        // ---- this piece's result ----
        const bool final_piece = u0 == 0 && u1 >= rg.n;
        const long long slot = 2ll * (static_cast<long long>(share) * p.rwarps + rw) + (u0 == 0 ? 1 : 0);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = nt * 8 + 2 * t4 + e;
                const float l = sum_over_g(l_run[nt][e]), m = m_run[nt][e];
                // (a row that sees nothing: l = 0 and O = 0, LSE = -inf; NaN where a score was)
                float f = l == 0.f ? 0.f : 1.f / l;
                if (F8 && l != 0.f) f *= ex2(mv_run[nt][e] - m);
                const float ls = (m == -INFINITY ? 0.f : m) + lg2(l);
                if (r >= rows) continue;
                constexpr int RUN = F8 ? D / 8 : 8;  // columns that lie together
                if (final_piece) {
                    const int hh = (row0 + r) / p.Nq, qi = (row0 + r) - hh * p.Nq, h = hk * p.G + hh;
                    __nv_bfloat16* dst = p.O + b * p.o_sb + static_cast<long long>(h) * p.o_sh + qi * p.o_sn;
#pragma unroll
                    for (int j = 0; j < MT; j += 4) {
                        const int col = (2 * j / RUN) * (8 * RUN) + RUN * g + 2 * j % RUN;
                        *reinterpret_cast<uint4*>(dst + col) =
                            make_uint4(pack_bf16(acc[nt][j][e] * f, acc[nt][j][e + 2] * f),
                                       pack_bf16(acc[nt][j + 1][e] * f, acc[nt][j + 1][e + 2] * f),
                                       pack_bf16(acc[nt][j + 2][e] * f, acc[nt][j + 2][e + 2] * f),
                                       pack_bf16(acc[nt][j + 3][e] * f, acc[nt][j + 3][e + 2] * f));
                    }
                    if (g == 0) p.LSE[(static_cast<long long>(b) * p.H + h) * p.Nq + qi] = ls * kLn2;
                } else {
                    float* dst = p.part_o + (slot * R + r) * D;
#pragma unroll
                    for (int j = 0; j < MT; j += 2) {
                        const int col = (2 * j / RUN) * (8 * RUN) + RUN * g + 2 * j % RUN;
                        *reinterpret_cast<float4*>(dst + col) =
                            make_float4(acc[nt][j][e] * f, acc[nt][j][e + 2] * f, acc[nt][j + 1][e] * f,
                                        acc[nt][j + 1][e + 2] * f);
                    }
                    if (g == 0) p.part_l[slot * R + r] = ls;
                }
            }
        }
        if (u0 == 0 && rw == 0 && lane == 0) {
            const int pieces = static_cast<int>(cut.of(seg_first + max(1, rg.n) - 1) - share) + 1;
            p.seg[static_cast<long long>(b) * segs_per_b + in_b] =
                make_int2(static_cast<int>(share), pieces);
        }
        if (!next()) return;
        __syncwarp();  // (the ring's last slots have been read)
    }
}

// Adds a segment's pieces: O = sum_s 2^(l_s - L) O_s, L = log2 sum_s 2^(l_s), in order.
// With few pieces per segment (on average, over full tables) a warp adds a row by itself,
// eight pieces' loads in flight at once; block (segment, y) takes the rows y, y + gridDim.y,
// ...  With many, block (segment, row, z) takes D / gridDim.z columns of one row, each warp 32
// of them and 32 pieces at a time: eight lanes to a piece's 128 bytes, eight loads in flight.
constexpr int kFewPieces = 16;
constexpr int kCombineWarps = 16;

template <int D, int NT, bool MANY>
__global__ void __launch_bounds__(32 * (MANY ? kCombineWarps : 8)) fa_paged_combine_kernel(const PagedParams p) {
    constexpr int R = 8 * NT, PER = D / 32, kBatch = 8;
    const int segs_per_b = p.H_kv * p.rgroups;
    const int b = static_cast<int>(blockIdx.x) / segs_per_b, in_b = static_cast<int>(blockIdx.x) - b * segs_per_b;
    const int hk = in_b / p.rgroups, row0 = (in_b - hk * p.rgroups) * p.rwarps * R;
    const int rows = min(p.rwarps * R, p.G * p.Nq - row0);
    const int warps = static_cast<int>(blockDim.x >> 5);
    const int warp = static_cast<int>(threadIdx.x >> 5), lane = threadIdx.x & 31;
    griddep_wait();
    const int2 sg = p.seg[blockIdx.x];
    const int n = sg.y;
    // (the bound holds unless the first kernel gave up before it wrote its headers)
    if (n <= 1 || sg.x < 0 || sg.x > p.shares - n) return;
    const int row_step = MANY ? rows : static_cast<int>(gridDim.y) * warps;
    for (int row = static_cast<int>(blockIdx.y) + (MANY ? 0 : warp * static_cast<int>(gridDim.y)); row < rows; row += row_step) {
        const int rw = row / R, r = row - rw * R;
        // piece 0 lies in its warp's second slot (it ends the share), the others in their first
        const auto at = [&](int s) {
            const long long w = static_cast<long long>(sg.x + s) * p.rwarps + rw;
            return (2 * w + (s == 0 ? 1 : 0)) * R + r;
        };
        const int hh = (row0 + row) / p.Nq, qi = (row0 + row) - hh * p.Nq, h = hk * p.G + hh;
        __nv_bfloat16* dst = p.O + b * p.o_sb + static_cast<long long>(h) * p.o_sh + qi * p.o_sn;
        float* lse = p.LSE + (static_cast<long long>(b) * p.H + h) * p.Nq + qi;
        if constexpr (MANY) {
            __shared__ float red[kCombineWarps][32], red_l[kCombineWarps], red_m[kCombineWarps];
            const int cw = D / 32 / static_cast<int>(gridDim.z), cg = warp % cw;  // 32-column groups of the block
            const int sub = lane >> 3, col = 32 * (static_cast<int>(blockIdx.z) * cw + cg) + 4 * (lane & 7);
            const int group = warp / cw, groups = warps / cw;  // of pieces
            float m = -INFINITY;
            for (int s = threadIdx.x; s < n; s += blockDim.x) m = fmaxf(m, p.part_l[at(s)]);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            if (lane == 0) red_m[warp] = m;
            __syncthreads();
            for (int k = 0; k < warps; ++k) m = fmaxf(m, red_m[k]);
            const float ref = m == -INFINITY ? 0.f : m;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            float sum = 0.f;
            for (int s0 = group * 4 * kBatch; s0 < n; s0 += groups * 4 * kBatch) {
                float4 v[kBatch];
                float l[kBatch];
#pragma unroll
                for (int k = 0; k < kBatch; ++k) {
                    const int s = s0 + 4 * k + sub;
                    if (s < n) {
                        l[k] = p.part_l[at(s)];
                        v[k] = *reinterpret_cast<const float4*>(p.part_o + at(s) * D + col);
                    }
                }
#pragma unroll
                for (int k = 0; k < kBatch; ++k) {
                    if (s0 + 4 * k + sub < n) {
                        const float w = ex2(l[k] - ref);
                        sum += w;
                        acc.x = fmaf(w, v[k].x, acc.x);
                        acc.y = fmaf(w, v[k].y, acc.y);
                        acc.z = fmaf(w, v[k].z, acc.z);
                        acc.w = fmaf(w, v[k].w, acc.w);
                    }
                }
            }
#pragma unroll
            for (int o = 8; o < 32; o <<= 1) {
                sum += __shfl_xor_sync(0xffffffffu, sum, o);
                acc.x += __shfl_xor_sync(0xffffffffu, acc.x, o);
                acc.y += __shfl_xor_sync(0xffffffffu, acc.y, o);
                acc.z += __shfl_xor_sync(0xffffffffu, acc.z, o);
                acc.w += __shfl_xor_sync(0xffffffffu, acc.w, o);
            }
            if (sub == 0) *reinterpret_cast<float4*>(&red[warp][4 * (lane & 7)]) = acc;
            if (lane == 0) red_l[warp] = sum;
            __syncthreads();
            if (group > 0) return;
            sum = 0.f;
            float o = 0.f;
            for (int k = cg; k < warps; k += cw) {
                sum += red_l[k];
                o += red[k][lane];
            }
            o = sum == 0.f ? 0.f : o / sum;  // (0: the row sees nothing)
            const float o1 = __shfl_down_sync(0xffffffffu, o, 1);
            if ((lane & 1) == 0) *reinterpret_cast<uint32_t*>(dst + col - 4 * (lane & 7) + lane) = pack_bf16(o, o1);
            if (threadIdx.x == 0 && blockIdx.z == 0) *lse = (ref + lg2(sum)) * kLn2;
        } else {
            float acc[PER], v[kBatch][PER];
#pragma unroll
            for (int e = 0; e < PER; ++e) acc[e] = 0.f;
            // pieces s0 .. s0 + 7 (below n)
            const auto load = [&](int s0) {
#pragma unroll
                for (int k = 0; k < kBatch; ++k) {
                    if (s0 + k < n) {
                        const float* src = p.part_o + at(s0 + k) * D + lane * PER;
                        if constexpr (PER == 4) {
                            const float4 y = *reinterpret_cast<const float4*>(src);
                            v[k][0] = y.x;
                            v[k][1] = y.y;
                            v[k][2] = y.z;
                            v[k][3] = y.w;
                        } else {
                            const float2 y = *reinterpret_cast<const float2*>(src);
                            v[k][0] = y.x;
                            v[k][1] = y.y;
                        }
                    }
                }
            };
            // ... with the weights of lanes from on
            const auto add = [&](int s0, float w, int from) {
#pragma unroll
                for (int k = 0; k < kBatch; ++k) {
                    const float wk = __shfl_sync(0xffffffffu, w, from + k);
                    if (s0 + k < n) {
#pragma unroll
                        for (int e = 0; e < PER; ++e) acc[e] = fmaf(wk, v[k][e], acc[e]);
                    }
                }
            };
            load(0);
            const float l = lane < n ? p.part_l[at(lane)] : -INFINITY;
            float m = l;
            for (int s = lane + 32; s < n; s += 32) m = fmaxf(m, p.part_l[at(s)]);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            const float ref = m == -INFINITY ? 0.f : m;
            float w = ex2(l - ref), sum = w;
            add(0, w, 0);
            for (int s0 = kBatch; s0 < n; s0 += kBatch) {
                load(s0);
                if ((s0 & 31) == 0) {  // (the next 32 pieces' weights, one per lane)
                    w = s0 + lane < n ? ex2(p.part_l[at(s0 + lane)] - ref) : 0.f;
                    sum += w;
                }
                add(s0, w, s0 & 31);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            const float inv = sum == 0.f ? 0.f : 1.f / sum;  // (0: the row sees nothing)
            if constexpr (PER == 4)
                *reinterpret_cast<uint2*>(dst + lane * PER) =
                    make_uint2(pack_bf16(acc[0] * inv, acc[1] * inv), pack_bf16(acc[2] * inv, acc[3] * inv));
            else
                *reinterpret_cast<uint32_t*>(dst + lane * PER) = pack_bf16(acc[0] * inv, acc[1] * inv);
            if (lane == 0) *lse = (ref + lg2(sum)) * kLn2;
        }
    }
}

// Query rows per warp: 8 for up to 8 rows of a key head, else 16.
int row_tiles(int rows) { return rows <= 8 ? 1 : 2; }

template <int D, int NT, bool F8>
constexpr int ctas_per_sm() { return PagedLayout<D, NT, F8>::kCtas; }

int ctas_for(int d, int nt, bool fp8) {
    if (d == 64) {
        if (nt == 1) return fp8 ? ctas_per_sm<64, 1, true>() : ctas_per_sm<64, 1, false>();
        return fp8 ? ctas_per_sm<64, 2, true>() : ctas_per_sm<64, 2, false>();
    }
    if (nt == 1) return fp8 ? ctas_per_sm<128, 1, true>() : ctas_per_sm<128, 1, false>();
    return fp8 ? ctas_per_sm<128, 2, true>() : ctas_per_sm<128, 2, false>();
}

// Whole segments up to this many tiles (of a full table, within the window; the row warps
// share a block's): ten per warp, of four warps, or where every segment has an SM to itself
// and more than two tiles per warp (kNarrowTiles) of eight; where SMs are left over, of a
// cluster of up to eight such blocks, which keeps five tiles or fewer per warp while it can.
// With several row warps eight warps pay for fewer tiles.
//   four warps: 640 keys of 64 sequences, 8 key heads, 34.3 us whole and 34.6 split; 1000
//     keys 49.8 and 46.3;
//   eight: 12 heads, 128 keys 4.6 us by eight and 3.9 by four, 517 keys 6.2 and 6.8; 64
//     segments, 1280 keys 10.5 and split 12.6, 2000 14.1 and 13.1; 8 segments of 32 rows (two
//     row warps), 320 keys 9.9 and 12.3, 640 13.4 and 10.2;
//   clusters: 8 segments, 1000 keys 8.2 us by two blocks and 8.9 by one, 3000 8.0 and split
//     10.6, 9000 11.7 and 12.6; 32 segments, 2000 8.5 and 11.5; 64, 3000 17.0 and 17.4; one
//     segment, 8000 keys 10.9 and 9.6.
constexpr int kWholeTiles = 40, kWideTiles = 80, kWideRowTiles = 53, kNarrowTiles = 8, kMaxClusterLog2 = 3, kFewBlocks = 32;
// Clusters of 1, 2, 4 and 8 blocks, one to an SM, that run at a time: a cluster's SMs lie in
// one processing cluster, some of which hold an odd number (cudaOccupancyMaxActiveClusters,
// alike on two chips).  More would take a second round: 16 segments of 3000 keys by eight
// blocks 13.8 us, by four 9.2; 37 of 2000 by four 14.4, by two 10.3.
constexpr int kClusters[kMaxClusterLog2 + 1] = {kSms, 76, 36, 15};

// Workspace: segment headers, then the pieces' sums and outputs, each 256-aligned; none
// for whole segments.
struct PagedPlan {
    int nt, rwarps, rgroups, ctas;
    bool whole, wide;  // whole segments, by eight warps
    int cluster_log2;  // wide: of the blocks per segment
    long long segs, tiles;  // tiles: of a full table, all segments
    size_t part_l, part_o, bytes;
};
PagedPlan paged_plan(const PagedCache& c, int H, int Nq, int window, int sinks, bool fp8) {
    const auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    PagedPlan pl;
    const int rows = H / c.H_kv * Nq;
    pl.nt = row_tiles(rows);
    const int rblocks = (rows + 8 * pl.nt - 1) / (8 * pl.nt);
    pl.rwarps = rblocks == 1 ? 1 : rblocks == 2 ? 2 : 4;
    pl.rgroups = (rblocks + pl.rwarps - 1) / pl.rwarps;
    pl.segs = static_cast<long long>(c.B) * c.H_kv * pl.rgroups;
    pl.ctas = kSms * ctas_for(c.d, pl.nt, fp8);
    // a full table's tiles, or with a window those of a long sequence (its ends may cut tiles)
    long long most = (static_cast<long long>(c.max_pages) << c.shift) / kPagedTile;
    if (window > 0)
        most = std::min(most, (static_cast<long long>(window) + Nq) / kPagedTile + 2 + (sinks + kPagedTile - 1ll) / kPagedTile);
    pl.tiles = pl.segs * most;
    const long long work = most * pl.rwarps, per_block = pl.rwarps == 1 ? kWideTiles : kWideRowTiles;
    pl.wide = pl.segs <= kSms && work > kNarrowTiles;
    pl.cluster_log2 = 0;
    if (pl.wide)
        while (pl.cluster_log2 < kMaxClusterLog2 && work > (per_block << pl.cluster_log2) / 2 &&
               pl.segs <= kClusters[pl.cluster_log2 + 1])
            ++pl.cluster_log2;
    // (where even clusters fill few SMs, a split takes over at half the length)
    const bool few = pl.wide && pl.segs << pl.cluster_log2 < kFewBlocks;
    pl.whole = work <= (pl.wide ? (per_block << pl.cluster_log2) / (few ? 2 : 1) : kWholeTiles);
    const size_t part_rows = pl.whole ? 0 : static_cast<size_t>(2) * kPagedWarps * pl.ctas * 8 * pl.nt;
    pl.part_l = pl.whole ? 0 : up(static_cast<size_t>(pl.segs) * sizeof(int2));
    pl.part_o = pl.part_l + up(part_rows * sizeof(float));
    pl.bytes = pl.part_o + part_rows * c.d * sizeof(float);
    return pl;
}

template <int D, int NT, bool F8, bool MOD>
cudaError_t launch_paged_t(const PagedArgs& a, const PagedPlan& pl, PagedParams& p, cudaStream_t stream) {
    constexpr auto kern = &fa_paged_kernel<D, NT, F8, 0, MOD>;
    constexpr auto kern_w = &fa_paged_kernel<D, NT, F8, kPagedWarps, MOD>;
    constexpr auto kern_w2 = &fa_paged_kernel<D, NT, F8, 2 * kPagedWarps, MOD>;
    constexpr int bytes = kPagedBytes<D, NT, F8, kPagedWarps, MOD>, bytes2 = kPagedBytes<D, NT, F8, 2 * kPagedWarps, MOD>;
    cudaError_t e = !pl.whole  ? set_max_dyn_smem_once<kern>(bytes)
                    : pl.wide ? set_max_dyn_smem_once<kern_w2>(bytes2)
                              : set_max_dyn_smem_once<kern_w>(bytes);
    if (e != cudaSuccess) return e;
    if (pl.whole) {
        const dim3 grid(static_cast<unsigned>(pl.segs << pl.cluster_log2));
        if (a.ev_start) cudaEventRecord(a.ev_start, stream);
        e = pl.wide ? launch_dependent_clusters(kern_w2, 1u << pl.cluster_log2, grid, dim3(2 * kThreads), bytes2, stream, p)
                    : launch_dependent(kern_w, grid, dim3(kThreads), bytes, stream, p);
        if (e == cudaSuccess && a.ev_stop) e = cudaEventRecord(a.ev_stop, stream);
        return e;
    }
    if (a.ev_start) cudaEventRecord(a.ev_start, stream);
    // (no more CTAs than a full table gives kMinTiles per warp)
    const int ctas = static_cast<int>(std::min<long long>(pl.ctas, pl.tiles * pl.rwarps / (kMinTiles * kPagedWarps) + 1));
    p.shares = ctas * (kPagedWarps / pl.rwarps);
    e = launch_dependent(kern, dim3(static_cast<unsigned>(ctas)), dim3(kThreads), bytes, stream, p);
    // pieces of an average segment of full tables
    const long long pieces = static_cast<long long>(ctas) * kPagedWarps / (pl.segs * pl.rwarps) + 1;
    const long long rows = std::min(p.G * p.Nq, 8 * NT * pl.rwarps);
    const unsigned segs = static_cast<unsigned>(pl.segs);
    if (e == cudaSuccess && pieces > kFewPieces) {
        // (a row's columns in one block while that block's warps suffice for the pieces)
        const long long groups = (std::min<long long>(pieces, kMaxResults) + 31) / 32;
        const unsigned z = groups * (D / 32) > kCombineWarps ? D / 32 : 1;
        const long long warps = std::min<long long>(kCombineWarps, groups * (D / 32 / z));
        e = launch_dependent(fa_paged_combine_kernel<D, NT, true>, dim3(segs, static_cast<unsigned>(rows), z),
                             dim3(static_cast<unsigned>(32 * warps)), 0, stream, p);
    } else if (e == cudaSuccess) {
        e = launch_dependent(fa_paged_combine_kernel<D, NT, false>, dim3(segs, static_cast<unsigned>((rows + 7) / 8)),
                             dim3(static_cast<unsigned>(32 * std::min(8ll, rows))), 0, stream, p);
    }
    if (e == cudaSuccess && a.ev_stop) e = cudaEventRecord(a.ev_stop, stream);
    return e;
}

template <bool MOD>
cudaError_t launch_paged(const PagedArgs& a, cudaStream_t stream) {
    const bool fp8 = a.cache.k_scale != nullptr;
    const PagedPlan pl = paged_plan(a.cache, a.H, a.Nq, a.window, a.sinks, fp8);
    PagedParams p;
    p.Q = static_cast<const __nv_bfloat16*>(a.Q);
    p.K = static_cast<const uint8_t*>(a.cache.K);
    p.V = static_cast<const uint8_t*>(a.cache.V);
    p.k_scale = a.cache.k_scale;
    p.v_scale = a.cache.v_scale;
    p.table = a.cache.page_table;
    p.lens = a.cache.lens;
    p.O = static_cast<__nv_bfloat16*>(a.O);
    p.LSE = a.LSE;
    uint8_t* ws = static_cast<uint8_t*>(a.workspace);
    p.seg = reinterpret_cast<int2*>(ws);
    p.part_l = reinterpret_cast<float*>(ws + pl.part_l);
    p.part_o = reinterpret_cast<float*>(ws + pl.part_o);
    p.q_sb = a.q_sb;
    p.q_sh = a.q_sh;
    p.q_sn = a.q_sn;
    p.o_sb = a.o_sb;
    p.o_sh = a.o_sh;
    p.o_sn = a.o_sn;
    p.B = a.cache.B;
    p.H = a.H;
    p.H_kv = a.cache.H_kv;
    p.G = a.H / a.cache.H_kv;
    p.Nq = a.Nq;
    p.rwarps = pl.rwarps;
    p.shares = 0;
    p.cluster_log2 = pl.cluster_log2;
    p.rgroups = pl.rgroups;
    p.num_pages = a.cache.num_pages;
    p.max_pages = a.cache.max_pages;
    p.shift = a.cache.shift;
    p.window = a.window;
    p.sinks = a.window > 0 ? a.sinks : 0;
    p.scale_log2 = a.tau * kLog2e;
    p.err = a.err;
    if constexpr (MOD) {
        p.cap_log2 = a.mod.softcap * kLog2e;
        p.cap_inv = a.mod.softcap > 0.f ? 1.f / p.cap_log2 : 0.f;
        p.slopes = a.mod.slopes;
        p.bias = a.mod.table;
        p.buckets = a.mod.buckets;
        p.bias_f32 = a.mod.table_f32;
        p.num_buckets = a.mod.num_buckets;
        p.far = a.mod.far;
    }
    const int key = (a.cache.d == 128 ? 4 : 0) + (fp8 ? 2 : 0) + (pl.nt - 1);
    switch (key) {
        case 0: return launch_paged_t<64, 1, false, MOD>(a, pl, p, stream);
        case 1: return launch_paged_t<64, 2, false, MOD>(a, pl, p, stream);
        case 2: return launch_paged_t<64, 1, true, MOD>(a, pl, p, stream);
        case 3: return launch_paged_t<64, 2, true, MOD>(a, pl, p, stream);
        case 4: return launch_paged_t<128, 1, false, MOD>(a, pl, p, stream);
        case 5: return launch_paged_t<128, 2, false, MOD>(a, pl, p, stream);
        case 6: return launch_paged_t<128, 1, true, MOD>(a, pl, p, stream);
        default: return launch_paged_t<128, 2, true, MOD>(a, pl, p, stream);
    }
}

}  // namespace
}  // namespace fa
