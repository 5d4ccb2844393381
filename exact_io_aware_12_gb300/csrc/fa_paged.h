// Index arithmetic of the paged key/value cache, shared by its kernels.  Plain
// C++: every function also runs on the host, where the tests call it.
//
// Sequence b's key j lives in page table[b][j / page_size], row j % page_size; page
// sizes are powers of two (shift = log2).  Lengths and page numbers are device data,
// so the kernels check each against the table's and the cache's bounds before use.
#pragma once

#include <cstdint>

#if defined(__CUDACC__)
#define FA_HD __host__ __device__ __forceinline__
#else
#define FA_HD inline
#endif

namespace fa {

constexpr int kPagedMinPage = 16, kPagedMaxPage = 256;
constexpr long long kPagedMaxKeys = 1ll << 30;  // of one sequence: key numbers plus a tile fit an int
// Keys per tile of the attention kernel, and warps of a block.
constexpr int kPagedTile = 16, kPagedWarps = 4;

// The page of key `key`, or -1 where the key lies outside the table or the table
// names no page of the cache.
FA_HD int page_of(const int* table_row, int max_pages, int num_pages, int shift, long long key) {
    if (key < 0 || (key >> shift) >= max_pages) return -1;
    const int pg = table_row[key >> shift];
    return pg >= 0 && pg < num_pages ? pg : -1;
}

// The keys that a step's rows (the last nq positions of a sequence of len keys) see, as
// a list of 16-key tiles: the tiles [0, ns) of the sinks that lie before the first row's
// window, then the tiles [lo, lo + n - ns) from that window's first key to the end.
struct PagedRange {
    int len;   // keys, inside the table
    int lo;    // first tile of the window part
    int ns;    // sink tiles before it
    int n;     // tiles in the list
    // first key of list entry s
    FA_HD int key0(int s) const { return kPagedTile * (s < ns ? s : lo + s - ns); }
};

FA_HD PagedRange paged_range(int len, int nq, int window, int sinks) {
    PagedRange r;
    r.len = len;
    const long long first = window > 0 ? static_cast<long long>(len) - nq - window + 1 : 0;
    r.lo = first > 0 ? static_cast<int>(first) / kPagedTile : 0;
    const int sink_tiles = sinks / kPagedTile + (sinks % kPagedTile != 0);
    r.ns = sink_tiles < r.lo ? sink_tiles : r.lo;
    r.n = r.ns + len / kPagedTile + (len % kPagedTile != 0) - r.lo;
    return r;
}

// Tiles counted for a segment: its own and, behind them, kSegmentTiles that stand for the
// time in which a warp changes segments (and make an empty sequence count too).  (1 and 6
// were slower on uneven batches.)
constexpr int kSegmentTiles = 3;
FA_HD int paged_tiles(const PagedRange& r) { return r.n + kSegmentTiles; }

// `total` tiles cut into `shares` shares that differ by at most one tile, the longer ones
// first: share c takes [start(c), start(c + 1)); of(x) is the share that takes tile x.
// 32-bit throughout: a 64-bit division costs a warp a few hundred cycles.
struct Shares {
    uint32_t base, rem;
    FA_HD Shares(uint32_t total, uint32_t shares) : base(total / shares), rem(total % shares) {}
    FA_HD uint32_t start(uint32_t c) const { return c * base + (c < rem ? c : rem); }
    FA_HD uint32_t of(uint32_t x) const {
        const uint32_t longer = rem * (base + 1);
        return x < longer ? x / (base + 1) : rem + (x - longer) / base;
    }
};

// Tiles of a share, at least: below, its start and end cost more than they save (one
// sequence of 1500 keys, 8 key heads: 1 tile 11.2 us, 2 9.6, 4 10.1).
constexpr int kMinTiles = 2;
// Pieces of a segment: more cost the combine kernel more than they save (one segment of
// 131072 keys: 512 pieces 19.5 us, 1024 17.4, 2048 21.8).
constexpr int kMaxResults = 1024;
// Shares that `total` tiles of `segs` segments are cut into, for `warps` takers: at least
// one, none of them empty.  (Past 2^20 segments the last bound is beyond any number of takers.)
FA_HD uint32_t share_count(uint32_t warps, uint32_t total, uint32_t segs) {
    const uint32_t few = total / kMinTiles, most = segs < (1u << 20) ? segs * kMaxResults : ~0u;
    const uint32_t n = warps < few ? warps : few;
    return n > most ? most : n > 0 ? n : 1u;
}

// A frequency (radians per position, the bits of a double) as turns per position: the
// fractional part in units of 2^-64, so that position * result mod 2^64 is the angle's
// exact place on the circle however far the position.  Integer arithmetic throughout
// (the GPU has few fp64 units): with m the 53-bit significand and 2 / pi as a 64-bit
// fraction, turns * 2^64 = m * (2 / pi) 2^64 * 2^(exponent - 1077).  Infinities and NaN give 0.
FA_HD uint64_t turn_fraction(uint64_t bits) {
    constexpr uint64_t kTwoOverPi = 0xA2F9836E4E441529ull;
    const int e = static_cast<int>((bits >> 52) & 0x7ff);
    if (e == 0x7ff) return 0;
    const uint64_t m = (bits & 0xfffffffffffffull) | (e > 0 ? 1ull << 52 : 0);
    const int s = 1077 - (e > 0 ? e : 1);
    const unsigned __int128 p = static_cast<unsigned __int128>(m) * kTwoOverPi;
    const uint64_t x = s >= 128 ? 0
                     : s >= 0   ? static_cast<uint64_t>(p >> s)
                     : s > -64  ? static_cast<uint64_t>(p << -s)
                                : 0;
    return bits >> 63 ? 0 - x : x;
}

// The scale of an 8-bit page: the exponent e of the smallest power of two 2^e with
// bound <= 448 * 2^e, from the bits of the fp32 bound (>= 0; 448 = 1.75 * 2^8), kept
// within [-100, 121], where 2^e and 2^-e are normal fp32 numbers.  A power of two loses
// nothing against any other scale (e4m3 keeps 3 mantissa bits wherever its normal range
// lies) and makes rescaling exact except where a value falls among the subnormals.
FA_HD int page_scale_exp(uint32_t bound_bits) {
    if (bound_bits >= 0x7f800000u) return 121;  // no finite bound
    const int x = static_cast<int>(bound_bits >> 23) - 127;
    const int e = x - 8 + ((bound_bits & 0x7fffffu) > 0x600000u ? 1 : 0);
    return e < -100 ? -100 : e > 121 ? 121 : e;
}

// Pages that n new tokens reach from position `past`, and the first unit of sequence b
// when every sequence is given n / page_size + 2 units of which it uses that many: the
// list needs only the running token counts cu, not the lengths.
FA_HD int pages_reached(long long past, int n, int shift) {
    return n > 0 ? static_cast<int>(((past + n - 1) >> shift) - (past >> shift)) + 1 : 0;
}
FA_HD long long first_unit(long long cu_b, int b, int shift) { return (cu_b >> shift) + 2ll * b; }

// Rows of d elements at [T][H] strides, first at `at`, all in elements of one address space.
struct RowSet {
    long long at, st, sh;
    int T, H;
    FA_HD long long span(int d) const { return (T - 1) * st + (H - 1) * sh + d; }
};
// Whether a row of `a` and one of `b` (as many tokens, strides not negative) share an element:
// slices of one projection's output may lie between one another.  Where the spans overlap and
// the token strides differ, or heads' strides do and pairs of heads are many, yes without a
// closer look.
FA_HD bool rows_meet(const RowSet& a, const RowSet& b, int d) {
    const long long delta = b.at - a.at;
    if (delta >= a.span(d) || -delta >= b.span(d)) return false;
    const long long st = a.T > 1 ? a.st : 0, last = a.T - 1;
    if (a.T > 1 && a.st != b.st) return true;
    const bool alike = a.sh == b.sh;
    if (!alike && static_cast<long long>(a.H) * b.H > (1 << 16)) return true;
    // (alike: only the difference of the heads counts)
    for (int ha = 0; ha < a.H; ++ha)
        for (int hb = 0; hb < (alike && ha > 0 ? 1 : b.H); ++hb) {
            // rows of tokens t and t + m are off + m st apart
            const long long off = delta + hb * b.sh - ha * a.sh;
            long long m = st > 0 ? -off / st : 0;  // the nearest, or next to it
            m = m < -last ? -last : m > last ? last : m;
            for (long long k = m - 1; k <= m + 1; ++k) {
                if (k < -last || k > last) continue;
                const long long gap = off + k * st;
                if (gap < d && -gap < d) return true;
            }
        }
    return false;
}

}  // namespace fa
