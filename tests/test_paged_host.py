"""The paged cache without a GPU: the index arithmetic that its kernels share (compiled here as
plain C++), refusals of the entry points, and checks of the Python ones."""
import ctypes
import math
import os
import struct
import subprocess

import pytest
import torch

from exact_io_aware_12_gb300 import _lib, api
from tests import _plain

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x7F0000000000
GB = 1 << 30

SHIM = r'''
#include "fa_paged.h"
using namespace fa;
extern "C" {
int t_page_of(const int* t, int mp, int np, int sh, long long k) { return page_of(t, mp, np, sh, k); }
void t_range(int len, int nq, int w, int s, int* o) {
    const PagedRange r = paged_range(len, nq, w, s);
    o[0] = r.lo; o[1] = r.ns; o[2] = r.n; o[3] = paged_tiles(r);
}
int t_key0(int len, int nq, int w, int s, int i) { return paged_range(len, nq, w, s).key0(i); }
long long t_start(long long c, long long t, long long s) { return Shares(t, s).start(c); }
long long t_share(long long x, long long t, long long s) { return Shares(t, s).of(x); }
uint32_t t_count(uint32_t w, uint32_t t, uint32_t s) { return share_count(w, t, s); }
uint64_t t_turn(uint64_t b) { return turn_fraction(b); }
int t_exp(uint32_t b) { return page_scale_exp(b); }
int t_reached(long long p, int n, int sh) { return pages_reached(p, n, sh); }
long long t_unit(long long c, int b, int sh) { return first_unit(c, b, sh); }
int t_meet(const long long* a, const long long* b, int t, int ha, int hb, int d) {
    return rows_meet({a[0], a[1], a[2], t, ha}, {b[0], b[1], b[2], t, hb}, d);
}
}
'''


@pytest.fixture(scope="module")
def shim(tmp_path_factory):
    d = tmp_path_factory.mktemp("paged")
    src, lib = d / "shim.cpp", d / "shim.so"
    src.write_text(SHIM)
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-fsanitize=undefined",
                    "-fno-sanitize-recover=undefined", "-static-libubsan",
                    "-I", os.path.join(ROOT, "exact_io_aware_12_gb300", "csrc"), str(src), "-o", str(lib)], check=True)
    L = ctypes.CDLL(str(lib))
    LL, I = ctypes.c_longlong, ctypes.c_int
    L.t_page_of.argtypes = [ctypes.POINTER(I), I, I, I, LL]
    L.t_start.argtypes = L.t_share.argtypes = [LL, LL, LL]
    L.t_start.restype = L.t_share.restype = L.t_unit.restype = LL
    L.t_turn.argtypes, L.t_turn.restype = [ctypes.c_uint64], ctypes.c_uint64
    L.t_exp.argtypes = [ctypes.c_uint32]
    L.t_reached.argtypes = [LL, I, I]
    L.t_unit.argtypes = [LL, I, I]
    L.t_count.argtypes, L.t_count.restype = [ctypes.c_uint32] * 3, ctypes.c_uint32
    return L


def test_bad_pages_and_positions_name_no_page(shim):
    t = (ctypes.c_int * 4)(2, -1, 7, 2 ** 31 - 1)
    at = lambda key, pages=7, shift=4: shim.t_page_of(t, 4, pages, shift, key)
    assert at(0) == 2 and at(15) == 2
    assert at(16) == -1                    # entry -1
    assert at(32) == -1 and at(32, pages=8) == 7   # entry == num_pages, and just inside
    assert at(48) == -1                    # entry far outside
    assert at(64) == -1 and at(2 ** 40) == -1 and at(-1) == -1 and at(-2 ** 40) == -1  # outside the table
    assert at(2 ** 31 + 5) == -1


@pytest.mark.parametrize("nq,window,sinks", [(1, 0, 0), (4, 0, 0), (1, 1, 0), (1, 40, 5), (4, 64, 17), (8, 100, 130), (3, 16, 16)])
def test_tile_lists_hold_every_visible_key_once(shim, nq, window, sinks):
    o = (ctypes.c_int * 4)()
    for length in list(range(0, 200)) + [511, 512, 513, 1000]:
        shim.t_range(length, nq, window, sinks, o)
        lo, ns, n, tiles = o
        starts = [shim.t_key0(length, nq, window, sinks, i) for i in range(n)]
        assert len(set(starts)) == n and all(k % 16 == 0 and 0 <= k < max(length, 1) for k in starts)
        assert tiles > n
        see = _plain.visible(min(nq, length), length, window, sinks).any(0) if length else torch.zeros(0)
        held = {k + i for k in starts for i in range(16)}
        assert all(int(j) in held for j in see.nonzero().flatten())
        # and no tile without a visible key, but where the window's first row looks further back than row 0 can
        if length >= nq:
            assert all(any(k + i < length and see[k + i] for i in range(16)) for k in starts)


def test_extreme_lengths_and_windows_do_not_overflow(shim):
    o = (ctypes.c_int * 4)()
    for length in (0, 1, 2 ** 31 - 1, 2 ** 31 - 17):
        for window in (0, 1, 2 ** 30):
            for sinks in (0, 1, 2 ** 30):
                shim.t_range(length, 8, window, sinks, o)
                assert o[2] >= 0 and o[3] >= 1


@pytest.mark.parametrize("total,shares", [(1, 1), (10, 3), (1000, 608), (607, 607), (12345, 304), (2 ** 31 - 1, 608)])
def test_shares_cover_every_step_once(shim, total, shares):
    assert shim.t_start(0, total, shares) == 0 and shim.t_start(shares, total, shares) == total
    for c in range(shares):
        a, b = shim.t_start(c, total, shares), shim.t_start(c + 1, total, shares)
        assert a < b
        for x in {a, (a + b) // 2, b - 1}:
            assert shim.t_share(x, total, shares) == c


def test_share_counts(shim):
    assert shim.t_count(608, 10 ** 6, 8) == 608
    assert shim.t_count(608, 100, 8) == 50            # two tiles each
    assert shim.t_count(608, 1, 1) == 1               # never none
    assert shim.t_count(1824, 10 ** 6, 1) == 1024     # pieces of one segment
    for segs in (2 ** 20 - 1, 2 ** 20, 2 ** 23, 2 ** 29, 2 ** 31 - 1):   # beyond 32 bits times that
        assert shim.t_count(1824, 2 ** 31 - 1, segs) == 1824


def test_turns_are_exact_far_out(shim):
    from fractions import Fraction
    # pi to 40 digits
    pi = Fraction(31415926535897932384626433832795028841972, 10 ** 40)
    for f in [1.0, 0.5, 10000.0 ** (-2 / 128), 1e-4, 3.7e-9, 2.5, 1234.5, -0.3, 5e-324, 0.0, 1e-30, 2.0 ** 60]:
        got = shim.t_turn(struct.unpack("<Q", struct.pack("<d", f))[0])
        for p in (1, 131072, 2 ** 24, 2 ** 31 - 1):
            want = Fraction(f) * p / (2 * pi)
            want -= math.floor(want)
            have = Fraction(got * p % 2 ** 64, 2 ** 64)
            off = abs(want - have)
            off = min(off, 1 - off)
            # 2 / pi is held to 2^-64 of itself, the turns to 2^-64, both times the position
            assert off <= abs(Fraction(f)) * p * Fraction(1, 2 ** 64) + Fraction(p, 2 ** 63), (f, p, float(off))
    for bits in (0x7FF0000000000000, 0xFFF0000000000000, 0x7FF8000000000000):
        assert shim.t_turn(bits) == 0


def test_page_scales(shim):
    bits = lambda x: struct.unpack("<I", struct.pack("<f", x))[0]
    for x in [0.0, 1e-45, 1e-30, 1.0, 447.9, 448.0, 448.00003, 449.0, 896.0, 896.1, 1.75, 1.7500001, 3e38, 3.4e38]:
        x32 = struct.unpack("<f", struct.pack("<f", x))[0]
        assert 2.0 ** shim.t_exp(bits(x)) == _plain.scale_of(x32), x
    assert shim.t_exp(bits(math.inf)) == 121


def test_units_fit_every_split_of_tokens(shim):
    """Each sequence's pages fit the units it is given, whatever its lengths and the others'."""
    g = torch.Generator().manual_seed(3)
    for shift in (4, 6):
        for _ in range(300):
            n = torch.randint(0, 100, (6,), generator=g).tolist()
            cu = [0]
            for x in n:
                cu.append(cu[-1] + x)
            for b in range(6):
                room = shim.t_unit(cu[b + 1], b + 1, shift) - shim.t_unit(cu[b], b, shift)
                for past in (0, 1, 15, 16, 63, 2 ** 31 - 60):
                    used = shim.t_reached(past, n[b], shift)
                    assert used <= room
                    assert used == len({(past + i) >> shift for i in range(n[b])})
            assert shim.t_unit(cu[6], 6, shift) <= (cu[6] >> shift) + 12


def cache(fp8=False, **kw):
    c = dict(K=FAKE, V=FAKE + GB, k_scale=FAKE + 2 * GB if fp8 else None, v_scale=FAKE + 3 * GB if fp8 else None,
             page_table=FAKE + 4 * GB, lens=FAKE + 5 * GB, B=2, H_kv=2, d=64, num_pages=8, page_size=16, max_pages=4000)
    c.update(kw)
    return _lib.PagedCache(*(c[n] for n, _ in _lib.PagedCache._fields_))


BAD_CACHES = [
    (dict(K=None), _lib.FA_ERR_INVALID_ARG),
    (dict(V=FAKE + GB + 8), _lib.FA_ERR_INVALID_ARG),
    (dict(V=FAKE + 64), _lib.FA_ERR_INVALID_ARG),               # V overlaps K
    (dict(page_table=None), _lib.FA_ERR_INVALID_ARG),
    (dict(lens=FAKE + 5 * GB + 2), _lib.FA_ERR_INVALID_ARG),
    (dict(B=-1), _lib.FA_ERR_INVALID_ARG),
    (dict(max_pages=0), _lib.FA_ERR_INVALID_ARG),
    (dict(num_pages=0), _lib.FA_ERR_INVALID_ARG),
    (dict(d=96), _lib.FA_ERR_UNSUPPORTED),
    (dict(page_size=8), _lib.FA_ERR_UNSUPPORTED),
    (dict(page_size=48), _lib.FA_ERR_UNSUPPORTED),
    (dict(page_size=512), _lib.FA_ERR_UNSUPPORTED),
    (dict(max_pages=2 ** 26 + 1), _lib.FA_ERR_UNSUPPORTED),
    (dict(k_scale=FAKE + 6 * GB, v_scale=None), _lib.FA_ERR_INVALID_ARG),
    (dict(B=0), _lib.FA_OK),
]


def append(c, fp8=False, **kw):
    a = dict(k=FAKE + 8 * GB, k_st=128, k_sh=64, v=FAKE + 9 * GB, v_st=128, v_sh=64, T=4, cu_new=FAKE + 10 * GB,
             q=FAKE + 11 * GB, q_st=256, q_sh=64, q_out=FAKE + 12 * GB, qo_st=256, qo_sh=64, H=4,
             inv_freq=FAKE + 13 * GB, rot=64, interleaved=0, stream=None)
    a.update(kw)
    return (_lib.fa_kv_append_fp8 if fp8 else _lib.fa_kv_append)(c, *a.values())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kw,code", BAD_CACHES)
def test_append_refuses_bad_caches(kw, code, fp8):
    assert append(cache(fp8, **kw), fp8) == code


NO_Q = dict(q=None, q_out=None, H=0)


@pytest.mark.parametrize("kw,code", [
    (dict(k=None), _lib.FA_ERR_INVALID_ARG),
    (dict(v=FAKE + 9 * GB + 2), _lib.FA_ERR_INVALID_ARG),
    (dict(k_sh=60), _lib.FA_ERR_INVALID_ARG),       # not a multiple of 8
    (dict(k_st=-128), _lib.FA_ERR_INVALID_ARG),
    (dict(k_st=2 ** 62), _lib.FA_ERR_INVALID_ARG),   # beyond any address
    (dict(v_st=4), _lib.FA_ERR_INVALID_ARG),
    (dict(k=FAKE + 16), _lib.FA_ERR_INVALID_ARG),               # inside the cache
    (dict(T=-1), _lib.FA_ERR_INVALID_ARG),
    (dict(T=3, cu_new=None), _lib.FA_ERR_INVALID_ARG),          # no even split over two sequences
    (dict(cu_new=FAKE + 10 * GB + 1), _lib.FA_ERR_INVALID_ARG),
    (dict(rot=24), _lib.FA_ERR_INVALID_ARG),
    (dict(rot=80), _lib.FA_ERR_INVALID_ARG),                    # wider than the head
    (dict(rot=0), _lib.FA_ERR_INVALID_ARG),                     # frequencies without rotation
    (dict(inv_freq=None), _lib.FA_ERR_INVALID_ARG),
    (dict(inv_freq=None, rot=0), _lib.FA_ERR_INVALID_ARG),      # queries without rotation
    (dict(inv_freq=FAKE + 13 * GB + 4), _lib.FA_ERR_INVALID_ARG),
    (dict(interleaved=2), _lib.FA_ERR_INVALID_ARG),
    (dict(q_out=None), _lib.FA_ERR_INVALID_ARG),
    (dict(H=0), _lib.FA_ERR_INVALID_ARG),
    (dict(q_out=FAKE + 11 * GB + 32), _lib.FA_ERR_INVALID_ARG),  # neither in place nor apart
    (dict(q_out=FAKE + 11 * GB, qo_st=512), _lib.FA_ERR_INVALID_ARG),
    (dict(qo_st=0), _lib.FA_ERR_INVALID_ARG),     # rows on top of each other
    (dict(q_out=FAKE + 8 * GB), _lib.FA_ERR_INVALID_ARG),       # over k
    (dict(q_out=FAKE + 5 * GB), _lib.FA_ERR_INVALID_ARG),       # over lens
    (dict(q_out=FAKE + 4 * GB + 16), _lib.FA_ERR_INVALID_ARG),  # over the page table
    (dict(inv_freq=FAKE + 128), _lib.FA_ERR_INVALID_ARG),       # inside the cache
    (dict(cu_new=FAKE + GB), _lib.FA_ERR_INVALID_ARG),
    (dict(T=0), _lib.FA_OK),
    (dict(T=0, k=None, v=None, **NO_Q), _lib.FA_OK),
])
@pytest.mark.parametrize("fp8", [False, True])
def test_append_refuses(kw, code, fp8):
    assert append(cache(fp8), fp8, **kw) == code


def test_a_cache_over_its_own_table_or_scales_is_refused():
    assert append(cache(page_table=FAKE + 64)) == _lib.FA_ERR_INVALID_ARG
    assert append(cache(lens=FAKE + GB)) == _lib.FA_ERR_INVALID_ARG
    assert append(cache(True, k_scale=FAKE + 64), True) == _lib.FA_ERR_INVALID_ARG
    assert append(cache(True, k_scale=FAKE + 3 * GB + 4), True) == _lib.FA_ERR_INVALID_ARG
    assert append(cache(True, v_scale=FAKE + 5 * GB), True) == _lib.FA_ERR_INVALID_ARG


def test_queries_without_key_heads_are_refused():
    assert append(cache(H_kv=0)) == _lib.FA_ERR_INVALID_ARG
    assert append(cache(H_kv=0), **NO_Q) == _lib.FA_OK
    assert paged(cache(H_kv=0)) == _lib.FA_ERR_INVALID_ARG
    assert paged(cache(H_kv=0), H=0) == _lib.FA_OK


def test_a_cache_of_the_other_kind_is_refused():
    assert append(cache(True), False) == _lib.FA_ERR_INVALID_ARG
    assert append(cache(False), True) == _lib.FA_ERR_INVALID_ARG
    assert paged(cache(True), False) == _lib.FA_ERR_INVALID_ARG
    assert paged(cache(False), True) == _lib.FA_ERR_INVALID_ARG
    assert paged(None) == _lib.FA_ERR_INVALID_ARG


def paged(c, fp8=False, **kw):
    a = dict(Q=FAKE + 8 * GB, q_sb=256, q_sh=64, q_sn=64, O=FAKE + 9 * GB, o_sb=256, o_sh=64, o_sn=64,
             LSE=FAKE + 10 * GB, H=4, Nq=1, tau=0.125, window=0, sinks=0, workspace=FAKE + 11 * GB, workspace_bytes=GB, stream=None)
    a.update(kw)
    return (_lib.fa_fwd_paged_fp8 if fp8 else _lib.fa_fwd_paged)(c, *a.values())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kw,code", BAD_CACHES)
def test_paged_refuses_bad_caches(kw, code, fp8):
    assert paged(cache(fp8, **kw), fp8) == code


@pytest.mark.parametrize("kw,code", [
    (dict(Q=None), _lib.FA_ERR_INVALID_ARG),
    (dict(O=FAKE + 9 * GB + 4), _lib.FA_ERR_INVALID_ARG),
    (dict(q_sh=63), _lib.FA_ERR_INVALID_ARG),
    (dict(LSE=None), _lib.FA_ERR_INVALID_ARG),
    (dict(o_sh=0), _lib.FA_ERR_INVALID_ARG),        # heads on top of each other
    (dict(o_sb=128), _lib.FA_ERR_INVALID_ARG),       # sequences overlap
    (dict(H=3), _lib.FA_ERR_INVALID_ARG),                           # not a multiple of H_kv
    (dict(H=-4), _lib.FA_ERR_INVALID_ARG),
    (dict(Nq=9), _lib.FA_ERR_UNSUPPORTED),
    (dict(tau=0.0), _lib.FA_ERR_INVALID_ARG),
    (dict(tau=math.nan), _lib.FA_ERR_INVALID_ARG),
    (dict(window=-1), _lib.FA_ERR_INVALID_ARG),
    (dict(sinks=4), _lib.FA_ERR_INVALID_ARG),                       # sinks without a window
    (dict(window=4, sinks=-1), _lib.FA_ERR_INVALID_ARG),
    (dict(workspace_bytes=1000), _lib.FA_ERR_WORKSPACE),
    (dict(workspace=FAKE + 11 * GB + 8), _lib.FA_ERR_INVALID_ARG),
    (dict(workspace=FAKE + 9 * GB), _lib.FA_ERR_INVALID_ARG),       # over O
    (dict(O=FAKE + 8 * GB), _lib.FA_ERR_INVALID_ARG),               # over Q
    (dict(LSE=FAKE + 5 * GB), _lib.FA_ERR_INVALID_ARG),             # over lens
    (dict(O=FAKE), _lib.FA_ERR_INVALID_ARG),                        # over the cache
    (dict(Nq=0), _lib.FA_OK),
    (dict(H=0), _lib.FA_OK),
])
@pytest.mark.parametrize("fp8", [False, True])
def test_paged_refuses(kw, code, fp8):
    assert paged(cache(fp8), fp8, **kw) == code


def test_too_many_tiles_are_refused():
    assert paged(cache(B=4096, H_kv=2, max_pages=2 ** 22)) == _lib.FA_ERR_UNSUPPORTED
    # a segment counts as three tiles more than its keys fill
    assert paged(cache(B=2 ** 23, H_kv=2, max_pages=125), q_sb=512, o_sb=512) == _lib.FA_ERR_UNSUPPORTED


def test_workspace_sizes():
    size = lambda H=8, Nq=1, window=0, sinks=0, **kw: _lib.fa_paged_workspace_size(
        cache(**dict(dict(max_pages=4096), **kw)), H, Nq, window, sinks)
    assert size() > 0 and size(fp8=True) > 0
    assert size(max_pages=4) == 0                     # short tables need none
    assert size(window=100, sinks=4) == 0             # nor short windows
    for bad in (dict(H=3), dict(Nq=9), dict(B=0), dict(d=96), dict(page_size=48), dict(window=-1), dict(H=0)):
        assert size(**bad) == 0
    assert _lib.fa_paged_workspace_size(None, 8, 1, 0, 0) == 0
    q, kc = torch.empty(2, 8, 1, 64, dtype=torch.bfloat16), torch.empty(8, 2, 16, 64, dtype=torch.bfloat16)
    assert api.paged_workspace_bytes(q, kc, torch.empty(2, 4096)) == size()
    assert api.paged_workspace_bytes(q, kc.to(torch.uint8), torch.empty(2, 4096)) == size(fp8=True)


@pytest.mark.parametrize("kw,code", [
    (dict(window=0), _lib.FA_ERR_INVALID_ARG),
    (dict(window=-3), _lib.FA_ERR_INVALID_ARG),
    (dict(sinks=-1), _lib.FA_ERR_INVALID_ARG),
    (dict(d=96), _lib.FA_ERR_UNSUPPORTED),
    (dict(N=0), _lib.FA_OK),
])
def test_sinks_argument_checks(kw, code):
    a = dict(B=1, H=1, N=128, d=64, tau=0.125, window=8, sinks=2)
    a.update(kw)
    p = [FAKE + i * GB for i in range(10)]
    assert _lib.fa_fwd_sinks(*p[:5], *a.values(), None) == code
    assert _lib.fa_bwd_sinks(*p[:6], *p[6:9], p[9], GB, *a.values(), None) == code


def test_python_checks():
    x = torch.zeros(1, 1, 128, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="sinks need a window"):
        api.fwd(x, x, x, True, sinks=4)
    with pytest.raises(ValueError, match="sinks need a window"):
        api.bwd(x, x, x, x, x, x, True, sinks=4)
    with pytest.raises(ValueError, match="causal"):
        api.fwd(x, x, x, False, window=8, sinks=4)
    with pytest.raises(ValueError, match="causal"):
        api.bwd(x, x, x, x, x, x, False, window=8, sinks=4)
    with pytest.raises(ValueError, match="CUDA"):
        api.fwd(x, x, x, True, window=8, sinks=4)
    with pytest.raises(ValueError, match="CUDA"):
        api.bwd(x, x, x, x, x, x, True, window=8, sinks=4)
    with pytest.raises(TypeError):
        api.fwd(x, x, None, True, window=8, sinks=4)
    kc = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    tb, ln = torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    q = torch.zeros(2, 4, 1, 64, dtype=torch.bfloat16)
    new = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    sc = torch.ones(4, 2)
    for args, kw, what in [
        ((q, kc, kc, tb, ln), {}, "CUDA"),
        ((q, kc, kc, tb.long(), ln), {}, "int32"),
        ((q, kc, kc, tb, ln[:1]), {}, "lens"),
        ((q, kc, kc[:2], tb, ln), {}, "alike"),
        ((q, kc, kc, tb, ln), dict(k_scale=sc), "both scales"),
        ((q, kc, kc, tb, ln), dict(k_scale=sc, v_scale=sc), "e4m3"),
        ((q, kc.view(torch.uint8), kc.view(torch.uint8), tb, ln), {}, "bf16"),
        ((q, kc.to(torch.uint8), kc.to(torch.uint8), tb, ln), dict(k_scale=sc[:2], v_scale=sc[:2]), "scales"),
    ]:
        with pytest.raises(ValueError, match=what):
            api.fwd_paged(*args, **kw)
    with pytest.raises(ValueError, match="CUDA"):
        api.kv_append(new, new, kc, kc, tb, ln)


def test_rows_that_meet(shim):
    """Against sets of elements: slices of one tensor in every order, rows that touch, tokens' strides
    smaller than a token's heads, single tokens."""
    g = torch.Generator().manual_seed(5)
    r = lambda lo, hi: int(torch.randint(lo, hi + 1, (1,), generator=g))
    d, seen = 4, set()

    def rows(x, t, h):
        return {x[0] + i * x[1] + j * x[2] + e for i in range(t) for j in range(h) for e in range(d)}
    for _ in range(6000):
        t, ha, hb = r(1, 4), r(1, 4), r(1, 3)
        a = [0, r(0, 40), r(0, 14)]
        b = [r(-70, 70), a[1] if r(0, 4) else r(0, 40), a[2] if r(0, 1) else r(0, 14)]
        want = bool(rows(a, t, ha) & rows(b, t, hb))
        LL3 = ctypes.c_longlong * 3
        got = bool(shim.t_meet(LL3(*a), LL3(*b), t, ha, hb, d))
        assert got == want or (got and t > 1 and a[1] != b[1]), (a, b, t, ha, hb)
        seen.add((got, want, a[2] == b[2]))
    assert len(seen) >= 5
    LL3 = ctypes.c_longlong * 3
    x = lambda at, st=3 * 64 * 32, sh=64: LL3(at, st, sh)
    assert not shim.t_meet(x(0), x(32 * 64), 2 ** 21, 32, 32, 64)          # [T][q heads | k heads | v heads]
    assert not shim.t_meet(x(0, sh=192), x(64, sh=192), 2 ** 21, 32, 32, 64)   # [T][head][q, k, v]
    assert shim.t_meet(x(0), x(31 * 64), 2 ** 21, 32, 32, 64)


@pytest.mark.parametrize("fp8", [False, True])
def test_queries_turned_in_place_over_the_keys_are_refused(fp8):
    q = dict(q=FAKE + 8 * GB, q_out=FAKE + 8 * GB, q_st=256, qo_st=256, H=2)
    assert append(cache(fp8), fp8, k_st=256, **q) == _lib.FA_ERR_INVALID_ARG                       # k itself
    assert append(cache(fp8), fp8, k=FAKE + 8 * GB + 128, k_st=256, **q) == _lib.FA_ERR_INVALID_ARG  # its second head
    q["q"] = q["q_out"] = FAKE + 9 * GB
    assert append(cache(fp8), fp8, v_st=256, **q) == _lib.FA_ERR_INVALID_ARG
    assert append(cache(fp8), fp8, v=FAKE + 9 * GB + 256, v_st=384, **q) == _lib.FA_ERR_INVALID_ARG  # other token strides


@pytest.mark.parametrize("scale", ["k_scale", "v_scale"])
def test_scales_over_the_new_rows_are_refused(scale):
    for at in (FAKE + 8 * GB, FAKE + 9 * GB + 64, FAKE + 11 * GB + 4):   # k, v and q
        assert append(cache(True, **{scale: at}), True) == _lib.FA_ERR_INVALID_ARG


def test_clusters_that_run_at_a_time():
    """3000 keys: whole segments by clusters of four blocks up to the 36 that the machine holds at a
    time, split from there on (two blocks are too few)."""
    size = lambda B: _lib.fa_paged_workspace_size(cache(B=B, H_kv=1, d=128, page_size=64, max_pages=47), 4, 1, 0, 0)
    assert [size(B) > 0 for B in (8, 15, 16, 19, 36, 37, 38, 39)] == [False] * 5 + [True] * 3
