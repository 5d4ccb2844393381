"""GPU parity of fa_kv_append and fa_kv_append_fp8 with the plain 64-bit form.

Tolerances.  A rotated value is formed in fp32 from exact bf16 inputs, x cos - y sin: the two
products and the difference round three times (2^-24 each, relative to |x| + |y|), the cosines
are sincospif's of an angle held to 2^-24 of a half turn (off by pi 2^-24 plus two units of
2^-24): together less than 2^-20 (|x| + |y|).  Rounding to bf16 adds 2^-8 |value|, to e4m3
2^-4 |value| + 2^-10 scale (half the subnormals' step).  What does not turn is copied or rounded
once from exact values: equal to the last bit.  Scales are powers of two of exact maxima: equal."""
import math

import pytest
import torch

from exact_io_aware_12_gb300 import api, _lib
from tests import _plain

pytestmark = pytest.mark.gpu
DEV = "cuda"
FP32_TURN = 2.0 ** -20


def build(past, new, Hkv, H, d, page, fp8, seed, rows_behind=0):
    g = torch.Generator().manual_seed(seed)
    P, table = _plain.make_pages([p + n for p, n in zip(past, new)], page, g)
    T = sum(new) + rows_behind
    x = torch.randn(T, H + 2 * Hkv, d, generator=g)
    x[:, H:H + Hkv] *= torch.exp(torch.randn(Hkv, d, generator=g))
    x = x.to(torch.bfloat16)
    if fp8:
        kc, vc = (torch.randint(0, 256, (P, Hkv, page, d), generator=g, dtype=torch.int64).to(torch.uint8) for _ in "kv")
        for c in (kc, vc):   # no NaN codes
            c[(c & 0x7F) == 0x7F] = 0x7E
        ks, vs = (2.0 ** torch.randint(-12, -5, (P, Hkv), generator=g).float() for _ in "kv")
    else:
        kc, vc = (torch.randn(P, Hkv, page, d, generator=g).to(torch.bfloat16) for _ in "kv")
        ks = vs = None
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    return dict(q=x[:, :H], k=x[:, H:H + Hkv], v=x[:, H + Hkv:], kc=kc, vc=vc, ks=ks, vs=vs, table=table,
                lens=torch.tensor(past, dtype=torch.int32), cu=torch.tensor(cu, dtype=torch.int32))


def freqs(rot, base=10000.0):
    return base ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64) / rot) if rot else None


def run(s, inv_freq, interleaved, cu=True, q=True, **kw):
    dev = {n: (t.to(DEV) if t is not None else None) for n, t in s.items()}
    # q, k, v as slices of one tensor, as they come from a projection
    H, Hkv = s["q"].shape[1], s["k"].shape[1]
    x = torch.cat((s["q"], s["k"], s["v"]), dim=1).to(DEV)
    out = api.kv_append(x[:, H:H + Hkv], x[:, H + Hkv:], dev["kc"], dev["vc"], dev["table"], dev["lens"],
                        cu_new=dev["cu"] if cu else None, q=x[:, :H] if q and H else None,
                        inv_freq=None if inv_freq is None else inv_freq.to(DEV), interleaved=interleaved,
                        k_scale=dev["ks"], v_scale=dev["vs"], **kw)
    torch.cuda.synchronize()
    return (out.cpu() if out is not None else None), {n: (t.cpu() if t is not None else None) for n, t in dev.items()}


def plain(s, inv_freq, interleaved, page):
    """(rotated q, {cache name: (values, tolerance)}, scales) in 64 bits."""
    fp8 = s["ks"] is not None
    kc, vc = (s[n].view(torch.float8_e4m3fn).double() if fp8 else s[n].double() for n in ("kc", "vc"))
    tol_k, tol_v = torch.zeros_like(kc), torch.zeros_like(vc)
    ks, vs = (s[n].double().clone() if fp8 else None for n in ("ks", "vs"))
    q = s["q"].double().clone()
    tol_q = torch.zeros_like(q)
    rot = 0 if inv_freq is None else 2 * inv_freq.shape[0]

    def size(x):   # |x| + |y| of each column's pair, 0 for columns that do not turn
        y = torch.zeros_like(x.double())
        if rot:
            a = x[..., :rot].double().abs()
            y[..., :rot] = (a.unflatten(-1, (-1, 2)).sum(-1).repeat_interleave(2, -1) if interleaved
                            else (a[..., :rot // 2] + a[..., rot // 2:]).repeat(1, 1, 2))
        return y
    for b in range(len(s["lens"])):
        c0, c1, past = int(s["cu"][b]), int(s["cu"][b + 1]), int(s["lens"][b])
        if c1 == c0:
            continue
        pos = torch.arange(past, past + c1 - c0)
        kn, vn = s["k"][c0:c1], s["v"][c0:c1]
        kr = _plain.rotate(kn, pos, inv_freq, interleaved) if rot else kn.double()
        if rot:
            q[c0:c1] = _plain.rotate(s["q"][c0:c1], pos, inv_freq, interleaved)
            tol_q[c0:c1] = torch.where(size(s["q"][c0:c1]) > 0,
                                       _plain.BF16_HALF * q[c0:c1].abs() + FP32_TURN * size(s["q"][c0:c1]), 0.0)
        for i in range(c1 - c0):
            p = past + i
            at, off = int(s["table"][b, p // page]), p % page
            if fp8 and (i == 0 or off == 0):
                m = min(page - off, c1 - c0 - i)
                for cache, sc, rows in ((kc, ks, kn.double().abs() * (1.5 if rot else 1.0)), (vc, vs, vn.double().abs())):
                    for h in range(cache.shape[1]):
                        need = _plain.scale_of(float(rows[i:i + m, h].max()))
                        if off:
                            to = max(need, float(sc[at, h]))
                            if to > float(sc[at, h]):
                                cache[at, h, :off] = _plain.to_e4m3(cache[at, h, :off] * (float(sc[at, h]) / to))
                            need = to
                        sc[at, h] = need
            if fp8:
                turned = size(kn[i:i + 1])[0]
                x = kr[i] / ks[at][:, None]
                kc[at, :, off] = torch.where(turned > 0, x, _plain.to_e4m3(x))
                tol_k[at, :, off] = torch.where(
                    turned > 0, _plain.E4M3_HALF * x.abs() + 2.0 ** -10 + FP32_TURN * turned / ks[at][:, None], 0.0)
                vc[at, :, off] = _plain.to_e4m3(vn[i].double() / vs[at][:, None])
                tol_v[at, :, off] = 0.0
            else:
                turned = size(kn[i:i + 1])[0]
                kc[at, :, off], vc[at, :, off] = kr[i], vn[i].double()
                tol_k[at, :, off] = torch.where(turned > 0, _plain.BF16_HALF * kr[i].abs() + FP32_TURN * turned, 0.0)
    return (q, tol_q), (kc, tol_k), (vc, tol_v), ks, vs


def within(got, want):
    ref, tol = want
    off = (got.double() - ref).abs()
    worst = (off - tol).max() if off.numel() else torch.zeros(())
    assert bool((off <= tol).all()), f"off by {float(off.max())}, {float(worst)} more than allowed"


def check(s, inv_freq, interleaved, page, **kw):
    q, got = run(s, inv_freq, interleaved, **kw)
    assert api.last_device_error() == _lib.FA_OK
    rq, rk, rv, rks, rvs = plain(s, inv_freq, interleaved, page)
    n = int(s["cu"][-1])
    if q is not None:
        within(q[:n], (rq[0][:n], rq[1][:n]))
    f8 = s["ks"] is not None
    within(got["kc"].view(torch.float8_e4m3fn) if f8 else got["kc"], rk)
    within(got["vc"].view(torch.float8_e4m3fn) if f8 else got["vc"], rv)
    if f8:
        assert torch.equal(got["ks"].double(), rks) and torch.equal(got["vs"].double(), rvs)
    return q, got


SHAPES = [  # past, new, H_kv, H, d, page
    ([0], [1], 1, 1, 64, 16),
    ([5], [1], 2, 6, 128, 16),
    ([0, 3, 0, 15, 16], [0, 1, 17, 1, 1], 3, 3, 64, 16),
    ([0, 63, 64, 65, 1000], [64, 2, 1, 63, 130], 2, 4, 128, 64),
    ([7, 0, 250], [300, 1, 9], 1, 8, 64, 256),
    ([31] * 40, [1] * 40, 4, 8, 128, 32),
    ([100, 0, 17], [0, 0, 0], 2, 2, 64, 16),      # nothing new
    ([12, 90, 3, 0, 77, 500], [3, 0, 41, 500, 1, 12], 5, 0, 128, 128),
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_append_matches_plain(shape, interleaved, fp8):
    past, new, Hkv, H, d, page = SHAPES[shape]
    s = build(past, new, Hkv, H, d, page, fp8, seed=100 + shape)
    check(s, freqs(d), interleaved, page)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("rot", [0, 16, 48, 96])
def test_part_of_the_columns_turn(rot, fp8):
    for il in (False, True):
        s = build([9, 0, 40], [30, 5, 1], 2, 3, 128, 32, fp8, seed=200 + rot)
        check(s, freqs(rot), il, 32, q=rot > 0)


@pytest.mark.parametrize("fp8", [False, True])
def test_far_positions(fp8):
    """Position 2^20: the plain form's angles are exact in 64 bits; fp32 angles would be off by 0.06."""
    page, past = 256, 2 ** 20 + 77
    s = build([77], [40], 2, 2, 128, page, fp8, seed=300)
    s["lens"] = torch.tensor([past], dtype=torch.int32)
    t = torch.full((1, past // page + 2), -1, dtype=torch.int32)
    t[0, past // page], t[0, past // page + 1] = int(s["table"][0, 0]), 0 if int(s["table"][0, 0]) else 1
    s["table"] = t
    check(s, freqs(128, 500000.0), False, page)


@pytest.mark.parametrize("fp8", [False, True])
def test_even_counts_without_cu_and_rows_behind_the_last_sequence(fp8):
    s = build([4, 20, 0], [2, 2, 2], 2, 4, 64, 16, fp8, seed=400)
    a = check(s, freqs(64), False, 16)
    b = check(s, freqs(64), False, 16, cu=False)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1]["kc"], b[1]["kc"])
    # rows behind cu[B]: nothing of them is written
    s = build([4, 20, 0], [2, 5, 1], 2, 4, 64, 16, fp8, seed=401, rows_behind=9)
    out = torch.full((17, 4, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    check(s, freqs(64), False, 16, q_out=out)
    assert bool((out[8:] == 7).all()) and not bool((out[:8] == 7).all())


@pytest.mark.parametrize("fp8", [False, True])
def test_in_place_queries_and_strided_output(fp8):
    s = build([3, 40], [20, 1], 2, 4, 128, 32, fp8, seed=500)
    want, _ = check(s, freqs(128), False, 32)
    dev = {n: (t.to(DEV) if t is not None else None) for n, t in s.items()}
    x = torch.cat((s["q"], s["k"], s["v"]), dim=1).to(DEV)
    kv = x[:, 4:].clone()
    args = (x[:, 4:6], x[:, 6:], dev["kc"], dev["vc"], dev["table"], dev["lens"])
    kw = dict(cu_new=dev["cu"], inv_freq=freqs(128).to(DEV), k_scale=dev["ks"], v_scale=dev["vs"])
    q = x[:, :4]
    first = q.clone()
    wide = torch.zeros(4, 21, 128, dtype=torch.bfloat16, device=DEV).transpose(0, 1)   # head-major
    assert api.kv_append(*args, q=first, q_out=wide, **kw) is wide
    assert torch.equal(wide.cpu(), want)
    assert api.kv_append(*args, q=q, q_out=q, **kw) is q
    assert torch.equal(q.cpu(), want) and torch.equal(x[:, 4:], kv)


def test_growing_scales_over_many_steps():
    """One token at a time into a page, each ten times the last: the page's scale grows, what it holds
    is rescaled, and every step equals the plain form on what the step before left."""
    page, d, Hkv = 16, 64, 2
    s = build([0], [40], Hkv, 1, d, page, True, seed=600)
    state = {n: s[n].clone() for n in ("kc", "vc", "ks", "vs")}
    for i in range(40):
        one = dict(s, **state, q=s["q"][i:i + 1], k=s["k"][i:i + 1] * 10.0 ** (i % 7 - 3),
                   v=s["v"][i:i + 1] * 10.0 ** (3 - i % 5), lens=torch.tensor([i], dtype=torch.int32),
                   cu=torch.tensor([0, 1], dtype=torch.int32))
        _, got = check(one, freqs(d), False, page)
        state = {n: got[n] for n in state}


def test_extreme_values():
    """Zeros, the largest and smallest bf16, infinities and NaN in 8-bit pages."""
    page, d = 16, 64
    s = build([0, 0, 0, 0, 0], [2, 2, 2, 2, 2], 1, 0, d, page, True, seed=700)
    k, v = s["k"].clone(), s["v"].clone()
    k[0:2], v[0:2] = 0, 0
    k[2:4], v[2:4] = 3.3895e38, -3.3895e38
    k[4:6], v[4:6] = 9.2e-41, 1e-38
    v[6, 0, 3], v[6, 0, 4], v[6, 0, 5] = math.inf, -math.inf, math.nan
    s["k"], s["v"] = k, v
    _, got = run(s, None, False, q=False)
    assert api.last_device_error() == _lib.FA_OK
    at = [int(s["table"][b, 0]) for b in range(5)]
    val = lambda c, sc, b: got[c].view(torch.float8_e4m3fn).double()[at[b], 0, :2] * got[sc].double()[at[b], 0]
    assert float(got["ks"][at[0], 0]) == 2.0 ** -100 and bool((val("kc", "ks", 0) == 0).all())
    assert float(got["ks"][at[1], 0]) == 2.0 ** 120
    big = float(torch.tensor(3.3895e38).bfloat16())
    assert float((val("kc", "ks", 1) - big).abs().max()) <= big / 16
    assert float((val("vc", "vs", 1) + big).abs().max()) <= big / 16
    assert float(got["vs"][at[2], 0]) == 2.0 ** -100 and float(val("vc", "vs", 2).abs().max()) <= 1e-37
    v3 = val("vc", "vs", 3)[0]
    s3 = float(got["vs"][at[3], 0])
    assert s3 == 2.0 ** 121 and float(v3[3]) == 448 * s3 and float(v3[4]) == -448 * s3 and math.isnan(float(v3[5]))
    check(dict(s, k=s["k"].clone(), v=torch.nan_to_num(s["v"], 0, 1, 1)), None, False, page, q=False)


@pytest.mark.parametrize("fp8", [False, True])
def test_bad_pages_and_lengths_store_nothing(fp8):
    page, d = 16, 64
    s = build([4, 10, 20, 0], [3, 10, 2, 2], 2, 2, d, page, fp8, seed=800)
    want = run(s, freqs(d), False)
    s2 = dict(s, table=s["table"].clone(), lens=s["lens"].clone())
    s2["table"][1, 1] = s["kc"].shape[0]     # sequence 1's second page: outside the cache
    s2["lens"][2] = -5                       # sequence 2: a negative length
    s2["lens"][3] = s["table"].shape[1] * page - 1   # sequence 3: its second token lies behind the table
    s2["table"][3, -1] = -1                  # and its first on no page
    q, got = run(s2, freqs(d), False)
    assert api.last_device_error() == _lib.FA_ERR_PAGE
    assert api.last_device_error() == _lib.FA_OK
    assert torch.equal(q[:13], want[0][:13])   # queries of the first two sequences, stored or not
    for n in ("kc", "vc"):
        ref = s[n].clone()
        for b, rows in ((0, range(4, 7)), (1, range(10, 16))):
            for p in rows:
                at = int(s["table"][b, p // page])
                ref[at, :, p % page] = want[1][n][at, :, p % page]
            if fp8:
                at = int(s["table"][b, 0])
                ref[at] = got[n][at]          # (held codes may have been rescaled: checked elsewhere)
        assert torch.equal(got[n], ref)


@pytest.mark.parametrize("fp8", [False, True])
def test_bad_token_counts_store_nothing(fp8):
    s = build([4, 10], [3, 10], 2, 2, 64, 16, fp8, seed=801)
    for cu in ([0, 20, 13], [-5, -2, -1], [13, 13, 13], [0, -7, 40]):
        s2 = dict(s, cu=torch.tensor(cu, dtype=torch.int32), lens=torch.tensor([-1, -1], dtype=torch.int32))
        _, got = run(s2, freqs(64), False)
        assert torch.equal(got["kc"], s["kc"]) and torch.equal(got["vc"], s["vc"])
    api.last_device_error()


@pytest.mark.parametrize("fp8", [False, True])
def test_counts_past_the_tokens_store_nothing_of_their_sequence(fp8):
    s = build([4, 10], [3, 10], 2, 2, 64, 16, fp8, seed=802)
    want = run(s, freqs(64), False)
    q, got = run(dict(s, cu=torch.tensor([0, 3, 14], dtype=torch.int32)), freqs(64), False)
    assert api.last_device_error() == _lib.FA_ERR_PAGE
    assert torch.equal(q, want[0])
    pages = s["table"][1].long()
    for n in ("kc", "vc"):
        assert torch.equal(got[n][pages], s[n][pages])
        assert torch.equal(got[n][int(s["table"][0, 0])], want[1][n][int(s["table"][0, 0])])


def test_replayed_graph_follows_lengths_and_values():
    page, d, Hkv, H = 16, 128, 2, 4
    s = build([15, 3], [30, 30], Hkv, H, d, page, False, seed=900)
    dev = {n: t.to(DEV) for n, t in s.items() if t is not None}
    x = torch.zeros(2, H + 2 * Hkv, d, dtype=torch.bfloat16, device=DEV)
    f = freqs(d).to(DEV)

    def step():
        q = api.kv_append(x[:, H:H + Hkv], x[:, H + Hkv:], dev["kc"], dev["vc"], dev["table"], dev["lens"],
                          q=x[:, :H], inv_freq=f)
        dev["lens"].add_(1)
        return q
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    dev["lens"].copy_(s["lens"])
    with torch.cuda.graph(graph):
        q = step()
    qs = []
    for i in range(30):
        rows = torch.stack([torch.cat((s["q"][b * 30 + i], s["k"][b * 30 + i], s["v"][b * 30 + i])) for b in range(2)])
        x.copy_(rows)
        graph.replay()
        torch.cuda.synchronize()
        qs.append(q.cpu())
    rq, rk, rv, _, _ = plain(s, freqs(d), False, page)
    within(dev["kc"].cpu(), rk)
    within(dev["vc"].cpu(), rv)
    within(torch.stack(qs, 1).flatten(0, 1), rq)
    assert api.last_device_error() == _lib.FA_OK


# Rows that belong to no sequence, before the first one's; as many as pages hold and more
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("page,before", [(16, 3), (16, 16), (16, 100), (64, 64), (64, 200)])
def test_counts_that_begin_behind_row_zero(page, before, fp8):
    """A part of a batch: cu_new[0] > 0 is no error, and the rows before it are left alone."""
    s = build([4, 20, 0], [30, 5, 70], 2, 4, 64, page, fp8, seed=803)
    want, ref = run(s, freqs(64), False)
    pad = lambda x: torch.cat((torch.full((before,) + x.shape[1:], 9.0, dtype=x.dtype), x))
    s2 = dict(s, q=pad(s["q"]), k=pad(s["k"]), v=pad(s["v"]), cu=s["cu"] + before)
    out = torch.full((before + 105, 4, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    q, got = run(s2, freqs(64), False, q_out=out)
    assert api.last_device_error() == _lib.FA_OK
    assert bool((q[:before] == 7).all()) and torch.equal(q[before:], want)
    for n in ("kc", "vc", "ks", "vs"):
        assert got[n] is None or torch.equal(got[n], ref[n])


# counts of three sequences and 40 rows, and which sequences they refuse
BAD_COUNTS = [([0, 5, 3, 9], [1]), ([0, 30, 3, 40], [1]), ([0, 41, 41, 41], [0, 1, 2]), ([-1, 10, 20, 30], [0]),
              ([0, 10, 20, 45], [2]), ([5, 3, 3, 40], [0]), ([0, 0, -4, 0], [1, 2]), ([39, 0, 0, 0], [0])]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("cu,refused", BAD_COUNTS)
def test_bad_token_counts_are_reported_and_the_others_stored(cu, refused, fp8):
    page = 16
    s = build([4, 10, 7], [40, 45, 45], 2, 2, 64, page, fp8, seed=804)
    s = dict(s, cu=torch.tensor(cu, dtype=torch.int32), **{n: s[n][:40] for n in "qkv"})
    _, got = run(s, freqs(64), False)
    assert api.last_device_error() == _lib.FA_ERR_PAGE
    assert api.last_device_error() == _lib.FA_OK
    for b in range(3):
        pages = s["table"][b].long()
        pages = pages[pages >= 0]
        if b in refused or cu[b] == cu[b + 1]:
            for n in ("kc", "vc", "ks", "vs"):
                assert got[n] is None or torch.equal(got[n][pages], s[n][pages])
            continue
        # alone, with good counts
        one = dict(s, table=s["table"][b:b + 1], lens=s["lens"][b:b + 1], cu=torch.tensor(cu[b:b + 2], dtype=torch.int32))
        _, want = run(one, freqs(64), False)
        if all(b == c or not (cu[c] < cu[b + 1] and cu[b] < cu[c + 1]) for c in range(3)):   # (its rows are only its own)
            for n in ("kc", "vc", "ks", "vs"):
                assert got[n] is None or torch.equal(got[n][pages], want[n][pages])


@pytest.mark.parametrize("fp8", [False, True])
def test_many_counts_are_all_looked_at(fp8):
    """One descending pair among 1000 sequences, wherever it stands, also where no row leads to it."""
    B = 1000
    s = build([3] * B, [1] * B, 1, 1, 64, 16, fp8, seed=805)
    for at in (None, 1, 400, 999):
        cu = s["cu"].clone()
        if at is not None:
            cu[at] = cu[at + 1] + 1
        for q in (True, False):
            run(dict(s, cu=cu), freqs(64), False, q=q)
            assert api.last_device_error() == (_lib.FA_OK if at is None else _lib.FA_ERR_PAGE)


@pytest.mark.parametrize("fp8", [False, True])
def test_heads_that_lie_between_one_another(fp8):
    """One head's query, key and value side by side (head stride 3 d), queries turned in place."""
    s = build([3, 40], [20, 1], 4, 4, 64, 16, fp8, seed=806)
    want, ref = check(s, freqs(64), False, 16)
    dev = {n: (t.to(DEV) if t is not None else None) for n, t in s.items()}
    x = torch.stack((s["q"], s["k"], s["v"]), dim=2).to(DEV)   # [T, H, 3, d]
    rest = x[:, :, 1:].clone()
    q = x[:, :, 0]
    assert api.kv_append(x[:, :, 1], x[:, :, 2], dev["kc"], dev["vc"], dev["table"], dev["lens"], cu_new=dev["cu"], q=q,
                         inv_freq=freqs(64).to(DEV), k_scale=dev["ks"], v_scale=dev["vs"], q_out=q) is q
    assert torch.equal(q.cpu(), want) and torch.equal(x[:, :, 1:], rest)
    assert torch.equal(dev["kc"].cpu(), ref["kc"]) and torch.equal(dev["vc"].cpu(), ref["vc"])
