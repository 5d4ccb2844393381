"""GPU parity of attention with capped, biased or masked scores (fa_fwd_score, fa_bwd_score) against the
plain 64-bit form, element by element within the bounds that its roundings give
(_plain_score.py), and how its calls behave: streams, graphs, workspaces, autograd."""
import ctypes
import math
import pathlib
import subprocess
import sys
import threading

import pytest
import torch

from exact_io_aware_12_gb300 import api, _lib
from tests import _plain_score
from tests._plain_score import BF16_HALF, Exact, within
from tests._parity import rel_l2

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


def inputs(B, H, Hkv, N, d, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    x = {n: torch.randn(B, h, N, d, generator=g) for n, h in (("q", H), ("k", Hkv), ("v", Hkv), ("do", H))}
    return {n: (t * (scale if n in "qk" else 1.0)).to(BF) for n, t in x.items()}


def dev(kw):
    return {n: v.to(DEV) if isinstance(v, torch.Tensor) else v for n, v in kw.items()}


def poison(t):
    return t.view(torch.uint8).fill_(0xff) if t.numel() else t


def gpu(x, causal, tau=None, backward=True, **kw):
    """Into outputs and a workspace full of NaN."""
    kw = dev(kw)
    q, k, v, do = (x[n].to(DEV) for n in ("q", "k", "v", "do"))
    ws = {n: kw.get(n) for n in ("bias", "buckets", "docs", "prefix")}
    out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device=DEV)
    space = torch.empty(api.score_workspace_bytes(q, causal, backward=False, **ws), dtype=torch.uint8, device=DEV)
    for t in (out, lse, space):
        poison(t)
    o, lse = api.fwd(q, k, v, causal, tau, out=out, lse=lse, workspace=space, **kw)
    grads = ()
    if backward:
        space = torch.empty(api.score_workspace_bytes(q, causal, **ws), dtype=torch.uint8, device=DEV)
        dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
        more = {}
        if "bias" in kw:
            more["dbias"] = torch.empty_like(kw["bias"])
        for t in (space, dq, dk, dv, *more.values()):
            poison(t)
        grads = api.bwd(q, k, v, o, do, lse, causal, tau, dq=dq, dk=dk, dv=dv, workspace=space, **more, **kw)
    torch.cuda.synchronize()
    assert api.last_device_error() == _lib.FA_OK
    return o, lse, grads


def check(x, causal, tau=None, backward=True, **kw):
    B, H, N, d = x["q"].shape
    o, lse, grads = gpu(x, causal, tau, backward, **kw)
    e = Exact(x["q"], x["k"], x["v"], causal, tau or 1 / math.sqrt(d), x["do"] if backward else None, **kw)
    within(o, e.o, e.b_o, "O")
    within(lse, e.lse, e.b_lse, "LSE")
    empty = ~e.see.any(-1).expand(B, H, N)
    assert not o.cpu()[empty].any() and bool((lse.cpu()[empty] == -math.inf).all())
    for got, n in zip(grads, ("dq", "dk", "dv", "dbias")):
        within(got, getattr(e, n), getattr(e, "b_" + n), n)
    if grads:
        assert not grads[0].cpu()[empty].any()
        unseen = ~e.see.any(-2).expand(B, x["k"].shape[1], N)
        assert not grads[1].cpu()[unseen].any() and not grads[2].cpu()[unseen].any()
    # (1.25: of the variances' sum over a few thousand elements, and of fp32)
    if N >= 64:
        for got, n in zip((o, *grads), ("o", "dq", "dk", "dv", "dbias")):
            off = float((got.cpu().double() - getattr(e, n)).norm())
            assert off <= 1.25 * getattr(e, "s_" + n) + 1e-7, f"{n}: {off:.3g} and {getattr(e, 's_' + n):.3g}"
    return e, o, lse, grads


def slopes_of(H):
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)])


def table_of(H, nb, far, both, seed, dtype=BF):
    m = api.distance_buckets(nb, far, both)
    return dict(bias=torch.randn(nb, H, generator=torch.Generator().manual_seed(seed)).to(dtype), buckets=m)


def docs_of(B, N, seed, padding=True):
    g = torch.Generator().manual_seed(seed)
    ids = torch.empty(B, N, dtype=torch.int32)
    for b in range(B):
        at, x = 0, 0
        while at < N:
            n = min(N - at, int(torch.randint(1, max(2, N // 2), (1,), generator=g)))
            x = int(torch.randint(-1 if padding else 0, 7, (1,), generator=g))
            ids[b, at:at + n] = x
            at += n
    return ids


LENGTHS = [1, 2, 77, 128, 129, 300, 517]
HEADS = {64: (2, 4, 2), 128: (1, 6, 2)}


# ------------------------------------------------------------------ the operators ----
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("N", LENGTHS)
def test_shared_heads_in_documents(N, causal, d):
    B, H, Hkv = HEADS[d]
    check(inputs(B, H, Hkv, N, d, N + d), causal, docs=docs_of(B, N, N))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("N", LENGTHS)
@pytest.mark.parametrize("cap,scale", [(50.0, 1.0), (20.0, 3.0), (2.0, 2.0)])
def test_cap(N, cap, scale, causal, d):
    """Scores of a small part of the cap, of more, and far beyond: each form of the tanh."""
    check(inputs(1, 3, 3, N, d, N + d, scale), causal, softcap=cap)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("N", LENGTHS)
def test_slopes(N, causal, d):
    check(inputs(2, 4, 2, N, d, N + d), causal, slopes=slopes_of(4))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("N", LENGTHS)
def test_table(N, causal, dtype, d):
    check(inputs(2, 3, 3, N, d, N + d), causal, **table_of(3, 32, 128, not causal, N, dtype))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N", LENGTHS)
def test_prefix(N, d):
    B, H, Hkv = 4, 2, 1
    prefix = torch.tensor([N // 2, 0, N, 2 * N + 5], dtype=torch.int32)
    check(inputs(B, H, Hkv, N, d, N + d), True, prefix=prefix)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kw", [
    dict(softcap=3.0, slopes=True), dict(softcap=3.0, table=(32, 128, False)), dict(table=(16, 40, True), prefix=True, docs=True),
    dict(softcap=8.0, window=100), dict(slopes=True, docs=True, prefix=True, window=150), dict(window=1, softcap=5.0),
    dict(table=(4, 1000, False), window=300), dict(prefix=True, window=64), dict(softcap=4.0, docs=True, window=33),
    dict(softcap=2.0, table=(48, 500, True), docs=True), dict(window=10 ** 6, slopes=True)],
    ids=lambda kw: "-".join(kw))
@pytest.mark.parametrize("N", [130, 700])
def test_together(N, kw, d):
    B, H = 2, 4
    kw = dict(kw)
    if kw.get("slopes"):
        kw["slopes"] = slopes_of(H)
    if "table" in kw:
        nb, far, both = kw.pop("table")
        kw.update(table_of(H, nb, far, both, 5))
    if kw.get("docs"):
        kw["docs"] = docs_of(B, N, 6)
    if kw.get("prefix"):
        kw["prefix"] = torch.tensor([N // 3, N - 1], dtype=torch.int32)
    check(inputs(B, H, 2, N, d, N + d), True, **kw)


@pytest.mark.parametrize("d", [64, 128])
def test_maps_of_any_kind(d):
    """Maps that name buckets in any order, twice, or none; one distance each side; more than there are keys."""
    N, H = 400, 3
    g = torch.Generator().manual_seed(1)
    for far, nb, causal in ((1, 1, False), (1, 3, True), (1024, 1024, False), (129, 7, False), (127, 5, True), (300, 40, True)):
        m = torch.randint(-2, nb + 2, (2 * far + 1,), generator=g, dtype=torch.int32)
        for ends in (m, m.clone()):
            if ends is not m:
                ends[0], ends[-1] = -1, nb - 1
            check(inputs(1, H, 1, N, d, far), causal, bias=torch.randn(nb, H, generator=g), buckets=ends)


@pytest.mark.parametrize("d", [64, 128])
def test_more_heads_than_a_grid_dimension_holds(d):
    H = 70000
    check(inputs(1, H, H, 2, d, 3), True, **table_of(H, 4, 3, False, 4))
    check(inputs(1, H, 7, 1, d, 3), False, slopes=torch.linspace(0, 1, H))


@pytest.mark.parametrize("d", [64, 128])
def test_large_biases(d):
    """Biases and slopes that leave most weights at 0."""
    N, H = 333, 2
    x = inputs(1, H, 2, N, d, 9)
    check(x, True, slopes=torch.tensor([40.0, 0.0]))
    t = table_of(H, 32, 128, False, 3)
    check(x, True, bias=(t["bias"].float() * 60).to(BF), buckets=t["buckets"])


@pytest.mark.parametrize("d", [64, 128])
def test_empty_tiles(d):
    """Whole tiles of padding, one in the middle, one at the end, and a batch with a sequence of nothing else."""
    N = 900
    ids = torch.zeros(3, N, dtype=torch.int32)
    ids[0, 200:600] = -1
    ids[0, 600:] = 4
    ids[1, 130:] = -7
    ids[2] = -1
    for causal in (True, False):
        check(inputs(3, 2, 1, N, d, 31), causal, docs=ids, softcap=10.0)
        check(inputs(3, 2, 2, N, d, 32), causal, docs=ids, **table_of(2, 32, 128, not causal, 3))


@pytest.mark.parametrize("d", [64, 128])
def test_equal_numbers_apart_are_two_documents(d):
    N = 300
    ids = torch.tensor([[3] * 100 + [5] * 50 + [3] * 150], dtype=torch.int32)
    check(inputs(1, 2, 2, N, d, 41), False, docs=ids)


@pytest.mark.parametrize("d", [64, 128])
def test_single_token_documents(d):
    N = 260
    x = inputs(1, 2, 1, N, d, 42)
    e, o, _, grads = check(x, True, docs=torch.arange(N, dtype=torch.int32)[None])
    assert torch.equal(o.cpu(), x["v"].expand(1, 2, N, d))  # (a weight of one)


def test_random_calls():
    """Sixty seeded calls with any of the options, over sizes, heads and lengths."""
    g = torch.Generator().manual_seed(123)
    r = lambda lo, hi: int(torch.randint(lo, hi + 1, (1,), generator=g))
    for i in range(60):
        d, Hkv, B, N = 64 * r(1, 2), r(1, 3), r(1, 3), r(1, 650)
        H = Hkv * r(1, 3)
        causal = r(0, 2) > 0
        kw = {}
        if r(0, 1):
            kw["softcap"] = float(2 ** r(0, 6))
        pick = r(0, 2)
        if pick == 1:
            kw["slopes"] = torch.rand(H, generator=g)
        if pick == 2:
            far, nb = r(1, 200), r(1, 50)
            kw["buckets"] = torch.randint(0, nb, (2 * far + 1,), generator=g, dtype=torch.int32)
            kw["bias"] = torch.randn(nb, H, generator=g).to(BF if r(0, 1) else torch.float32)
        if r(0, 1):
            kw["docs"] = docs_of(B, N, i)
        if causal and r(0, 2) == 0:
            kw["prefix"] = torch.randint(-2, N + 3, (B,), generator=g, dtype=torch.int32)
        if causal and r(0, 2) == 0:
            kw["window"] = r(1, N + 5)
        if kw:
            check(inputs(B, H, Hkv, N, d, 500 + i, 1 + r(0, 2) / 2), causal, **kw)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [False, True])
def test_small_scores_beside_scores_of_a_large_cap(causal, d):
    """Rows whose scores are of deviation one, between rows whose scores reach a cap of 2^20: 2^-23 of the
    cap would be 0.1 of a score.  The weights of the former are flat, so that O and dQ of these rows are within
    sqrt(2/3) 2^-8 (as above), and their LSE within what fp32 gives a score of one."""
    N, cap = 300, 2.0 ** 20
    x = inputs(2, 2, 1, N, d, 14)
    # (powers of two, exact in bf16: sqrt(d) deviates q.k; 8 = 64^(1/2))
    grow = torch.full((N, 1), 2.0 ** 8)
    grow[::2] = 2.0 ** -11
    x["q"], x["k"] = (x["q"].float() * grow).to(BF), (x["k"].float() * 2.0 ** 8).to(BF)
    o, lse, (dq, dk, dv) = gpu(x, causal, 1.0, softcap=cap)
    e = Exact(x["q"], x["k"], x["v"], causal, 1.0, x["do"], softcap=cap)
    far = (x["q"].double() @ x["k"].double().mT).abs().amax(-1)
    assert float(far[..., 1::2].amax()) > 0.6 * cap and float(far[..., ::2].amax()) < 100
    for got, n in ((o, "o"), (dq, "dq")):
        assert rel_l2(got[:, :, ::2], getattr(e, n)[:, :, ::2]) <= 1.25 * math.sqrt(2 / 3) * 2.0 ** -8, n
    assert float((lse.cpu().double() - e.lse)[:, :, ::2].abs().max()) < 1e-4


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bias", ["none", "slopes", "table"])
@pytest.mark.parametrize("grow", [2.0 ** 8, 2.0 ** 10, 2.0 ** 12])
def test_scores_that_fp32_holds_coarsely(grow, bias, d):
    """Scores of 2^19 to 2^23 under a larger cap: their fp32 steps are 2^-4 to 1, so weights may be off by as many
    powers of e, but stay finite, and so do all gradients."""
    x = inputs(1, 2, 2, 300, d, 14)
    x["q"], x["k"] = (x["q"].float() * grow).to(BF), (x["k"].float() * 2.0 ** 8).to(BF)
    kw = {"none": {}, "slopes": dict(slopes=slopes_of(2)), "table": table_of(2, 32, 128, False, 3, torch.float32)}[bias]
    o, lse, grads = gpu(x, True, 1.0, softcap=2.0 ** 40, **kw)
    for t in (o, lse, *grads):
        assert bool(t.isfinite().all())


def test_other_scales_of_scores():
    x = inputs(1, 2, 2, 200, 64, 8)
    for tau in (1e-3, 1.0, 4.0):
        check(x, True, tau, softcap=30.0)
        check(x, True, tau, slopes=slopes_of(2))
    for cap in (2.0 ** -20, 2.0 ** 60):
        check(x, True, softcap=cap)


@pytest.mark.parametrize("causal", [False, True])
def test_bias_gradient_is_as_exact_at_length(causal):
    """2500 tokens: a far bucket sums almost all of a row's weight, where an error of D would add up (it
    was off by 1e-2).  sum_j dY_ij = 0, so the far bucket is minus the sum of the near ones, a few of a row's
    keys, and its own pairs' roundings are the square root of the ratio of keys larger beside it than
    theirs: of 2^-11 / sqrt(3), what s_dbias says, and below 2^-10."""
    x = inputs(1, 4, 4, 2500, 64, 77)
    t = table_of(4, 32, 128, not causal, 7, torch.float32)
    *_, grads = gpu(x, causal, **t)
    e = Exact(x["q"], x["k"], x["v"], causal, 0.125, x["do"], **t)
    off = float((grads[3].cpu().double() - e.dbias).norm())
    assert off <= 1.25 * e.s_dbias and off <= 2.0 ** -10 * float(e.dbias.norm())


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [False, True])
def test_capped_bias_gradient_is_as_exact_at_length(causal, d):
    """The same with a cap.  P of the sums as fp16 leaves 2^-11 / sqrt(3) of each pair's dY, 4.2e-4 of the whole at
    most on these inputs by the variances' sum (with bf16, 3.4e-3): below 2^-10 with twice that and fp32's part."""
    x = inputs(1, 2, 2, 2500, d, 77)
    t = table_of(2, 32, 128, not causal, 7, torch.float32)
    *_, grads = gpu(x, causal, softcap=50.0, **t)
    e = Exact(x["q"], x["k"], x["v"], causal, d ** -0.5, x["do"], softcap=50.0, **t)
    assert float((grads[3].cpu().double() - e.dbias).norm()) <= 2.0 ** -10 * float(e.dbias.norm())


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N,nb,far,causal,cap", [(77, 4, 9, True, 3.0), (300, 32, 128, False, 8.0), (517, 32, 40, True, 50.0),
                                                 (700, 8, 300, False, 2.0 ** 12)])
def test_capped_bias_gradient_by_buckets(N, nb, far, causal, cap, d):
    """Bucket by bucket: P off by 2^-11 of itself, as without a cap."""
    x = inputs(2, 4, 2, N, d, N + d)
    t = table_of(4, nb, far, not causal, 7, torch.float32)
    *_, grads = gpu(x, causal, softcap=cap, **t)
    e = Exact(x["q"], x["k"], x["v"], causal, d ** -0.5, x["do"], softcap=cap, **t)
    do, v = x["do"].double(), x["v"].double().repeat_interleave(2, 1)
    dy = e.p * (do @ v.mT - (do * e.o).sum(-1, keepdim=True))
    L = t["buckets"].numel() // 2
    dist = torch.arange(N)[:, None] - torch.arange(N)[None, :]
    at = t["buckets"].long()[dist.clamp(-L, L) + L].flatten()
    size = torch.zeros(nb, 4, dtype=torch.float64).index_add_(0, at, dy.abs().sum(0).flatten(1).T)
    within(grads[3], e.dbias, e.b_dbias - BF16_HALF * size, "dbias")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kw", [
    dict(prefix=True), dict(softcap=50.0), dict(softcap=3.0), dict(slopes=True, docs=True), dict(softcap=6.0, slopes=True),
    dict(table=(32, 128, False)), dict(softcap=20.0, table=(32, 40, True), docs=True), dict(window=200, softcap=8.0)],
    ids=lambda kw: "-".join(kw))
def test_more_tiles_than_the_sms_hold(kw, d):
    """52 heads of 6 tiles, more than two for each SM, which one softmax warpgroup per tile takes."""
    B, H, N = 2, 26, 700
    kw = dict(kw)
    if kw.get("slopes"):
        kw["slopes"] = slopes_of(H)
    if "table" in kw:
        nb, far, both = kw.pop("table")
        kw.update(table_of(H, nb, far, both, 5))
    if kw.get("docs"):
        kw["docs"] = docs_of(B, N, 6)
    if kw.get("prefix"):
        kw["prefix"] = torch.tensor([N // 3, N - 1], dtype=torch.int32)
    x = inputs(B, H, 13, N, d, N + d)
    check(x, True, backward=False, **kw)
    a, b = gpu(x, True, backward=False, **kw), gpu(x, True, backward=False, **kw)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N,scale,kw", [
    (8200, 1.5, dict(softcap=50.0, window=4096)), (4200, 1.5, dict(softcap=50.0)), (4200, 1.0, dict(slopes=True)),
    (4200, 1.0, dict(table=(32, 128, False))), (4200, 1.5, dict(softcap=30.0, prefix=True)), (4200, 1.0, dict(softcap=20.0, table=(32, 128, False)))],
    ids=str)
def test_long_sequences(N, scale, kw, d):
    """Tens of blocks per tile, most of them wholly visible and far from the diagonal: element by element as the
    short ones."""
    kw, H = dict(kw), 1 if N > 5000 else 2
    if kw.get("slopes"):
        kw["slopes"] = slopes_of(H)
    if "table" in kw:
        kw.update(table_of(H, *kw.pop("table"), 5))
    if kw.get("prefix"):
        kw["prefix"] = torch.tensor([N // 3], dtype=torch.int32)
    check(inputs(1, H, 1, N, d, N + d, scale), True, **kw)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N,H,Hkv", [(300, 52, 52), (100, 170, 170), (260, 120, 40)])
@pytest.mark.parametrize("kw", [
    dict(softcap=5.0), dict(slopes=True, docs=True), dict(table=(32, 128, False)), dict(softcap=20.0, table=(8, 40, True), docs=True),
    dict(prefix=True, window=90)], ids=lambda kw: "-".join(kw))
def test_backward_of_more_tiles_than_sms(kw, N, H, Hkv, d):
    """Two sequences whose key tiles are 240 and more, of one step and of several: an SM takes two or three."""
    B = 2
    kw = dict(kw)
    if kw.get("slopes"):
        kw["slopes"] = slopes_of(H)
    if "table" in kw:
        nb, far, both = kw.pop("table")
        kw.update(table_of(H, nb, far, both, 5))
    if kw.get("docs"):
        kw["docs"] = docs_of(B, N, 6)
    if kw.get("prefix"):
        kw["prefix"] = torch.tensor([N // 3, N - 1], dtype=torch.int32)
    x = inputs(B, H, Hkv, N, d, N + d)
    check(x, True, **kw)
    a, b = gpu(x, True, **kw), gpu(x, True, **kw)
    assert all(torch.equal(p, q) for p, q in zip(a[2][1:], b[2][1:]))


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("lengths", [[300, 33000, 31, 1, 700, 128, 35000, 577], [66000, 2], [65536, 65536, 500]], ids=str)
def test_documents_of_long_sequences(lengths, causal):
    """Runs longer than the tokens that are looked at together, across their limits and up to them, each against
    the formula in 64 bits.  Where a row sees many keys of like weight, the 2^-8 / sqrt(3) of its
    weights' roundings and of the result's give an O, dQ, dK and dV within sqrt(2/3) 2^-8; 1.25 as above."""
    d, gap = 64, 70  # (padding behind each)
    N = sum(lengths) + gap * len(lengths)
    ids = torch.full((1, N), -1, dtype=torch.int32)
    at = 0
    for i, n in enumerate(lengths):
        ids[0, at:at + n] = i % 2
        at += n + gap
    x = inputs(1, 1, 1, N, d, 51)
    o, lse, (dq, dk, dv) = gpu(x, causal, docs=ids)
    none = ids[0] < 0
    for t in (o, dq, dk, dv):
        assert not t[0, 0].cpu()[none].any()
    assert bool((lse[0, 0].cpu()[none] == -math.inf).all())
    at = 0
    for n in lengths:
        q, k, v, do = (x[i][0, 0, at:at + n].to(DEV).double() for i in ("q", "k", "v", "do"))
        eo, el, eq, ek, ev = torch.empty_like(q), torch.empty_like(q[:, 0]), torch.empty_like(q), torch.zeros_like(k), torch.zeros_like(v)
        for r in range(0, n, 4096):
            z = slice(r, min(n, r + 4096))
            y = q[z] @ k.T * d ** -0.5
            if causal:
                y.masked_fill_(torch.arange(n, device=DEV)[None, :] > torch.arange(r, z.stop, device=DEV)[:, None], -math.inf)
            el[z] = torch.logsumexp(y, -1)
            w = (y - el[z, None]).exp_()
            eo[z] = w @ v
            ev += w.T @ do[z]
            w *= do[z] @ v.T - (do[z] * eo[z]).sum(-1, keepdim=True)
            eq[z] = w @ k * d ** -0.5
            ek += w.T @ q[z] * d ** -0.5
        assert float((lse[0, 0, at:at + n] - el).abs().max()) < 1e-4
        if n >= 64:
            for got, want in ((o, eo), (dq, eq), (dk, ek), (dv, ev)):
                assert rel_l2(got[0, 0, at:at + n], want) <= 1.25 * math.sqrt(2 / 3) * 2.0 ** -8
        at += n + gap


# --------------------------------------------------------------------- behaviour ----
def test_without_options_it_is_plain_attention():
    """All fields 0: the forward and backward of grouped heads."""
    x = inputs(2, 6, 2, 300, 128, 3)
    d = {n: t.to(DEV) for n, t in x.items()}
    o, lse = torch.empty_like(d["q"]), torch.empty(2, 6, 300, device=DEV)
    dq, dk, dv = (torch.empty_like(d[n]) for n in "qkv")
    s = _lib.Score(0.0, None, None, None, 0, 0, 0, None, None, 0)
    st = torch.cuda.current_stream().cuda_stream
    at = lambda *n: [d[i].data_ptr() for i in n]
    _lib.check(_lib.fa_fwd_score(*at("q", "k", "v"), o.data_ptr(), lse.data_ptr(), 2, 6, 2, 300, 128, 0.09, 1, s, None, 0, st), "f")
    _lib.check(_lib.fa_bwd_score(*at("q", "k", "v"), o.data_ptr(), *at("do"), lse.data_ptr(), dq.data_ptr(), dk.data_ptr(),
                                 dv.data_ptr(), None, 2, 6, 2, 300, 128, 0.09, 1, s, None, 0, st), "b")
    torch.cuda.synchronize()
    assert api.last_device_error() == _lib.FA_OK
    e = Exact(x["q"], x["k"], x["v"], True, 0.09, x["do"])
    for got, n in ((o, "o"), (lse, "lse"), (dq, "dq"), (dk, "dk"), (dv, "dv")):
        within(got, getattr(e, n), getattr(e, "b_" + n), n)


@pytest.mark.parametrize("d", [64, 128])
def test_runs_repeat_bitwise(d):
    """The forward, dK, dV and the bias's gradient (dQ's sums have no fixed order)."""
    x = inputs(2, 4, 2, 700, d, 11)
    kw = dict(softcap=6.0, docs=docs_of(2, 700, 3), **table_of(4, 32, 128, False, 2))
    a, b = gpu(x, True, **kw), gpu(x, True, **kw)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    for i in (1, 2, 3):
        assert torch.equal(a[2][i], b[2][i])


@pytest.mark.parametrize("d", [64, 128])
def test_batches_and_heads_do_not_mix(d):
    B, H, N = 3, 4, 333
    x = inputs(B, H, 2, N, d, 12)
    kw = dict(softcap=6.0, docs=docs_of(B, N, 3), slopes=slopes_of(H))
    o, lse, g = gpu(x, True, **kw)
    for b in range(B):
        for hk in range(2):
            xs = {n: t[b:b + 1, 2 * hk:2 * hk + 2] if n in ("q", "do") else t[b:b + 1, hk:hk + 1] for n, t in x.items()}
            xs = {n: t.contiguous() for n, t in xs.items()}
            os, ls, gs = gpu(xs, True, softcap=6.0, docs=kw["docs"][b:b + 1].contiguous(),
                             slopes=kw["slopes"][2 * hk:2 * hk + 2].contiguous())
            assert torch.equal(o[b:b + 1, 2 * hk:2 * hk + 2], os) and torch.equal(lse[b:b + 1, 2 * hk:2 * hk + 2], ls)
            assert torch.equal(g[1][b:b + 1, hk:hk + 1], gs[1]) and torch.equal(g[2][b:b + 1, hk:hk + 1], gs[2])


def test_autograd():
    x = inputs(2, 4, 2, 200, 64, 21)
    kw = dict(softcap=5.0, docs=docs_of(2, 200, 8), **table_of(4, 16, 64, False, 4, torch.float32))
    q, k, v, bias = (t.to(DEV).requires_grad_() for t in (x["q"], x["k"], x["v"], kw["bias"]))
    rest = dev({n: t for n, t in kw.items() if n != "bias"})
    o = api.attention(q, k, v, True, bias=bias, **rest)
    o.backward(x["do"].to(DEV).transpose(1, 2).contiguous().transpose(1, 2))
    e = Exact(x["q"], x["k"], x["v"], True, 0.125, x["do"], **kw)
    within(o, e.o, e.b_o, "O")
    for t, n in ((q, "dq"), (k, "dk"), (v, "dv"), (bias, "dbias")):
        within(t.grad, getattr(e, n), getattr(e, "b_" + n), n)
    # a frozen bias costs and gets no gradient
    q.grad = None
    api.attention(q, k, v, True, bias=bias.detach(), **rest).backward(x["do"].to(DEV))
    within(q.grad, e.dq, e.b_dq, "dq")
    with pytest.raises(ValueError, match="no gradient"):
        api.attention(q, k, v, True, slopes=torch.ones(4, device=DEV, requires_grad=True))
    torch.cuda.synchronize()
    assert api.last_device_error() == _lib.FA_OK


@pytest.mark.parametrize("d", [64, 128])
def test_a_frozen_bias_in_its_workspace(d):
    """Without the gradient, in a workspace of that size with a border behind it: dK and dV bit for bit the same."""
    x = {n: t.to(DEV) for n, t in inputs(2, 4, 2, 700, d, 23).items()}
    t = dev(table_of(4, 32, 128, True, 4))
    for kw in (dict(t), dict(t, softcap=20.0), dict(t, docs=docs_of(2, 700, 3).to(DEV))):
        o, lse = api.fwd(x["q"], x["k"], x["v"], False, **kw)
        all4 = api.bwd(x["q"], x["k"], x["v"], o, x["do"], lse, False, **kw)
        size = api.score_workspace_bytes(x["q"], False, t["bias"], t["buckets"], kw.get("docs"), bias_grad=False)
        space = torch.full((size + 4096,), 0xff, dtype=torch.uint8, device=DEV)
        three = api.bwd(x["q"], x["k"], x["v"], o, x["do"], lse, False, bias_grad=False, workspace=space[:size], **kw)
        assert bool((space[size:] == 0xff).all())
        assert torch.equal(all4[1], three[1]) and torch.equal(all4[2], three[2])
        assert rel_l2(three[0].cpu(), all4[0].cpu()) < 2.0 ** -8  # (dQ's order of summation is free)
        with pytest.raises(_lib.FAError) as err:
            api.bwd(x["q"], x["k"], x["v"], o, x["do"], lse, False, workspace=space[:size], **kw)
        assert err.value.code == _lib.FA_ERR_WORKSPACE


@pytest.mark.parametrize("kw", [{}, dict(softcap=4.0), dict(window=30, sinks=2)])
def test_second_derivatives_raise(kw):
    x = {n: t.to(DEV) for n, t in inputs(1, 2, 2, 150, 64, 61).items()}
    q = x["q"].requires_grad_()
    want, = torch.autograd.grad(api.attention(q, x["k"], x["v"], True, **kw), q, x["do"])
    g, = torch.autograd.grad(api.attention(q, x["k"], x["v"], True, **kw), q, x["do"], create_graph=True)
    assert rel_l2(g.detach().cpu(), want.cpu()) < 1e-3  # (dQ's order of summation is free)
    with pytest.raises(RuntimeError, match="no derivative"):
        torch.autograd.grad(g.float().pow(2).sum() + q.float().sum(), q)


def test_bias_gradient_only_on_request():
    x = {n: t.to(DEV) for n, t in inputs(1, 2, 2, 150, 64, 22).items()}
    t = dev(table_of(2, 16, 64, False, 4))
    o, lse = api.fwd(x["q"], x["k"], x["v"], True, **t)
    all4 = api.bwd(x["q"], x["k"], x["v"], o, x["do"], lse, True, **t)
    three = api.bwd(x["q"], x["k"], x["v"], o, x["do"], lse, True, bias_grad=False, **t)
    assert len(all4) == 4 and len(three) == 3
    assert torch.equal(all4[1], three[1]) and torch.equal(all4[2], three[2])


def test_no_rows():
    """Empty batches and lengths: nothing written but a bias's gradient of zeros."""
    for B, N in ((0, 5), (2, 0)):
        q = torch.empty(B, 4, N, 64, dtype=BF, device=DEV)
        t = dev(table_of(4, 16, 64, False, 4))
        o, lse = api.fwd(q, q, q, True, **t)
        assert o.shape == q.shape and lse.shape == q.shape[:3]
        g = api.bwd(q, q, q, o, q, lse, True, dbias=torch.ones_like(t["bias"]), **t)
        assert not g[3].any()


def test_keys_that_no_query_head_reads():
    """No query heads beside key heads: dK and dV are zeros."""
    q, k = torch.empty(2, 0, 300, 64, dtype=BF, device=DEV), torch.ones(2, 3, 300, 64, dtype=BF, device=DEV)
    for kw in (dict(softcap=5.0), dict(docs=torch.zeros(2, 300, dtype=torch.int32, device=DEV))):
        o, lse = api.fwd(q, k, k, True, **kw)
        dk, dv = torch.ones_like(k), torch.ones_like(k)
        g = api.bwd(q, k, k, o, o, lse, True, dk=dk, dv=dv, **kw)
        assert g[0].shape == q.shape and not g[1].any() and not g[2].any()


def test_a_bias_of_no_heads():
    """As empty as a call without one."""
    q, m = torch.empty(2, 0, 300, 64, dtype=BF, device=DEV), api.distance_buckets(16, 64, device=DEV)
    bias = torch.empty(16, 0, device=DEV)
    o, lse = api.fwd(q, q, q, True, bias=bias, buckets=m)
    assert o.shape == q.shape and lse.shape == q.shape[:3]
    g = api.bwd(q, q, q, o, o, lse, True, bias=bias, buckets=m)
    assert len(g) == 4 and g[3].shape == bias.shape and g[3].dtype == bias.dtype
    given = torch.empty_like(bias)
    assert api.bwd(q, q, q, o, o, lse, True, bias=bias, buckets=m, dbias=given)[3] is given


def test_side_stream_and_device_argument():
    """Inputs made on another stream, the call on a stream of its own."""
    x = inputs(1, 4, 4, 900, 128, 33)
    kw = dev(dict(docs=docs_of(1, 900, 2), **table_of(4, 32, 128, False, 1)))
    want = gpu(x, True, **kw)
    s = torch.cuda.Stream()
    d = {n: t.to(DEV) for n, t in x.items()}
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        late = {n: t * 1 for n, t in d.items()}
        o, lse = api.fwd(late["q"], late["k"], late["v"], True, **kw)
        g = api.bwd(late["q"], late["k"], late["v"], o, late["do"], lse, True, **kw)
    s.synchronize()
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    for i in (1, 2, 3):
        assert torch.equal(g[i], want[2][i])


def test_captured_and_replayed():
    """Forward and backward captured once and replayed on new inputs, documents, prefixes and biases,
    with two graphs that have workspaces of their own."""
    B, H, N, d = 2, 4, 400, 64
    t = dev(table_of(H, 16, 64, False, 1))
    graphs = []
    for i in range(2):
        x = {n: v.to(DEV) for n, v in inputs(B, H, 2, N, d, i).items()}
        extra = dev(dict(docs=docs_of(B, N, i), prefix=torch.tensor([5, 100], dtype=torch.int32), bias=t["bias"].clone(),
                         buckets=t["buckets"]))

        def step(x=x, extra=extra):
            o, lse = api.fwd(x["q"], x["k"], x["v"], True, softcap=9.0, **extra)
            return o, lse, api.bwd(x["q"], x["k"], x["v"], o, x["do"], lse, True, softcap=9.0, **extra)
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            step()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step()
        graphs.append((g, x, extra, out))
    for trial in range(3):
        want = []
        for i, (g, x, extra, out) in enumerate(graphs):
            new = inputs(B, H, 2, N, d, 50 + 2 * trial + i)
            more = dict(docs=docs_of(B, N, 9 + trial), prefix=torch.tensor([N, trial], dtype=torch.int32),
                        bias=torch.randn(16, H, generator=torch.Generator().manual_seed(trial)).to(BF))
            for n, v in new.items():
                x[n].copy_(v)
            for n, v in more.items():
                extra[n].copy_(v)
            want.append(Exact(new["q"], new["k"], new["v"], True, 0.125, new["do"], softcap=9.0, buckets=t["buckets"].cpu(), **more))
        for g, *_ in graphs:
            g.replay()
        torch.cuda.synchronize()
        for e, (_, _, _, (o, lse, grads)) in zip(want, graphs):
            for got, n in zip((o, lse, *grads), ("o", "lse", "dq", "dk", "dv", "dbias")):
                within(got, getattr(e, n), getattr(e, "b_" + n), n)
    assert api.last_device_error() == _lib.FA_OK


def test_autograd_captured():
    """Forward and backward through autograd in a graph.  (No eager graph of the same leaves may live then:
    torch ties a leaf's gradient to the stream that made it, which a capture may not wait for.)"""
    x = inputs(1, 2, 2, 150, 64, 61)
    do = x["do"].to(DEV)
    q, k, v = (x[n].to(DEV).requires_grad_() for n in "qkv")
    want = torch.autograd.grad(api.attention(q, k, v, True, softcap=4.0), (q, k, v), do)
    q, k, v = (t.detach().clone().requires_grad_() for t in (q, k, v))
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.autograd.grad(api.attention(q, k, v, True, softcap=4.0), (q, k, v), do)
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(g):
        got = torch.autograd.grad(api.attention(q, k, v, True, softcap=4.0), (q, k, v), do)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])


@pytest.mark.parametrize("kw", ["softcap=4.0", "slopes=torch.ones(2, device='cuda')", "prefix=torch.ones(1, dtype=torch.int32, device='cuda')"])
def test_first_backward_of_a_process(kw):
    """Autograd's thread has no CUDA context until something binds one; the call's descriptors need it."""
    code = f"""
import torch
from exact_io_aware_12_gb300 import api
q, k, v = (torch.randn(1, 2, 150, 64, device="cuda").bfloat16().requires_grad_() for _ in range(3))
grads = torch.autograd.grad(api.attention(q, k, v, True, {kw}), (q, k, v), q.detach().clone())
torch.cuda.synchronize()
assert all(bool(t.isfinite().all()) for t in grads)
"""
    root = pathlib.Path(__file__).resolve().parent.parent
    done = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stderr[-2000:]


def test_a_context_of_the_caller_stays():
    """A context made and bound through the driver's interface is current after a call as before it."""
    code = """
import ctypes
from exact_io_aware_12_gb300 import _lib
cuda = ctypes.CDLL("libcuda.so.1")
own, now = ctypes.c_void_p(), ctypes.c_void_p()
assert cuda.cuInit(0) == 0 and cuda.cuCtxCreate_v2(ctypes.byref(own), 0, 0) == 0
code = _lib.fa_last_device_error(None)
assert cuda.cuCtxGetCurrent(ctypes.byref(now)) == 0
assert cuda.cuCtxDestroy_v2(own) == 0
assert code == _lib.FA_OK and now.value == own.value
"""
    root = pathlib.Path(__file__).resolve().parent.parent
    done = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stderr[-2000:]


def test_a_thread_whose_context_is_taken_away():
    """Two backward calls of a thread that drops its context behind each."""
    x = {n: t.to(DEV) for n, t in inputs(1, 2, 2, 150, 64, 22).items()}
    o, lse = api.fwd(x["q"], x["k"], x["v"], True, softcap=3.0)
    want = api.bwd(x["q"], x["k"], x["v"], o, x["do"], lse, True, softcap=3.0)
    g = [torch.empty_like(x["q"]) for _ in range(3)]
    ws = torch.empty(api.score_workspace_bytes(x["q"], True), dtype=torch.uint8, device=DEV)
    at = [t.data_ptr() for t in (x["q"], x["k"], x["v"], o, x["do"], lse, *g)]
    torch.cuda.synchronize()
    cuda, codes = ctypes.CDLL("libcuda.so.1"), []

    def work():
        for _ in range(2):
            codes.append(_lib.fa_bwd_score(*at, None, 1, 2, 2, 150, 64, 0.125, 1, _lib.Score(softcap=3.0), ws.data_ptr(), ws.numel(), None))
            codes.append(cuda.cuCtxSetCurrent(None))
    t = threading.Thread(target=work)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert codes == [0, 0, 0, 0]
    assert torch.equal(g[1], want[1]) and torch.equal(g[2], want[2])


def test_python_refusals_on_the_device():
    x = {n: t.to(DEV) for n, t in inputs(1, 4, 2, 100, 64, 5).items()}
    f = lambda **kw: api.fwd(x["q"], kw.pop("k", x["k"]), kw.pop("v", x["v"]), kw.pop("causal", True), **kw)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device=DEV)
    t = dev(table_of(4, 16, 64, False, 1))
    for kw, what in [
        (dict(softcap=0.0), "above 0"), (dict(softcap=-3.0), "above 0"), (dict(slopes=torch.ones(3, device=DEV)), "slopes"),
        (dict(slopes=torch.ones(4)), "slopes"), (dict(slopes=torch.ones(4, device=DEV).double()), "slopes"),
        (dict(bias=t["bias"]), "needs buckets"), (dict(buckets=t["buckets"]), "needs buckets"),
        (dict(slopes=torch.ones(4, device=DEV), **t), "not both"), (dict(t, bias=t["bias"][:, :3]), "bias"),
        (dict(t, bias=t["bias"].half()), "bias"), (dict(t, buckets=t["buckets"][1:]), "buckets"),
        (dict(t, buckets=t["buckets"].long()), "buckets"), (dict(docs=i32(1, 99)), "docs"), (dict(docs=i32(1, 100).long()), "docs"),
        (dict(docs=i32(1, 200)[:, ::2]), "docs"), (dict(prefix=i32(2)), "prefix"), (dict(prefix=i32(1), causal=False), "causal"),
        (dict(softcap=1.0, window=4, causal=False), "causal"), (dict(softcap=1.0, window=0), "at least one"),
        (dict(softcap=1.0, k=x["k"][:, :, :50].contiguous(), v=x["v"][:, :, :50].contiguous()), "keys and values"),
        (dict(softcap=1.0, k=x["q"][:, :3].contiguous(), v=x["q"][:, :3].contiguous()), "multiple"),
        (dict(softcap=1.0, k=x["k"].transpose(1, 2)), "contiguous"),
    ]:
        with pytest.raises(ValueError, match=what):
            f(**kw)
    with pytest.raises(_lib.FAError) as err:
        f(docs=i32(1, 100), workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    assert err.value.code == _lib.FA_ERR_WORKSPACE
    with pytest.raises(_lib.FAError):
        f(softcap=1.0, out=x["q"])
    torch.cuda.synchronize()
    assert api.last_device_error() == _lib.FA_OK
