"""Attention with capped, biased or masked scores without a GPU: the arithmetic that its kernels
share, compiled here as plain C++ with checks for overflow, against the mask's definition; the
gradients' formulas against differences; the buckets' borders; refusals."""
import ctypes
import math
import os
import random
import subprocess

import pytest
import torch

from exact_io_aware_12_gb300 import _lib, api
from tests import _plain_score

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE, GB = 1 << 40, 1 << 30

SHIM = r'''
#include "fa_score.h"
using namespace fa;
extern "C" {
void t_keys(int i, int s, int e, int c, int p, int w, int* out) { ScoreRange r = keys_of(i, s, e, c, p, w); out[0] = r.lo; out[1] = r.hi; }
void t_queries(int j, int s, int e, int c, int p, int w, int* out) { ScoreRange r = queries_of(j, s, e, c, p, w); out[0] = r.lo; out[1] = r.hi; }
void t_blocks(int lo, int hi, int b, int* out) { ScoreRange r = blocks_of(lo, hi, b); out[0] = r.lo; out[1] = r.hi; }
int t_side(int q, int k, int n, int far) { return far_side(q, k, n, far); }
int t_near(int far, int block) { return near_tiles(far, block); }
}
'''


@pytest.fixture(scope="module")
def shim(tmp_path_factory):
    d = tmp_path_factory.mktemp("score")
    src, lib = d / "shim.cpp", d / "shim.so"
    src.write_text(SHIM)
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-fsanitize=undefined",
                    "-fno-sanitize-recover=undefined", "-static-libubsan",
                    "-I", os.path.join(ROOT, "exact_io_aware_12_gb300", "csrc"), str(src), "-o", str(lib)], check=True)
    return ctypes.CDLL(str(lib))


def two(f, *a):
    out = (ctypes.c_int * 2)()
    f(*a, out)
    return out[0], out[1]


def random_ids(r, N):
    ids, x = [], 0
    while len(ids) < N:
        x = -1 if r.random() < 0.2 else r.randint(0, 5)
        ids += [x] * r.randint(1, max(1, N // 3))
    return ids[:N]


def spans(ids):
    """(first, end) of each token's run, (i, i) for padding."""
    run = _plain_score.runs_of(ids)
    out = []
    for i, x in enumerate(run):
        if x < 0:
            out.append((i, i))
            continue
        a = b = i
        while a > 0 and run[a - 1] == x:
            a -= 1
        while b + 1 < len(run) and run[b + 1] == x:
            b += 1
        out.append((a, b + 1))
    return out


def test_ranges_are_the_mask(shim):
    """Every query's and every key's range is its row and column of the mask, both ends ascend, and a
    tile's blocks hold all that its rows see."""
    r = random.Random(3)
    for _ in range(300):
        N, block = r.randint(1, 40), r.choice([1, 4, 8])
        ids = random_ids(r, N) if r.random() < 0.7 else [0] * N
        causal = r.random() < 0.7
        prefix = r.randint(0, N) if causal and r.random() < 0.5 else 0
        window = r.randint(1, N) if causal and r.random() < 0.4 else 0
        see = _plain_score.seen(1, N, causal, torch.tensor([ids]), torch.tensor([prefix]), window or None)[0, 0]
        sp = spans(ids)
        rows = [two(shim.t_keys, i, *sp[i], int(causal), prefix, window) for i in range(N)]
        cols = [two(shim.t_queries, j, *sp[j], int(causal), prefix, window) for j in range(N)]
        for i in range(N):
            assert see[i].tolist() == [rows[i][0] <= j < rows[i][1] for j in range(N)], (ids, causal, prefix, window, i)
            assert see[:, i].tolist() == [cols[i][0] <= q < cols[i][1] for q in range(N)]
            assert 0 <= rows[i][0] <= rows[i][1] <= N and 0 <= cols[i][0] <= cols[i][1] <= N
        for t in (rows, cols):
            for x, y in zip(t, t[1:]):
                assert x[0] <= y[0] and x[1] <= y[1]
            for a in range(0, N, block):
                z = min(N, a + block) - 1
                lo, hi = two(shim.t_blocks, t[a][0], t[z][1], block)
                assert lo < hi and lo * block < N
                for i in range(a, z + 1):
                    if t[i][0] < t[i][1]:
                        assert lo * block <= t[i][0] and t[i][1] <= hi * block
                # keys that every row sees lie in [last row's first, first row's end)
                for j in range(N):
                    every = all(t[i][0] <= j < t[i][1] for i in range(a, z + 1))
                    assert every == (t[z][0] <= j < t[a][1])


def test_ranges_at_the_largest_sizes(shim):
    N = 65535 * 128
    assert two(shim.t_keys, N - 1, 0, N, 1, N, N) == (0, N)
    assert two(shim.t_queries, N - 1, 0, N, 1, 0, N) == (N - 1, N)
    assert two(shim.t_queries, 0, 0, N, 1, N, 1) == (0, 1)


def test_near_and_far_tiles(shim):
    for far in (1, 2, 127, 128, 129, 130, 255, 256, 257, 1024):
        n = shim.t_near(far, 128)
        for off in range(-12, 13):
            q, k = 2048 + 128 * off, 2048
            dist = [q + a - k - b for a in (0, 127) for b in (0, 127)]
            want = 1 if min(dist) >= far else -1 if max(dist) <= -far else 0
            assert shim.t_side(q, k, 128, far) == want
            assert (abs(off) <= n) == (want == 0)


@pytest.mark.parametrize("case", range(6))
def test_formulas_against_differences(case):
    """The gradients that the kernels are held to, against central differences in 64 bits."""
    g = torch.Generator().manual_seed(case)
    B, H, Hkv, N, d = 2, 4, 2, 13, 8
    x = [torch.randn(B, h, N, d, generator=g, dtype=torch.float64) for h in (H, Hkv, Hkv, H)]
    kw = dict(causal=case % 2 == 0)
    if case in (0, 1, 4):
        kw["softcap"] = 1.5
    if case in (1, 2):
        kw["slopes"] = torch.rand(H, generator=g)
    if case >= 3:
        kw["bias"] = torch.randn(6, H, generator=g, dtype=torch.float64)
        kw["buckets"] = torch.tensor([5, 4, 9, 0, 1, 2, 3])
    if case in (0, 3, 5):
        kw["docs"] = torch.tensor([[0] * 5 + [1] * 6 + [-1] * 2, [-3] + [2] * 12])
    if case == 2:
        kw["prefix"], kw["window"] = torch.tensor([0, 6]), 9
    w = torch.randn(B, H, N, d, generator=g, dtype=torch.float64)
    e = _plain_score.Exact(*x[:3], tau=0.4, do=w, **kw)
    names = {"dq": x[0], "dk": x[1], "dv": x[2]}
    if "bias" in kw:
        names["dbias"] = kw["bias"]
    for name, t in names.items():
        for at in [tuple(int(torch.randint(n, (1,), generator=g)) for n in t.shape) for _ in range(6)]:
            h, keep, got = 1e-5, float(t[at]), []
            for s in (1, -1):
                t[at] = keep + s * h
                got.append(float((_plain_score.Exact(*x[:3], tau=0.4, **kw).o * w).sum()))
            t[at] = keep
            # truncation h^2 / 6 of third derivatives of order 10^3, cancellation 2^-53 of sums of order 10^2 / h
            assert abs((got[0] - got[1]) / (2 * h) - float(getattr(e, name)[at])) <= 1e-6, (name, at)


def border(n, exact, far, x):
    """A side's bucket by logarithms of many digits."""
    from decimal import Decimal, getcontext
    getcontext().prec = 60
    if x <= exact:
        return min(x, n - 1)
    y = (Decimal(x) / exact).ln() / (Decimal(far) / exact).ln() * (n - exact)
    near = y.to_integral_value()
    y = near if abs(y - near) < Decimal(10) ** -40 else y
    return min(n - 1, exact + int(y))


@pytest.mark.parametrize("n,far,both", [(32, 128, True), (32, 128, False), (16, 64, True), (48, 500, False), (2, 9, False),
                                        (4, 1024, True), (3, 10, False), (1024, 1024, False), (64, 1000, True)])
def test_buckets(n, far, both):
    m = api.distance_buckets(n, far, both)
    L = m.numel() // 2
    side = n // 2 if both else n
    want = [border(side, side // 2, far, x) for x in range(L + 1)]
    assert m[L:].tolist() == want
    assert want[-1] == side - 1 and (L == 1 or want[-2] < side - 1)
    assert m[:L].tolist() == ([side + x for x in want[:0:-1]] if both else [0] * L)


def test_buckets_refuse():
    for a in [(1, 128), (32, 16), (31, 128, True), (3, 1, True), (2000, 1024), (32, 2000)]:
        with pytest.raises(ValueError):
            api.distance_buckets(*a)


def score(**kw):
    f = dict(softcap=0.0, slopes=None, bias=None, buckets=None, bias_f32=0, num_buckets=0, max_distance=0, docs=None,
             prefix=None, window=0)
    f.update(kw)
    return _lib.Score(*f.values())


def calls(sc, **kw):
    """The status of the forward and of the backward."""
    a = dict(B=2, H=4, H_kv=2, N=300, d=64, tau=0.125, causal=1)
    a.update({k: v for k, v in kw.items() if k in a})
    p = {n: FAKE + i * GB for i, n in enumerate(("Q", "K", "V", "O", "dO", "LSE", "dQ", "dK", "dV", "ws"))}
    p.update({k: v for k, v in kw.items() if k in p})
    n = kw.get("ws_bytes", GB)
    f = _lib.fa_fwd_score(p["Q"], p["K"], p["V"], p["O"], p["LSE"], *a.values(), sc, p["ws"], n, None)
    b = _lib.fa_bwd_score(p["Q"], p["K"], p["V"], p["O"], p["dO"], p["LSE"], p["dQ"], p["dK"], p["dV"], kw.get("dBias"),
                          *a.values(), sc, p["ws"], n, None)
    return f, b


TABLE = dict(bias=FAKE + 20 * GB, buckets=FAKE + 21 * GB, num_buckets=32, max_distance=100)
BAD, UN, WS, OK = _lib.FA_ERR_INVALID_ARG, _lib.FA_ERR_UNSUPPORTED, _lib.FA_ERR_WORKSPACE, _lib.FA_OK


@pytest.mark.parametrize("f,kw,code", [
    (dict(softcap=-1.0), {}, BAD), (dict(softcap=math.nan), {}, BAD), (dict(softcap=math.inf), {}, BAD),
    (dict(softcap=1e-9), {}, BAD), (dict(softcap=1e30), {}, BAD),
    (dict(slopes=FAKE + 20 * GB + 2), {}, BAD), (dict(TABLE, slopes=FAKE + 22 * GB), {}, BAD),
    (dict(TABLE, buckets=None), {}, BAD), (dict(TABLE, bias=None), {}, BAD), (dict(TABLE, num_buckets=0), {}, BAD),
    (dict(TABLE, max_distance=0), {}, BAD), (dict(TABLE, num_buckets=1025), {}, UN), (dict(TABLE, max_distance=1025), {}, UN),
    (dict(TABLE, bias_f32=2), {}, BAD), (dict(TABLE, bias=FAKE + 20 * GB + 1), {}, BAD),
    (dict(TABLE, bias=FAKE + 20 * GB + 2, bias_f32=1), {}, BAD), (dict(TABLE, buckets=FAKE + 21 * GB + 2), {}, BAD),
    (dict(docs=FAKE + 22 * GB + 1), {}, BAD), (dict(prefix=FAKE + 22 * GB + 2), {}, BAD),
    (dict(prefix=FAKE + 22 * GB), dict(causal=0), BAD), (dict(window=-1), {}, BAD), (dict(window=5), dict(causal=0), BAD),
    ({}, dict(H=3), BAD), ({}, dict(H_kv=0), BAD), ({}, dict(H_kv=-2), BAD), ({}, dict(H=-4), BAD), ({}, dict(N=-1), BAD),
    ({}, dict(d=96), UN), ({}, dict(tau=0.0), BAD), ({}, dict(tau=math.nan), BAD), ({}, dict(causal=2), BAD),
    ({}, dict(N=65535 * 128 + 1), UN), ({}, dict(B=2 ** 20, H=2 ** 8, H_kv=2 ** 8, N=2048), UN),
    ({}, dict(Q=None), BAD), ({}, dict(K=FAKE + 8), BAD), ({}, dict(LSE=None), BAD), ({}, dict(ws=FAKE + 9 * GB + 8), BAD),
    (dict(docs=FAKE + 22 * GB), dict(ws_bytes=100), WS),
    (dict(docs=FAKE + 9 * GB), {}, BAD),                     # over the workspace
    ({}, dict(B=0), OK), ({}, dict(N=0), OK), ({}, dict(H=0, H_kv=0), OK),
])
def test_refusals(f, kw, code):
    assert calls(score(**f), **kw) == (code, code)


def test_refusals_of_one_side():
    assert calls(None) == (BAD, BAD)
    # the forward's outputs over what it reads
    for kw in (dict(O=FAKE), dict(O=FAKE + GB), dict(LSE=FAKE + 2 * GB), dict(O=FAKE + 5 * GB)):
        assert calls(score(), **kw)[0] == BAD
    for name in ("slopes", "docs", "prefix"):
        assert calls(score(**{name: FAKE + 3 * GB}))[0] == BAD
    assert calls(score(**dict(TABLE, buckets=FAKE + 5 * GB)))[0] == BAD
    # the backward's
    for kw in (dict(dQ=FAKE), dict(dK=FAKE + 5 * GB), dict(dV=FAKE + 7 * GB), dict(ws=FAKE + 6 * GB), dict(dO=None),
               dict(dK=FAKE + 6 * GB + 16), dict(ws_bytes=1000)):
        assert calls(score(), **kw)[1] == (WS if "ws_bytes" in kw else BAD)
    assert calls(score(), dBias=FAKE + 23 * GB)[1] == BAD                  # without a bias
    t = score(**TABLE)
    assert calls(t, dBias=FAKE + 20 * GB)[1] == BAD                        # over the bias
    assert calls(t, dBias=FAKE + 8 * GB)[1] == BAD                         # over dV
    assert calls(t, dBias=FAKE + 23 * GB + 1)[1] == BAD
    assert calls(score(**dict(TABLE, bias_f32=1)), dBias=FAKE + 23 * GB + 2)[1] == BAD


def test_keys_that_no_query_head_reads():
    """H = 0 beside H_kv key heads: the backward still writes dK and dV, and checks them."""
    for kw, code in [(dict(dK=None), BAD), (dict(dV=None), BAD), (dict(dK=FAKE + 7 * GB + 8), BAD), (dict(dV=FAKE + 7 * GB), BAD),
                     (dict(dK=FAKE + GB), BAD), (dict(dV=FAKE + 2 * GB), BAD), (dict(d=96), UN), (dict(N=65535 * 128 + 1), UN)]:
        assert calls(score(), H=0, **kw)[1] == code, kw
    assert calls(score(docs=FAKE + 7 * GB), H=0)[1] == BAD
    assert calls(score(), H=0, N=0, dK=None) == calls(score(), H=0, B=0, dV=None) == (OK, OK)


def test_documents_of_nothing():
    """No sequences of no tokens are as empty with documents or a prefix as without."""
    for f in (dict(docs=FAKE + 22 * GB), dict(prefix=FAKE + 22 * GB), TABLE):
        assert calls(score(**f), B=0, N=0) == (OK, OK)


def test_workspace_sizes():
    size = lambda B=2, H=4, N=300, d=64, causal=1, **f: _lib.fa_bwd_score_workspace_size(B, H, N, d, causal, score(**f))
    base = size()
    assert base >= 2 * 4 * 300 * (64 + 1) * 4
    assert size(docs=FAKE) >= base + 2 * 300 * 8
    table = size(**TABLE)
    assert table > base and size(**dict(TABLE, max_distance=200)) > table
    assert size(**dict(TABLE, prefix=FAKE)) > table                        # keys behind the query, too
    assert size(d=96) == size(N=0) == size(window=-1) == size(causal=0, window=4) == 0
    assert _lib.fa_bwd_score_workspace_size(2, 4, 300, 64, 1, None) == 0
    assert _lib.fa_fwd_score_workspace_size(2, 300, score()) == 0
    with_docs = _lib.fa_fwd_score_workspace_size(2, 300, score(docs=FAKE))
    assert 2 * 300 * 8 <= with_docs <= 2 * 300 * 8 + 1024
    assert _lib.fa_fwd_score_workspace_size(2, 300, None) == 0
    q = torch.empty(2, 4, 300, 64, dtype=torch.bfloat16)
    assert api.score_workspace_bytes(q, True) == base
    docs = torch.zeros(2, 300, dtype=torch.int32)
    assert api.score_workspace_bytes(q, True, docs=docs, backward=False) == with_docs
    m = api.distance_buckets(32, 128)
    assert api.score_workspace_bytes(q, True, torch.zeros(32, 4), m) == size(**dict(TABLE, max_distance=m.numel() // 2))


def test_a_frozen_bias_takes_no_workspace_for_its_gradient():
    """Without dBias the call takes what it takes without a bias, and the biases by distance."""
    frozen = lambda **f: _lib.fa_bwd_score_frozen_workspace_size(2, 4, 3000, 64, 0, score(**f))
    whole = lambda **f: _lib.fa_bwd_score_workspace_size(2, 4, 3000, 64, 0, score(**f))
    assert frozen() == whole() and frozen(docs=FAKE) == whole(docs=FAKE)
    t = dict(TABLE, max_distance=1024)
    assert whole() < frozen(**t) <= whole() + 4 * 2049 * 4 + 512
    assert whole(**t) > frozen(**t) + 2 * 4 * 24 * 17 * 4096
    assert _lib.fa_bwd_score_frozen_workspace_size(2, 4, 300, 96, 1, score()) == 0
    a = dict(B=2, H=4, H_kv=4, N=3000, d=64, causal=0)
    n = frozen(**t)
    assert calls(score(**t), ws_bytes=n - 1, **a)[1] == WS and calls(score(**t), ws_bytes=n, dBias=FAKE + 23 * GB, **a)[1] == WS
    # (refused for its workspace's place, not for its size)
    assert calls(score(**t), ws=FAKE + 6 * GB, ws_bytes=n, **a)[1] == BAD
    q = torch.empty(2, 4, 3000, 64, dtype=torch.bfloat16)
    m = torch.zeros(2049, dtype=torch.int32)
    assert api.score_workspace_bytes(q, False, torch.zeros(32, 4), m, bias_grad=False) == n
    assert api.score_workspace_bytes(q, False, torch.zeros(32, 4), m) == whole(**t)


def test_paged_refusals():
    cache = _lib.PagedCache(FAKE, FAKE + GB, None, None, FAKE + 4 * GB, FAKE + 5 * GB, 2, 2, 64, 8, 16, 4)

    def call(sc, fp8=False, **kw):
        fn = _lib.fa_fwd_paged_score_fp8 if fp8 else _lib.fa_fwd_paged_score
        return fn(cache, FAKE + 8 * GB, 256, 64, 64, kw.get("O", FAKE + 9 * GB), 256, 64, 64, FAKE + 10 * GB, 4, 1, 0.125, 0, 0,
                  sc, None, 0, None)
    for f in (dict(docs=FAKE + 20 * GB), dict(prefix=FAKE + 20 * GB), dict(window=4), dict(softcap=-2.0),
              dict(slopes=FAKE + 20 * GB + 1), dict(slopes=FAKE + 9 * GB), dict(TABLE, bias=FAKE + 10 * GB),
              dict(TABLE, buckets=FAKE + 9 * GB), dict(TABLE, slopes=FAKE + 20 * GB)):
        assert call(score(**f)) == BAD, f
    assert call(score(**dict(TABLE, num_buckets=2000))) == UN
    assert call(None) == BAD and call(score(), fp8=True) == BAD


def test_python_checks():
    x = torch.zeros(1, 2, 128, 64, dtype=torch.bfloat16)
    docs = torch.zeros(1, 128, dtype=torch.int32)
    for kw, what in [(dict(softcap=1.0, o_fp32=True), "bf16 O"), (dict(softcap=1.0, window=8, sinks=2), "no sinks"),
                     (dict(docs=docs, blocks=torch.ones(1, 1, dtype=torch.uint8)), "no block mask"),
                     (dict(softcap=1.0), "CUDA"), (dict(workspace=docs), "no workspace")]:
        with pytest.raises(ValueError, match=what):
            api.fwd(x, x, x, True, **kw)
    with pytest.raises(ValueError, match="no sinks"):
        api.bwd(x, x, x, x, x, x, True, softcap=1.0, window=8, sinks=2)
    with pytest.raises(ValueError, match="dbias"):
        api.bwd(x, x, x, x, x, x, True, dbias=x)
    with pytest.raises(ValueError, match="dbias"):
        api.bwd(x, x, x, x, x, x, True, bias=x, buckets=docs, dbias=x, bias_grad=False)
    with pytest.raises(ValueError, match="no sinks"):
        api.attention(x, x, x, True, softcap=1.0, window=8, sinks=2)
    with pytest.raises(ValueError, match="no gradient"):
        api.attention(x, x, x, True, slopes=torch.ones(2, requires_grad=True))
    with pytest.raises(TypeError):
        api.fwd(x, x, None, True, softcap=1.0)


def test_a_bias_gradient_needs_a_bias():
    x, i = torch.zeros(1, 2, 128, 64, dtype=torch.bfloat16), torch.zeros(1, 128, dtype=torch.int32)
    for kw in (dict(softcap=1.0), dict(slopes=torch.ones(2)), dict(docs=i), dict(prefix=i[0, :1])):
        with pytest.raises(ValueError, match="dbias without a bias"):
            api.bwd(x, x, x, x, x, x, True, dbias=x, **kw)


@pytest.mark.parametrize("how", ["plain", "capped", "biased"])
def test_second_derivatives_raise(how, monkeypatch):
    """The kernels' gradients are no constants: whatever of q, k, v, the bias or the incoming gradient they are
    differentiated to, also beside terms that have a derivative.  (Calls of the library replaced by tensors.)"""
    x = [torch.randn(1, 2, 4, 8, requires_grad=True) for _ in range(4)]
    bias = torch.randn(3, 2, requires_grad=True)
    monkeypatch.setattr(api, "fwd", lambda q, *a, **kw: (q.detach().clone(), torch.zeros(1, 2, 4)))
    monkeypatch.setattr(api, "bwd", lambda q, k, v, *a, bias=None, **kw:
                        tuple(t.detach().clone() for t in (q, k, v) + (() if bias is None else (bias,))))
    kw = {"plain": {}, "capped": dict(softcap=2.0), "biased": dict(bias=bias, buckets=torch.zeros(3, dtype=torch.int32))}[how]
    leaves = x[:3] + ([bias] if how == "biased" else [])
    o = api.attention(*x[:3], True, **kw)
    first = torch.autograd.grad(o, leaves, torch.ones_like(o), retain_graph=True)
    assert all(torch.equal(g, t) and not g.requires_grad for g, t in zip(first, leaves))
    for do in (torch.ones_like(o), x[3] * 2):
        grads = torch.autograd.grad(o, leaves, do, create_graph=True)
        for g, t in zip(grads, leaves):
            assert torch.equal(g, t)
            with pytest.raises(RuntimeError, match="no derivative"):
                torch.autograd.grad(g.sum() + x[0].sum() + x[3].sum(), [x[0]], retain_graph=True)
    # frozen inputs, and gradients that are only used
    o = api.attention(x[0].detach(), x[1], x[2].detach(), True, **kw)
    g, = torch.autograd.grad(o, x[1], torch.ones_like(o), create_graph=True)
    with pytest.raises(RuntimeError, match="no derivative"):
        torch.autograd.grad((g * x[1]).sum(), x[1])
    x[1].grad = None
    o = api.attention(*x[:3], True, **kw)
    o.sum().backward(create_graph=True)
    assert torch.equal(x[1].grad, x[1])
