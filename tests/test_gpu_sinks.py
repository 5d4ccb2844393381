"""GPU parity of windowed attention with sinks (fa_fwd_sinks, fa_bwd_sinks) against the
plain 64-bit form: key j is visible from query i iff j <= i and (j > i - w or j < s).
Bars as for the sliding window, whose kernels these are (see _parity.py)."""
import math

import pytest
import torch

from exact_io_aware_12_gb300 import api, _lib
from exact_io_aware_12_gb300.workloads import draw
from tests import _plain
from tests._parity import check_grad, check_lse, check_o, rel_l2

pytestmark = pytest.mark.gpu
DEV = "cuda"


def gpu(x, tau, window, sinks, backward=True):
    q, k, v = (x[n].to(DEV) for n in ("q", "k", "v"))
    o, lse = api.fwd(q, k, v, True, tau, window=window, sinks=sinks)
    grads = None
    if backward:
        grads = api.bwd(q, k, v, o, x["do"].to(DEV), lse, True, tau, window=window, sinks=sinks)
    torch.cuda.synchronize()
    assert api.last_device_error() == _lib.FA_OK
    return o, lse, grads


def check(x, tau, window, sinks):
    o, lse, g = gpu(x, tau, window, sinks)
    N = x["q"].shape[2]
    see = _plain.visible(N, N, window, sinks)
    o_ref, l_ref, _ = _plain.attention(x["q"], x["k"], x["v"], tau, see)
    check_o(o, o_ref.numpy())
    check_lse(lse, l_ref.numpy())
    for got, ref, name in zip(g, _plain.attention_bwd(x["q"], x["k"], x["v"], x["do"], tau, see), ("dQ", "dK", "dV")):
        check_grad(got, ref.numpy(), name)


# lengths of one and of a few keys, a tile and one key beside it, several tiles; sinks that end
# inside the first block, on its edge, behind it, and that meet the window
CASES = [(1, 1, 1), (5, 2, 1), (127, 40, 3), (128, 64, 64), (129, 1, 1), (300, 1, 4), (300, 100, 130), (300, 17, 128),
         (700, 128, 129), (1000, 129, 4), (1000, 256, 300), (1000, 300, 1), (1025, 128, 256), (1300, 500, 640),
         (640, 300, 400)]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N,w,s", CASES)
def test_sinks_match_plain(N, w, s, d):
    check(draw(2, 2, N, d, seed=1500 + N + w + s + d), 1 / math.sqrt(d), w, s)


def test_random_sizes():
    """Forty seeded sizes: any sum of window and sinks, any raggedness."""
    g = torch.Generator().manual_seed(77)
    r = lambda n: int(torch.randint(1, n + 1, (1,), generator=g))
    for i in range(40):
        N, d = r(900), 64 * r(2)
        check(draw(1, r(3), N, d, seed=3000 + i), 1 / math.sqrt(d), r(N), r(N))


# d = 64 with more (key tile, head) items than SMs: the persistent kernels, whose lists of long (sink)
# and short tiles are dealt over the SMs; long tiles fewer than, equal to and more than SMs
@pytest.mark.parametrize("B,H,N,w,s", [(4, 24, 640, 130, 5), (1, 152, 500, 40, 3), (1, 77, 900, 200, 140),
                                       (4, 48, 333, 100, 1), (2, 160, 300, 64, 129), (1, 31, 1100, 128, 128)])
def test_many_short_heads(B, H, N, w, s):
    check(draw(B, H, N, 64, seed=94 + H), 0.125, w, s)


@pytest.mark.parametrize("d", [64, 128])
def test_heads_do_not_mix(d):
    """A head's forward gives the same bits alone and among others, its dK and dV the same values (the
    order of a long tile's sums may differ)."""
    B, H, N, w, s = 1, 64, 1100, 300, 140
    x = draw(B, H, N, d, seed=95)
    tau = 1 / math.sqrt(d)
    o, lse, g = gpu(x, tau, w, s)
    for h in (0, 31, 63):
        xh = {n: x[n][:, h:h + 1].contiguous() for n in x}
        ho, hl, hg = gpu(xh, tau, w, s)
        assert torch.equal(o[:, h:h + 1], ho) and torch.equal(lse[:, h:h + 1], hl)
        for a, b in zip(g, hg):
            # (two bf16 roundings of values that differ in the last bits of fp32)
            assert rel_l2(a[:, h:h + 1], b) <= 2.0 ** -8


@pytest.mark.parametrize("d", [64, 128])
def test_no_sinks_is_the_window_and_all_sinks_is_causal_bitwise(d):
    N, w = 700, 200
    x = draw(1, 2, N, d, seed=95)
    q, k, v, do = (x[n].to(DEV) for n in ("q", "k", "v", "do"))
    tau = 1 / math.sqrt(d)
    o, lse = torch.empty_like(q), torch.empty(1, 2, N, device=DEV)
    st = torch.cuda.current_stream().cuda_stream
    for sinks, window in ((0, w), (N - w, w), (10 ** 9, w), (3, 10 ** 9)):
        _lib.check(_lib.fa_fwd_sinks(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), 1, 2, N,
                                     d, tau, window, sinks, st), "fa_fwd_sinks")
        want = api.fwd(q, k, v, True, tau, window=w if sinks == 0 else None)
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
        if sinks > 0:   # (dS keeps the precision of sinks: the next test)
            check(x, tau, window, sinks)
            continue
        g = api.bwd(q, k, v, o, do, lse, True, tau, window=window, sinks=sinks)
        gw = api.bwd(q, k, v, o, do, lse, True, tau, window=w)
        assert torch.equal(g[1], gw[1]) and torch.equal(g[2], gw[2])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("w,s", [(200, 5), (200, 500), (10 ** 9, 1)])
def test_ds_is_rounded_once(d, w, s):
    """dQ and dK are sums of products with dS, whose rounding errors are independent: one rounding to
    bf16 of each dS and one of the result, each of about 2^-8 / sqrt(6) = 1.6e-3 (a relative error even
    over half a step, the step relative to the value between 2^-8 and 2^-7), give 2.3e-3 together; a
    third rounding would give 2.8e-3, a fourth 3.2e-3.  The bar is between the two and the three."""
    x = draw(1, 4, 700, d, seed=96)
    tau = 1 / math.sqrt(d)
    _, _, g = gpu(x, tau, w, s)
    see = _plain.visible(700, 700, w, s)
    ref = _plain.attention_bwd(x["q"], x["k"], x["v"], x["do"], tau, see)
    for got, want in zip(g[:2], ref[:2]):
        assert rel_l2(got, want.numpy()) <= 2.65e-3


def test_gradients_against_differences():
    """Directional derivatives of the plain 64-bit forward.  The kernel's gradients are within 1e-2
    of the exact ones (2-norm), so a derivative along a direction u is within 1e-2 |g| |u|, and the
    central difference's own error (step 1e-4, third derivatives of order one) is far below that."""
    N, d, w, s = 260, 64, 50, 5
    tau = 1 / math.sqrt(d)
    x = draw(1, 2, N, d, seed=96)
    _, _, grads = gpu(x, tau, w, s)
    see = _plain.visible(N, N, w, s)
    gen = torch.Generator().manual_seed(5)

    def loss(**kw):
        y = {n: kw.get(n, x[n].double()) for n in ("q", "k", "v")}
        return float((_plain.attention(y["q"], y["k"], y["v"], tau, see)[0] * x["do"].double()).sum())

    for name, g in zip(("q", "k", "v"), grads):
        g = g.cpu().double()
        for _ in range(4):
            u = torch.randn(g.shape, generator=gen, dtype=torch.float64)
            h = 1e-4
            num = (loss(**{name: x[name].double() + h * u}) - loss(**{name: x[name].double() - h * u})) / (2 * h)
            assert abs(num - float((g * u).sum())) <= 1e-2 * float(g.norm() * u.norm())


def test_long_context_rows_and_sink_gradients():
    """16384 tokens, a 4096-token window, four sinks: sampled rows, and the gradients of the sink keys
    and of a late key tile (heads 0 and 15), against the plain form of the rows that reach them."""
    N, d, w, s, H = 16384, 128, 4096, 4, 16
    tau = 1 / math.sqrt(d)
    x = draw(1, H, N, d, seed=97)
    o, lse, (dq, dk, dv) = gpu(x, tau, w, s)
    for h in (0, 15):
        q, k, v, do = (x[n][0, h].double() for n in ("q", "k", "v", "do"))
        o_all, l_all = torch.empty(N, d, dtype=torch.float64), torch.empty(N, dtype=torch.float64)
        keys = torch.cat((torch.arange(s), torch.arange(12160, 12288)))  # sinks and one key tile
        ref_k, ref_v = torch.zeros(len(keys), d, dtype=torch.float64), torch.zeros(len(keys), d, dtype=torch.float64)
        ref_q = torch.empty(N, d, dtype=torch.float64)
        for r0 in range(0, N, 2048):
            r = torch.arange(r0, r0 + 2048)
            j = torch.arange(max(0, r0 - w + 1), r0 + 2048)
            j = torch.cat((torch.arange(min(s, int(j[0]))), j))
            see = (j[None] <= r[:, None]) & ((j[None] > r[:, None] - w) | (j[None] < s))
            oo, ll, p = _plain.attention(q[r], k[j], v[j], tau, see)
            o_all[r], l_all[r] = oo, ll
            ds = p * (do[r] @ v[j].T - (do[r] * oo).sum(-1, keepdim=True)) * tau
            ref_q[r] = ds @ k[j]
            for i, key in enumerate(keys.tolist()):
                at = (j == key).nonzero()
                if len(at):
                    ref_k[i] += ds[:, at[0, 0]] @ q[r]
                    ref_v[i] += p[:, at[0, 0]] @ do[r]
        check_o(o[0, h], o_all.numpy())
        check_lse(lse[0, h], l_all.numpy())
        check_grad(dq[0, h], ref_q.numpy(), "dQ")
        for lo, hi in ((0, s), (s, len(keys))):
            idx = keys[lo:hi].to(DEV)
            check_grad(dk[0, h][idx], ref_k[lo:hi].numpy(), "dK")
            check_grad(dv[0, h][idx], ref_v[lo:hi].numpy(), "dV")


def test_attention_autograd_with_window_and_sinks():
    N, d, w, s = 333, 64, 60, 7
    x = draw(1, 2, N, d, seed=98)
    q, k, v = (x[n].to(DEV).requires_grad_() for n in ("q", "k", "v"))
    api.attention(q, k, v, True, window=w, sinks=s).backward(x["do"].to(DEV))
    see = _plain.visible(N, N, w, s)
    for t, ref, n in zip((q, k, v), _plain.attention_bwd(x["q"], x["k"], x["v"], x["do"], 1 / math.sqrt(d), see), "QKV"):
        check_grad(t.grad, ref.numpy(), "d" + n)


def test_captured_step_replays_on_new_values_and_another_stream():
    N, d, w, s = 520, 128, 100, 9
    tau = 1 / math.sqrt(d)
    xs = [draw(1, 3, N, d, seed=990 + i) for i in range(2)]
    buf = {n: xs[0][n].to(DEV) for n in ("q", "k", "v", "do")}
    ws = torch.empty(api.workspace_bytes(1, 3, N, d), dtype=torch.uint8, device=DEV)

    def step():
        o, lse = api.fwd(buf["q"], buf["k"], buf["v"], True, tau, window=w, sinks=s)
        return (o, lse) + api.bwd(buf["q"], buf["k"], buf["v"], o, buf["do"], lse, True, tau, window=w, sinks=s,
                                  workspace=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for x in xs[::-1]:
        for n in buf:
            buf[n].copy_(x[n])
        graph.replay()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            want = step()
        side.synchronize()
        for i in (0, 1, 3, 4):  # (dQ's sum order differs from run to run)
            assert torch.equal(outs[i], want[i])
        assert rel_l2(outs[2], want[2]) <= 1e-3
    assert api.last_device_error() == _lib.FA_OK


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N", [300, 2049])
def test_all_keys_as_the_largest_number(N, d):
    """sinks and window up to the largest int: plain causal attention, bit by bit."""
    x = draw(1, 2, N, d, seed=101)
    q, k, v = (x[n].to(DEV) for n in ("q", "k", "v"))
    tau, most = 1 / math.sqrt(d), 2 ** 31 - 1
    want = api.fwd(q, k, v, True, tau)
    for w, s in ((1, most), (most, 1), (most, most), (7, most - 126), (7, N - 7)):
        got = api.fwd(q, k, v, True, tau, window=w, sinks=s)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    check(x, tau, 1, most)
    check(x, tau, most, most)


@pytest.mark.parametrize("d", [64, 128])
def test_ds_of_weights_far_below_a_dominant_sink(d):
    """Key 0 outweighs the others by e^17 in every row: their dS = P (dP - D) is a product with P near
    2^-25, and their dK a sum of products with it.  One rounding of dS and one of the result, as above."""
    N, w, s = 700, 200, 5
    tau = 1 / math.sqrt(d)
    x = draw(1, 4, N, d, seed=99)
    x = {n: t.clone() for n, t in x.items()}
    for n in "qk":
        x[n][..., 0] = 0
        x[n] *= 0.5
    x["q"][..., 0] = 8.0
    x["k"][:, :, 0] = 0
    x["k"][:, :, 0, 0] = 17.0 / (8.0 * tau)
    x["v"][:, :, 0] *= 0.0625
    _, _, g = gpu(x, tau, w, s)
    see = _plain.visible(N, N, w, s)
    ref = _plain.attention_bwd(x["q"], x["k"], x["v"], x["do"], tau, see)
    # (all but the last rows of the sequence have hundreds of summands)
    for got, want in zip(g[1:], ref[1:]):
        assert rel_l2(got[:, :, s:500], want[:, :, s:500].numpy()) <= 2.65e-3


def test_ds_of_a_long_flat_window():
    """Keys of zero: every row's weights are 1 over the number of keys that it sees, about 2^-17 behind
    the window, so prefix sums give O and single keys' gradients.  151827 + 3 visible keys: in steps of
    2^-24 that weight would be 110.5 steps, 0.45% from a whole number of them."""
    N, d, w, s = 180000, 128, 151827, 3
    tau = 1 / math.sqrt(d)
    x = draw(1, 1, N, d, seed=100)
    x = {n: t.clone() for n, t in x.items()}
    x["k"].zero_()
    o, lse, (dq, dk, dv) = gpu(x, tau, w, s)
    q, v, do = (x[n][0, 0].double() for n in ("q", "v", "do"))
    i = torch.arange(N)
    first = (i - w + 1).clamp(min=s)          # first key of the window behind the sinks
    seen = torch.where(i < s, i + 1, s + i + 1 - first)
    run = torch.cat((torch.zeros(1, d, dtype=torch.float64), v.cumsum(0)))
    ref_o = torch.where((i < s)[:, None], run[i + 1], run[s] + run[i + 1] - run[first]) / seen[:, None]
    check_o(o[0, 0], ref_o.numpy())
    check_lse(lse[0, 0], seen.double().log().numpy())
    D = (do * ref_o).sum(1)
    for keys in (torch.arange(s), torch.arange(90000, 90032), torch.arange(20000, 20032)):
        ref_k, ref_v = [], []
        for j in keys.tolist():
            rows = slice(j, N if j < s else min(N, j + w))
            p = 1.0 / seen[rows].double()
            ref_v.append(p @ do[rows])
            ref_k.append(tau * ((p * (do[rows] @ v[j] - D[rows])) @ q[rows]))
        # The sinks' dK is mostly of the first rows, P = 1 / n for the n keys that they see, and there D, taken
        # from O in bf16 (off by about 2^-8 / sqrt(6) of |O| = |V| / sqrt(n)), adds to the two roundings:
        # relative to dP - D, of norm sqrt(1 - 1 / n), in all 2^-8 / sqrt(6) times the root of
        # sum n^-3 / sum (n^-2 - n^-3) = 1.202 / 0.443: 2.6e-3, with the 2.3e-3 3.5e-3.
        assert rel_l2(dk[0, 0][keys.to(DEV)], torch.stack(ref_k).numpy()) <= (4e-3 if int(keys[0]) < s else 2.65e-3)
        assert rel_l2(dv[0, 0][keys.to(DEV)], torch.stack(ref_v).numpy()) <= 2.65e-3
    assert float(dq.abs().max()) == 0.0
