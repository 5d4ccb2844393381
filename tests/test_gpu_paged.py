"""GPU parity of fa_fwd_paged and fa_fwd_paged_fp8 with the plain 64-bit form.

Tolerances, per element, from the exact weights P and scores s (natural units):
  scores  fp32 sums of d exact products and two scalings: off by ds <= (d + 4) 2^-24 tau sum_c |q_c k_c|;
  weights off by e^(2 ds) - 1 (numerator and sum) plus 2^-20 for the exponentials and logarithms,
          and rounded to bf16 (2^-8; fp16 for 8-bit pages: 2^-11) in the numerator only;
  O       rounded once more (2^-8 |O|); fp32 sums over n keys in pieces: at most 2^-24 * 64 + 2^-18 in all;
  LSE     2 ds + 2^-19 + 2^-23 |LSE|."""
import math

import pytest
import torch

from exact_io_aware_12_gb300 import api, _lib
from tests import _plain
from tests._plain import BF16_HALF, FP16_HALF, FP32_HALF

pytestmark = pytest.mark.gpu
DEV = "cuda"


def build(lens, H, Hkv, Nq, d, page, fp8, seed, poison=True, q_gain=1.0, one_scale=False):
    g = torch.Generator().manual_seed(seed)
    P, table = _plain.make_pages(lens, page, g)
    s = dict(table=table, lens=torch.tensor(lens, dtype=torch.int32),
             q=(q_gain * torch.randn(len(lens), H, Nq, d, generator=g)).to(torch.bfloat16))
    for n in "kv":
        x = torch.randn(P, Hkv, page, d, generator=g)
        if fp8:
            sc = 2.0 ** torch.randint(-9, -6, (P, Hkv), generator=g).float()
            if not one_scale:   # (any positive scale is allowed)
                sc = sc * (1 + torch.rand(P, Hkv, generator=g))
            x = (x / sc[:, :, None, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
            s[n + "_scale"] = sc
        else:
            x = x.to(torch.bfloat16)
            s[n + "_scale"] = None
        if poison:
            # rows behind a sequence's end, and pages of no sequence, hold NaN
            raw = x.view(torch.uint8) if fp8 else x.view(torch.int16)
            used = torch.zeros(P, page, dtype=torch.bool)
            for b, ln in enumerate(lens):
                j = torch.arange(ln)
                used[table[b, j // page].long(), j % page] = True
            raw[~used[:, None].expand(P, Hkv, page)] = 0x7F if fp8 else 0x7FC0
        s[n + "c"] = x
    return s


def run(s, window=None, sinks=0, **kw):
    dev = {n: (t.to(DEV) if t is not None else None) for n, t in s.items()}
    o, lse = api.fwd_paged(dev["q"], dev["kc"], dev["vc"], dev["table"], dev["lens"], window=window, sinks=sinks,
                           k_scale=dev["k_scale"], v_scale=dev["v_scale"], **kw)
    torch.cuda.synchronize()
    return o.cpu(), lse.cpu()


def check(s, window=None, sinks=0, got=None, tau=None, seqs=None):
    """Compares with the plain form, sequence by sequence."""
    o, lse = got if got is not None else run(s, window, sinks, **({} if tau is None else dict(tau=tau)))
    B, H, Nq, d = s["q"].shape
    fp8 = s["k_scale"] is not None
    Hkv = s["kc"].shape[1]
    tau = 1 / math.sqrt(d) if tau is None else tau
    for b in (range(B) if seqs is None else seqs):
        n = int(s["lens"][b])
        k, v = (_plain.gather(s[c + "c"], s["table"][b], n, s[c + "_scale"]) for c in "kv")
        k, v = (x.repeat_interleave(H // Hkv, 0) for x in (k, v))
        see = _plain.visible(Nq, n, window or 0, sinks)
        any_row = see.any(0)
        k, v = (torch.where(any_row[None, :, None], x, torch.zeros_like(x)) for x in (k, v))
        q = s["q"][b].double()
        ref, l_ref, p = _plain.attention(q, k, v, tau, see)
        ds = (d + 4) * FP32_HALF * tau * (q.abs() @ k.abs().transpose(-1, -2))
        ds = torch.where(see, ds, torch.zeros_like(ds)).amax(-1, keepdim=True) if n else torch.zeros(H, Nq, 1)
        spread = p @ v.abs()                    # sum_j P |v|
        w = torch.expm1(2 * ds) + 2.0 ** -20 + (FP16_HALF if fp8 else BF16_HALF)
        tol = w * spread + BF16_HALF * ref.abs() + (64 * FP32_HALF + 2.0 ** -18) * spread + 1e-30
        off = (o[b].double() - ref).abs()
        assert bool((off <= tol).all()), f"sequence {b} (len {n}): O off by {float(off.max())}, {float((off - tol).max())} over"
        fin = torch.isfinite(l_ref)
        assert torch.equal(fin, torch.isfinite(lse[b])) and bool((lse[b][~fin] == -math.inf).all())
        l_tol = 2 * ds[..., 0] + 2.0 ** -19 + 2 * FP32_HALF * l_ref.abs()
        assert bool(((lse[b].double() - l_ref).abs()[fin] <= l_tol[fin]).all()), f"sequence {b}: LSE"
        assert bool((o[b][~fin] == 0).all())
    return o, lse


# lengths 0 and 1, fewer keys than rows, page and tile borders, several shares
LENS = [0, 1, 2, 7, 15, 16, 17, 63, 64, 65, 127, 130, 300, 1000, 4097]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,Hkv,Nq,page", [(1, 1, 1, 16), (4, 4, 1, 32), (8, 1, 1, 64), (12, 4, 2, 64), (16, 2, 1, 128),
                                           (6, 2, 5, 16), (8, 2, 8, 256), (20, 1, 2, 32), (24, 3, 8, 64), (3, 1, 7, 64)])
def test_paged_matches_plain(H, Hkv, Nq, page, d, fp8):
    s = build(LENS, H, Hkv, Nq, d, page, fp8, seed=H + Hkv + Nq + d)
    check(s)
    assert api.last_device_error() == _lib.FA_OK


# tables short enough for a block per segment, with rows that need one, two and four warps; more rows
# than one group of warps takes
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("H,Hkv,Nq,d,page,longest", [(3, 3, 1, 64, 16, 600), (8, 2, 1, 128, 32, 640), (4, 1, 3, 128, 16, 300),
                                                     (8, 2, 8, 64, 64, 256), (24, 3, 8, 128, 16, 160), (40, 1, 3, 64, 16, 100),
                                                     (12, 1, 8, 128, 32, 1500), (1, 1, 8, 64, 16, 17), (2, 1, 1, 128, 16, 1)])
def test_short_tables_and_many_rows(H, Hkv, Nq, d, page, longest, fp8):
    lens = [longest] + [n for n in LENS if n < longest]
    s = build(lens, H, Hkv, Nq, d, page, fp8, seed=H + Nq + longest)
    check(s)
    check(s, 37, 6)


# tables too long for whole segments, split over all warps: every number of row warps and groups, short
# and empty sequences among long ones, shares that cut a segment many times and segments that share one
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,Hkv,Nq,page", [(2, 2, 1, 64), (8, 1, 1, 16), (4, 2, 5, 64), (8, 2, 8, 128), (7, 1, 8, 32), (12, 1, 8, 64)])
def test_long_tables_are_split(H, Hkv, Nq, page, d, fp8):
    s = build([11111, 0, 3, 4097, 700, 1, 90], H, Hkv, Nq, d, page, fp8, seed=7 * H + Nq + d)
    assert api.paged_workspace_bytes(s["q"], s["kc"], s["table"]) > 0
    check(s)
    check(s, 10500, 40)


# more short segments than SMs: four warps to a block (eight above, where each has an SM to itself)
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("H,Hkv,Nq,d,longest", [(8, 4, 1, 128, 600), (24, 3, 8, 128, 150), (12, 3, 5, 64, 300), (4, 4, 1, 64, 100)])
def test_many_short_segments(H, Hkv, Nq, d, longest, fp8):
    s = build([longest] + [(7 * i) % longest for i in range(59)], H, Hkv, Nq, d, 16, fp8, seed=H + longest)
    check(s)
    check(s, 37, 6)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (5, 3), (16, 16), (64, 0), (100, 17), (128, 200), (5000, 4)])
def test_window_and_sinks(window, sinks, fp8):
    for H, Hkv, Nq, d, page in ((4, 2, 1, 128, 64), (6, 3, 4, 64, 16), (16, 1, 8, 128, 32)):
        s = build(LENS, H, Hkv, Nq, d, page, fp8, seed=window + sinks + Nq)
        check(s, window, sinks)
    assert api.last_device_error() == _lib.FA_OK


@pytest.mark.parametrize("fp8", [False, True])
def test_random_batches(fp8):
    g = torch.Generator().manual_seed(4)
    r = lambda lo, hi: int(torch.randint(lo, hi + 1, (1,), generator=g))
    for i in range(30):
        Hkv, G, Nq = r(1, 5), r(1, 9), r(1, 8)
        lens = [r(0, 10 ** r(1, 3) * 3) for _ in range(r(1, 40))]
        window = r(1, 700) if r(0, 1) else None
        check(build(lens, Hkv * G, Hkv, Nq, 64 * r(1, 2), 16 << r(0, 4), fp8, seed=i), window, r(0, 90) if window else 0)


@pytest.mark.parametrize("fp8", [False, True])
def test_long_and_many(fp8):
    """One long cache cut into a piece per resident CTA, and many short ones (whole segments)."""
    check(build([70001], 8, 2, 1, 128, 64, fp8, seed=1))
    check(build([40000, 3], 2, 1, 4, 64, 16, fp8, seed=2))
    g = torch.Generator().manual_seed(3)
    lens = torch.randint(0, 200, (700,), generator=g).tolist()
    check(build(lens, 4, 2, 1, 64, 32, fp8, seed=4), seqs=list(range(0, 700, 37)) + [699])


@pytest.mark.parametrize("fp8", [False, True])
def test_peaked_and_flat_scores(fp8):
    """One dominant key, equal scores, and scores that rise along the keys by far more than the
    running max's slack."""
    s = build([500], 4, 2, 1, 128, 32, fp8, seed=5, q_gain=30.0)
    check(s)
    s = build([500], 4, 2, 2, 128, 32, fp8, seed=6)
    s["q"].zero_()
    check(s)
    s = build([600], 2, 1, 1, 64, 16, fp8, seed=7, one_scale=True)
    ids = s["table"][0].long()
    for j in range(600):
        row = torch.full((64,), (j - 300) / 300.0)
        at = (ids[j // 16], 0, j % 16)
        if fp8:
            s["kc"].view(torch.uint8)[at] = (row / s["k_scale"][at[0], 0]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        else:
            s["kc"][at] = row.bfloat16()
    s["q"].fill_(40.0)
    check(s)


def test_8_bit_pages_of_very_different_scales():
    """V scales from 2^-60 to 2^60 page by page, the large ones under small weights and the other way
    round: each row's error stays relative to what it sums."""
    for up in (True, False):
        s = build([320], 4, 2, 1, 128, 16, True, seed=8, one_scale=True)
        ids = s["table"][0, :20].long()
        e = torch.linspace(-60, 60, 20).round()
        s["v_scale"][ids] = (2.0 ** (e if up else -e))[:, None].float().expand(20, 2).contiguous()
        check(s)
        s["k_scale"][ids] = (2.0 ** torch.linspace(-14, -7, 20).round())[:, None].expand(20, 2).contiguous()
        check(s)
    # rows of large and tiny queries
    s = build([100], 4, 2, 2, 64, 16, True, seed=9, one_scale=True)
    s["q"][:, 0] *= 2.0 ** 100
    s["k_scale"] *= 2.0 ** -100
    check(s, seqs=[0])
    s = build([100], 4, 2, 2, 64, 16, True, seed=9)
    s["q"][0, 0, 0, 1:] *= 2.0 ** -20   # (one large column, the rest far below it)
    s["q"][0, 1] *= 2.0 ** -60
    check(s)


@pytest.mark.parametrize("fp8", [False, True])
def test_strides_orders_and_given_buffers(fp8):
    s = build([40, 0, 77], 4, 2, 3, 64, 16, fp8, seed=10)
    want = check(s)
    B, H, Nq, d = s["q"].shape
    for perm in ((0, 2, 1, 3), (1, 0, 2, 3), (2, 1, 0, 3)):
        inv = [perm.index(i) for i in range(4)]
        wide = torch.zeros([s["q"].shape[i] for i in perm[:3]] + [d + 8], dtype=torch.bfloat16)
        view = wide[..., :d].permute(inv)
        view.copy_(s["q"])
        dev = wide.to(DEV)[..., :d].permute(inv)
        out = torch.full(wide.shape, 3.0, dtype=torch.bfloat16, device=DEV)
        lse = torch.empty(B, H, Nq, device=DEV)
        ws = torch.empty(max(1, api.paged_workspace_bytes(s["q"], s["kc"], s["table"])), dtype=torch.uint8, device=DEV)
        d2 = {n: (t.to(DEV) if t is not None else None) for n, t in s.items()}
        o, l = api.fwd_paged(dev, d2["kc"], d2["vc"], d2["table"], d2["lens"], k_scale=d2["k_scale"],
                             v_scale=d2["v_scale"], out=out[..., :d].permute(inv), lse=lse, workspace=ws)
        assert l is lse and torch.equal(o.cpu(), want[0]) and torch.equal(lse.cpu(), want[1])
        assert bool((out[..., d:] == 3).all())   # what lies between the rows stays
    # one query broadcast over rows (stride 0)
    q1 = s["q"][:, :, :1].expand(B, H, Nq, d)
    check(dict(s, q=q1.contiguous()), got=run(dict(s, q=s["q"][:, :, :1].to(DEV).expand(B, H, Nq, d))))


def test_workspace_given_or_taken_by_the_library():
    s = build([14000, 5], 4, 2, 1, 64, 16, False, seed=11)   # (too long for whole segments)
    assert api.paged_workspace_bytes(s["q"], s["kc"], s["table"]) > 0
    want = run(s)
    dev = {n: t.to(DEV) for n, t in s.items() if t is not None}
    P, Hkv, page, d = dev["kc"].shape
    c = _lib.PagedCache(dev["kc"].data_ptr(), dev["vc"].data_ptr(), None, None, dev["table"].data_ptr(),
                        dev["lens"].data_ptr(), 2, Hkv, d, P, page, dev["table"].shape[1])
    o, lse = torch.empty_like(dev["q"]), torch.empty(2, 4, 1, device=DEV)
    code = _lib.fa_fwd_paged(c, dev["q"].data_ptr(), *dev["q"].stride()[:3], o.data_ptr(), *o.stride()[:3], lse.data_ptr(),
                             4, 1, 0.125, 0, 0, None, 0, torch.cuda.current_stream().cuda_stream)
    assert code == _lib.FA_OK
    torch.cuda.synchronize()
    assert torch.equal(o.cpu(), want[0]) and torch.equal(lse.cpu(), want[1])


@pytest.mark.parametrize("fp8", [False, True])
def test_nan_and_infinity_in_hidden_keys(fp8):
    """Keys that no row of the call sees - behind the window, past the sinks - may hold anything."""
    s = build([300], 4, 2, 3, 128, 16, fp8, seed=12)
    window, sinks = 60, 5
    j = torch.arange(300)
    hidden = ~_plain.visible(3, 300, window, sinks).any(0)
    j = j[hidden]
    at = (s["table"][0, j // 16].long(), slice(None), j % 16)
    for n in "kv":
        if fp8:
            s[n + "c"].view(torch.uint8)[at] = 0x7F
        else:
            s[n + "c"][at] = math.inf if n == "k" else math.nan
    check(s, window, sinks)


@pytest.mark.parametrize("fp8", [False, True])
def test_nan_that_is_seen_shows(fp8):
    s = build([100, 100], 2, 1, 1, 64, 16, fp8, seed=13)
    page = int(s["table"][0, 3])
    if fp8:
        s["kc"].view(torch.uint8)[page, 0, 2] = 0x7F
    else:
        s["kc"][page, 0, 2] = math.nan
    o, lse = run(s)
    assert bool(torch.isnan(o[0]).all()) and bool(torch.isnan(lse[0]).all())
    check(s, got=(o, lse), seqs=[1])
    # every key NaN
    s = build([40], 2, 1, 1, 64, 16, fp8, seed=14)
    (s["kc"].view(torch.uint8) if fp8 else s["kc"]).fill_(0x7F if fp8 else math.nan)
    o, lse = run(s)
    assert bool(torch.isnan(o).all()) and bool(torch.isnan(lse).all())


@pytest.mark.parametrize("fp8", [False, True])
def test_bad_pages_are_hidden_and_reported(fp8):
    s = build([100, 50, 64, 30], 4, 2, 1, 64, 16, fp8, seed=15)
    s2 = dict(s, table=s["table"].clone(), lens=s["lens"].clone())
    s2["table"][0, 2] = s["kc"].shape[0]
    s2["table"][0, 4] = -7
    s2["lens"][1] = -3
    s2["lens"][2] = 10 ** 6       # cut to the table's 7 pages, of which this sequence has 4
    o, lse = run(s2)
    assert api.last_device_error() == _lib.FA_ERR_PAGE
    assert api.last_device_error() == _lib.FA_OK
    # the plain form of what is left: sequence 0 without keys 32-47 and 64-79
    j = torch.arange(100)
    keep = j[~((j // 16 == 2) | (j // 16 == 4))]
    k, v = (_plain.gather(s[c + "c"], s["table"][0], 100, s[c + "_scale"])[:, keep].repeat_interleave(2, 0) for c in "kv")
    ref, l_ref, _ = _plain.attention(s["q"][0], k, v, 0.125, torch.ones(1, len(keep), dtype=torch.bool))
    assert float((o[0].double() - ref).abs().max()) <= 1e-2 and float((lse[0].double() - l_ref).abs().max()) <= 1e-4
    assert bool((o[1] == 0).all()) and bool((lse[1] == -math.inf).all())
    check(s, got=(o, lse), seqs=[2, 3])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("longest", [300, 2000])
def test_pages_shared_by_sequences_and_named_twice(fp8, longest):
    s = build([longest, longest - 40, 90], 8, 2, 2, 64, 16, fp8, seed=39, poison=False)
    s["table"][1, :5] = s["table"][0, :5]      # a common beginning
    s["table"][2, :4] = s["table"][0, 1:5]
    s["table"][0, 7] = s["table"][0, 2]        # one page twice
    check(s)
    check(s, 50, 20)


def test_errors_of_the_library_are_raised():
    s = build([100], 2, 1, 1, 64, 16, False, seed=40)
    q = s["q"].to(DEV).expand(1, 2, 9, 64).contiguous()
    with pytest.raises(_lib.FAError) as e:
        api.fwd_paged(q, *(s[n].to(DEV) for n in ("kc", "vc", "table", "lens")))
    assert e.value.code == _lib.FA_ERR_UNSUPPORTED
    with pytest.raises(_lib.FAError) as e:
        api.fwd_paged(s["q"].to(DEV), *(s[n].to(DEV) for n in ("kc", "vc", "table", "lens")), tau=-1.0)
    assert e.value.code == _lib.FA_ERR_INVALID_ARG


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("longest", [200, 2900, 12000])
def test_calls_in_a_row_wait_for_one_another(fp8, longest):
    """Each call's inputs are written by the kernel right before it, without a pause between: the same
    bits as with one after each."""
    H, Hkv, d, page = 8, 2, 128, 64
    lens = [longest, 1, longest // 2]
    s = build(lens, H, Hkv, 1, d, page, fp8, seed=41, one_scale=True)
    room = (longest + 30) // page + 1
    P = 3 * room
    table = torch.arange(P, dtype=torch.int32).reshape(3, room).to(DEV)
    x0 = torch.randn(3, H + 2 * Hkv, d, generator=torch.Generator().manual_seed(42)).to(torch.bfloat16).to(DEV)
    f = (10000.0 ** (-torch.arange(d // 2, dtype=torch.float64) * 2 / d)).to(DEV)
    outs = []
    for pause in (True, False):
        kc, vc = (torch.zeros(P, Hkv, page, d, dtype=torch.uint8 if fp8 else torch.bfloat16, device=DEV) for _ in "kv")
        ks, vs = ((torch.full((P, Hkv), 2.0 ** -7, device=DEV) for _ in "kv") if fp8 else (None, None))
        ln, x, o = torch.tensor(lens, dtype=torch.int32, device=DEV), x0.clone(), None
        q = torch.empty(3, H, d, dtype=torch.bfloat16, device=DEV)
        out = torch.empty(3, H, 1, d, dtype=torch.bfloat16, device=DEV)
        torch.cuda.synchronize()
        for i in range(25):
            x.mul_(0.9375).add_(x.roll(1, 2), alpha=0.5)
            for step in (lambda: api.kv_append(x[:, H:H + Hkv], x[:, H + Hkv:], kc, vc, table, ln, q=x[:, :H],
                                               inv_freq=f, k_scale=ks, v_scale=vs, q_out=q),
                         lambda: ln.add_(1),
                         lambda: api.fwd_paged(q.unsqueeze(2), kc, vc, table, ln, k_scale=ks, v_scale=vs, out=out),
                         lambda: x[:, :H].copy_(out.squeeze(2))):
                step()
                if pause:
                    torch.cuda.synchronize()
        torch.cuda.synchronize()
        outs.append((x.cpu(), kc.cpu(), vc.cpu(), out.cpu()))
    for a, b in zip(*outs):
        assert torch.equal(a, b)
    assert bool(torch.isfinite(outs[0][3].float()).all()) and api.last_device_error() == _lib.FA_OK


@pytest.mark.parametrize("longest", [200, 3000, 11000])
def test_captured_behind_a_copy_and_a_join(longest):
    """A graph in which the calls follow a copy, a fork and a join of streams, and two graphs with buffers
    of their own that run at the same time."""
    H, Hkv, d, page = 8, 2, 64, 16
    s = build([longest - 1, 77], H, Hkv, 1, d, page, False, seed=43, poison=False)
    dev = {n: s[n].to(DEV) for n in ("kc", "vc", "table", "lens")}
    g = torch.Generator().manual_seed(44)
    xs = [torch.randn(2, H + 2 * Hkv, d, generator=g).to(torch.bfloat16).to(DEV) for _ in range(3)]
    f = (10000.0 ** (-torch.arange(d // 2, dtype=torch.float64) * 2 / d)).to(DEV)

    def step(st, fork):
        st["x"].copy_(st["src"])
        main = torch.cuda.current_stream()
        fork.wait_stream(main)
        with torch.cuda.stream(fork):
            st["ln"].copy_(dev["lens"])
            st["ln1"].copy_(dev["lens"]).add_(1)
        st["x"].mul_(2.0)
        main.wait_stream(fork)
        q = api.kv_append(st["x"][:, H:H + Hkv], st["x"][:, H + Hkv:], st["kc"], st["vc"], dev["table"], st["ln"],
                          q=st["x"][:, :H], inv_freq=f)
        o, lse = api.fwd_paged(q.unsqueeze(2), st["kc"], st["vc"], dev["table"], st["ln1"])
        st["o"].copy_(o)

    def state():
        return dict(src=xs[0].clone(), x=torch.zeros_like(xs[0]), kc=dev["kc"].clone(), vc=dev["vc"].clone(),
                    ln=torch.zeros_like(dev["lens"]), ln1=torch.zeros_like(dev["lens"]),
                    o=torch.zeros(2, H, 1, d, dtype=torch.bfloat16, device=DEV))
    fork, sides = torch.cuda.Stream(), [torch.cuda.Stream(), torch.cuda.Stream()]
    want, ref = [], state()
    for x in xs:
        ref["src"].copy_(x)
        step(ref, fork)
        torch.cuda.synchronize()
        want.append(ref["o"].clone())
    states, graphs = [state(), state()], [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    for st, gr in zip(states, graphs):
        with torch.cuda.graph(gr):
            step(st, fork)
    for i in range(6):
        for k in range(2):
            states[k]["src"].copy_(xs[(i + k) % 3])
        torch.cuda.synchronize()
        for side, gr in zip(sides, graphs):
            with torch.cuda.stream(side):
                gr.replay()
        torch.cuda.synchronize()
        for k in range(2):
            assert torch.equal(states[k]["o"], want[(i + k) % 3])
    assert api.last_device_error() == _lib.FA_OK


def test_two_streams_two_workspaces():
    a, b = build([12000, 10, 500], 8, 2, 1, 128, 64, False, seed=16), build([11500], 8, 2, 2, 128, 64, True, seed=17)
    dev = [{n: (t.to(DEV) if t is not None else None) for n, t in s.items()} for s in (a, b)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = [None, None]
    for _ in range(20):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                x = dev[i]
                outs[i] = api.fwd_paged(x["q"], x["kc"], x["vc"], x["table"], x["lens"], k_scale=x["k_scale"],
                                        v_scale=x["v_scale"])
    torch.cuda.synchronize()
    for s, got in zip((a, b), outs):
        check(s, got=tuple(t.cpu() for t in got))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("longest", [5000, 13000])
def test_runs_are_bitwise_alike(fp8, longest):
    s = build([longest, 1, 777, 64], 8, 2, 3, 128, 64, fp8, seed=18)
    a = run(s)
    for _ in range(3):
        b = run(s)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_equals_the_contiguous_decode():
    """A full batch of equal lengths in pages against fa_fwd_decode on the same keys."""
    B, H, Nq, Nk, d = 2, 4, 4, 1000, 128
    s = build([Nk] * B, H, H, Nq, d, 64, False, seed=19)
    o, lse = run(s)
    k, v = (torch.stack([_plain.gather(s[c + "c"], s["table"][b], Nk) for b in range(B)]).to(torch.bfloat16).to(DEV) for c in "kv")
    od, ld = api.fwd_decode(s["q"].to(DEV), k, v, True)
    assert float((o.float() - od.cpu().float()).abs().max()) <= 1e-2
    assert float((lse - ld.cpu()).abs().max()) <= 1e-4


@pytest.mark.parametrize("fp8", [False, True])
def test_generation_append_then_attend(fp8):
    """As a server uses them: a prompt appended in two chunks, then tokens one at a time in a captured
    graph (append, lengths, attention with window and sinks), each step against the plain form on the
    cache as it then is, and the cache against all the keys at the end."""
    B, H, Hkv, d, page, window, sinks = 3, 8, 2, 128, 16, 70, 4
    g = torch.Generator().manual_seed(20)
    prompt, gen = [50, 7, 33], 40
    P, table = _plain.make_pages([n + gen for n in prompt], page, g)
    dt = torch.uint8 if fp8 else torch.bfloat16
    kc, vc = (torch.zeros(P, Hkv, page, d, dtype=dt, device=DEV) for _ in "kv")
    ks, vs = (torch.ones(P, Hkv, device=DEV) if fp8 else None for _ in "kv")
    table, lens = table.to(DEV), torch.zeros(B, dtype=torch.int32, device=DEV)
    f = (10000.0 ** (-2.0 * torch.arange(d // 2, dtype=torch.float64) / d)).to(DEV)
    sc = dict(k_scale=ks, v_scale=vs)
    keys = [[] for _ in range(B)]
    for part in (0, 1):
        n = [p - p // 2 if part else p // 2 for p in prompt]
        x = torch.randn(sum(n), 2 * Hkv, d, generator=g).to(torch.bfloat16)
        cu = torch.tensor([0, n[0], n[0] + n[1], sum(n)], dtype=torch.int32, device=DEV)
        xd = x.to(DEV)
        api.kv_append(xd[:, :Hkv], xd[:, Hkv:], kc, vc, table, lens, cu_new=cu, inv_freq=f, **sc)
        lens.add_(cu[1:] - cu[:-1])
        for b in range(B):
            keys[b].append(x[int(cu[b]):int(cu[b + 1])])
    x = torch.zeros(B, H + 2 * Hkv, d, dtype=torch.bfloat16, device=DEV)
    ws = torch.empty(max(1, api.paged_workspace_bytes(torch.empty(B, H, 1, d), kc, table, window, sinks)),
                     dtype=torch.uint8, device=DEV)

    def step():
        q = api.kv_append(x[:, H:H + Hkv], x[:, H + Hkv:], kc, vc, table, lens, q=x[:, :H], inv_freq=f, **sc)
        lens.add_(1)
        return (q,) + api.fwd_paged(q[:, :, None], kc, vc, table, lens, window=window, sinks=sinks, workspace=ws, **sc)
    saved = [t.clone() if t is not None else None for t in (kc, vc, lens, ks, vs)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    for t, o in zip((kc, vc, lens, ks, vs), saved):
        if t is not None:
            t.copy_(o)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q, o, lse = step()
    for i in range(gen):
        rows = torch.randn(B, H + 2 * Hkv, d, generator=g).to(torch.bfloat16)
        x.copy_(rows)
        graph.replay()
        torch.cuda.synchronize()
        for b in range(B):
            keys[b].append(rows[b:b + 1, H:])
        if i % 6 == 0 or i == gen - 1:
            view = lambda c: c.cpu().view(torch.float8_e4m3fn) if fp8 else c.cpu()
            s = dict(q=q.cpu()[:, :, None], kc=view(kc), vc=view(vc), table=table.cpu(), lens=lens.cpu(),
                     k_scale=ks.cpu() if fp8 else None, v_scale=vs.cpu() if fp8 else None)
            check(s, window, sinks, got=(o.cpu(), lse.cpu()))
    assert lens.tolist() == [n + gen for n in prompt] and api.last_device_error() == _lib.FA_OK
    for b in range(B):
        x = torch.cat(keys[b])
        pos = torch.arange(len(x))
        k_ref = _plain.rotate(x[:, :Hkv], pos, f.cpu(), False).transpose(0, 1)
        v_ref = x[:, Hkv:].double().transpose(0, 1)
        view = lambda c: c.cpu().view(torch.float8_e4m3fn) if fp8 else c.cpu()
        k_got = _plain.gather(view(kc), table[b].cpu(), len(x), ks.cpu() if fp8 else None)
        v_got = _plain.gather(view(vc), table[b].cpu(), len(x), vs.cpu() if fp8 else None)
        if fp8:
            # one rounding, and for held codes rescaling that is exact above the subnormals: half a
            # step, plus half the subnormals' step per rescaling (a page of 16 grows fewer than 16 times)
            for got, ref, scale in ((k_got, k_ref, ks), (v_got, v_ref, vs)):
                ids = table[b, :-(-len(x) // page)].long().cpu()
                step_ = scale.cpu().double()[ids].repeat_interleave(page, 0)[:len(x)].T[..., None]
                assert bool(((got - ref).abs() <= _plain.E4M3_HALF * ref.abs() + 16 * 2.0 ** -10 * step_ + 1e-5).all())
        else:
            assert bool(((k_got - k_ref).abs() <= BF16_HALF * k_ref.abs() + 2.0 ** -18).all())
            assert torch.equal(v_got, v_ref)


@pytest.mark.parametrize("fp8", [False, True])
def test_offsets_past_32_bits(fp8):
    """A cache of more than 2^32 bytes (and, in bf16, elements): pages at its far end."""
    Hkv, page, d = 16, 256, 128
    P = 2 ** 33 // (Hkv * page * d) + 8
    kc = torch.zeros(P, Hkv, page, d, dtype=torch.uint8 if fp8 else torch.bfloat16, device=DEV)
    vc = torch.zeros_like(kc)
    ids = [P - 1, 3, P - 2]
    table = torch.tensor([ids], dtype=torch.int32, device=DEV)
    lens = torch.zeros(1, dtype=torch.int32, device=DEV)
    sc = dict(k_scale=torch.ones(P, Hkv, device=DEV), v_scale=torch.ones(P, Hkv, device=DEV)) if fp8 else {}
    g = torch.Generator().manual_seed(21)
    x = torch.randn(700, 2 * Hkv, d, generator=g).to(torch.bfloat16).to(DEV)
    api.kv_append(x[:, :Hkv], x[:, Hkv:], kc, vc, table, lens, **sc)
    lens.fill_(700)
    q = torch.randn(1, Hkv, 1, d, generator=g).to(torch.bfloat16)
    o, lse = api.fwd_paged(q.to(DEV), kc, vc, table, lens, **sc)
    torch.cuda.synchronize()
    assert api.last_device_error() == _lib.FA_OK
    view = lambda c: c[ids].cpu().view(torch.float8_e4m3fn) if fp8 else c[ids].cpu()
    s = dict(q=q, kc=view(kc), vc=view(vc), table=torch.tensor([[0, 1, 2]]), lens=lens.cpu(),
             k_scale=sc["k_scale"][ids].cpu() if fp8 else None, v_scale=sc["v_scale"][ids].cpu() if fp8 else None)
    check(s, got=(o.cpu(), lse.cpu()))
    if not fp8:
        assert torch.equal(_plain.gather(s["vc"], s["table"][0], 700).float(), x[:, Hkv:].cpu().transpose(0, 1).float())


# Weights of 8-bit pages are rounded to fp16.  One key of value zero (a sink) that outweighs the others
# leaves O to weights far below the running max: they keep fp16's 2^-11 down to 2^-28 of it (e^-19.4).
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,Nq,lens", [(4, 1, [300, 17]), (4, 4, [300, 3]), (4, 1, [700] * 60), (4, 1, [2900]),
                                       (4, 8, [2900]), (4, 1, [14000, 900]), (4, 8, [14000])])
def test_8_bit_weights_far_below_a_dominant_key(H, Nq, lens, d):
    page = 16
    s = build(lens, H, 1, Nq, d, page, True, seed=50 + d, poison=False)
    k = s["kc"].view(torch.uint8)
    k.zero_()
    s["k_scale"].fill_(2.0 ** -8)
    s["v_scale"].fill_(2.0 ** -8)
    for b in range(len(lens)):
        at = (int(s["table"][b, 0]), 0, 0)
        k[at] = torch.full((d,), 256.0).to(torch.float8_e4m3fn).view(torch.uint8)   # key 0: ones
        s["vc"].view(torch.uint8)[at] = 0
    # its score: 0, 12, 17 and 19 above the others', by head (some rows of a warp each)
    for h, gap in enumerate((0.0, 12.0, 17.0, 19.0)):
        s["q"][:, h] = gap / math.sqrt(d)
    o, _ = check(s)
    assert float(o[0, 3].abs().max()) > 0


def test_8_bit_scales_as_far_apart_as_they_come():
    """A page of zero values (scale 2^-100) that holds the dominant key, the others at 2^60: the factor
    between the two references passes fp32, and weights of zero stay zero."""
    for length in (40, 14000):
        s = build([length], 2, 1, 1, 64, 16, True, seed=51, poison=False)
        k, v = (s[n].view(torch.uint8) for n in ("kc", "vc"))
        k.zero_()
        page = int(s["table"][0, 0])
        v[page] = 0
        k[page, 0, 0] = torch.full((64,), 256.0).to(torch.float8_e4m3fn).view(torch.uint8)
        s["k_scale"].fill_(2.0 ** -8)
        s["v_scale"].fill_(2.0 ** 60)
        s["v_scale"][page] = 2.0 ** -100
        s["q"].fill_(200.0 / 8 * math.log(2.0))      # the others lie 2^-200 below
        o, lse = run(s)
        # (17.25 in bf16: 2^-199.1) |O| <= 2^-199 * length * 448 * 2^60
        assert bool((o.double().abs() <= 2.0 ** -115).all()) and bool(torch.isfinite(lse).all())
    # one scale for all, at the ends of their range
    for e in (-110, -100, 100, 125):
        s = build([300], 2, 1, 1, 64, 16, True, seed=53, poison=False)
        s["k_scale"].fill_(2.0 ** -8)
        s["v_scale"].fill_(2.0 ** e)
        s["vc"] = (torch.rand(s["vc"].shape, generator=torch.Generator().manual_seed(54)) < 0.5).float().to(torch.float8_e4m3fn)
        o, _ = run(s)
        s["v_scale"].fill_(1.0)
        check(s, got=((o.double() * 2.0 ** -e).to(torch.float32), run(s)[1]))


def test_a_bad_page_does_not_hide_a_timeout():
    s = build([100], 2, 1, 1, 64, 16, False, seed=52)
    s["table"][0, 2] = -1
    run(s)
    st = torch.cuda.current_stream().cuda_stream
    assert _lib.fa_watchdog_selftest(50_000_000, st) == _lib.FA_OK
    run(s)
    assert api.last_device_error() == _lib.FA_ERR_TIMEOUT
    assert api.last_device_error() == _lib.FA_ERR_PAGE
    assert api.last_device_error() == _lib.FA_OK
