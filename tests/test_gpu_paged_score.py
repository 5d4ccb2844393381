"""GPU parity of decoding from a paged cache with capped or biased scores (fa_fwd_paged_score) against the
plain 64-bit form, and a run of prompt, append and decode steps with one learned bias."""
import math

import pytest
import torch

from exact_io_aware_12_gb300 import api, _lib
from tests import _plain, _plain_score
from tests._plain_score import BF16_HALF, FP16_HALF, FP32_HALF, Exact, within
from tests.test_gpu_score import dev, slopes_of, table_of

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


def pool(lens, Hkv, page, d, seed, fp8):
    g = torch.Generator().manual_seed(seed)
    total, table = _plain.make_pages(lens, page, g)
    k, v = (torch.randn(total, Hkv, page, d, generator=g) for _ in range(2))
    c = {"table": table, "lens": torch.tensor(lens, dtype=torch.int32), "gen": g}
    for n, x in (("k", k), ("v", v)):
        if fp8:
            scale = 2.0 ** torch.ceil(torch.log2(x.abs().amax(dim=(2, 3)) / 448))
            c[n], c[n + "_scale"] = (x / scale[..., None, None]).to(torch.float8_e4m3fn), scale
        else:
            c[n] = x.to(BF)
    return c


def exact(c, q, tau, window=0, sinks=0, softcap=None, slopes=None, bias=None, buckets=None):
    """(O, LSE) in 64 bits and their bounds: as in _plain_score, P as bf16, or as fp16 of an 8-bit cache."""
    B, H, Nq, d = q.shape
    o = torch.zeros(B, H, Nq, d, dtype=torch.float64)
    lse = torch.full((B, H, Nq), -math.inf, dtype=torch.float64)
    b_o, b_l = torch.full_like(o, 1e-9), torch.full_like(lse, 1e-9)
    for b, n in enumerate(c["lens"].tolist()):
        if n == 0:
            continue
        k, v = (_plain.gather(c[x], c["table"][b], n, c.get(x + "_scale")) for x in "kv")
        G = H // k.shape[0]
        k, v, qq = k.repeat_interleave(G, 0), v.repeat_interleave(G, 0), q[b].double()
        see = _plain.visible(Nq, n, window, sinks) & (torch.arange(n - Nq, n) >= 0)[:, None]
        x = qq @ k.mT * tau
        size = (qq.abs() @ k.abs().mT * tau).amax() * FP32_HALF * (d + 8)
        if softcap:
            x = softcap * torch.tanh(x / softcap)
            size = size + softcap * 8 * FP32_HALF
        dist = torch.arange(n - Nq, n)[:, None] - torch.arange(n)[None, :]
        if slopes is not None:
            x = x - slopes.double()[:, None, None] * dist.abs()
        if bias is not None:
            far = buckets.numel() // 2
            e = buckets.long()[dist.clamp(-far, far) + far]
            x = x + torch.where(((e >= 0) & (e < bias.shape[0]))[..., None], bias.double()[e.clamp(0, bias.shape[0] - 1)],
                                0.0).permute(2, 0, 1)
        size = float(size + 8 * FP32_HALF * x.abs().masked_fill(~see, 0).amax())
        x = x.masked_fill(~see, -math.inf)
        lse[b] = torch.logsumexp(x, -1)
        p = torch.where(see, torch.exp(x - lse[b].clamp(min=-1e300)[..., None]), 0.0)
        o[b] = p @ v
        rel = 2 * size + 2.0 ** -19
        half = FP16_HALF if "k_scale" in c else BF16_HALF
        tiny = 2.0 ** -36 * n * v.abs().amax() if "k_scale" in c else 0.0
        b_o[b] = (2 * half + rel) * (p @ v.abs()) + BF16_HALF * o[b].abs() + tiny + 1e-9
        b_l[b] = size + 2.0 ** -16 + 2 * FP32_HALF * lse[b].clamp(min=-1e30).abs()
    return o, lse, b_o, b_l


def run(c, q, **kw):
    kw = dev(kw)
    a = dev({n: t for n, t in c.items() if n != "gen"})
    window = kw.pop("window", 0) or None
    out = api.fwd_paged(q.to(DEV), a["k"], a["v"], a["table"], a["lens"], k_scale=a.get("k_scale"), v_scale=a.get("v_scale"),
                        window=window, **kw)
    torch.cuda.synchronize()
    assert api.last_device_error() == _lib.FA_OK
    return out


def check(lens, H, Hkv, Nq, d, page, fp8, seed=1, scale=1.0, **kw):
    c = pool(lens, Hkv, page, d, seed, fp8)
    q = (torch.randn(len(lens), H, Nq, d, generator=c["gen"]) * scale).to(BF)
    tau = 1 / math.sqrt(d)
    o, lse = run(c, q, **kw)
    eo, el, bo, bl = exact(c, q, tau, **kw)
    within(o, eo, bo, "O")
    within(lse, el, bl, "LSE")


MODS = {"cap": lambda H: dict(softcap=20.0), "low-cap": lambda H: dict(softcap=1.5), "slopes": lambda H: dict(slopes=slopes_of(H)),
        "table": lambda H: table_of(H, 32, 128, False, 4), "fp32-table": lambda H: table_of(H, 16, 40, True, 4, torch.float32),
        "cap-slopes": lambda H: dict(softcap=3.0, slopes=slopes_of(H)),
        "cap-table": lambda H: dict(softcap=3.0, **table_of(H, 4, 1000, False, 4))}


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("mod", list(MODS))
@pytest.mark.parametrize("lens,H,Hkv,Nq,d,page", [
    ([1], 2, 2, 1, 64, 16), ([0, 1, 15, 16, 17, 3], 4, 2, 1, 128, 16), ([130, 517, 33], 12, 12, 1, 64, 16),
    ([700, 40], 8, 2, 4, 128, 32), ([300, 5, 900], 16, 1, 8, 64, 64), ([6, 2, 40], 4, 4, 8, 128, 16)])
def test_short_tables(lens, H, Hkv, Nq, d, page, mod, fp8):
    check(lens, H, Hkv, Nq, d, page, fp8, scale=2.0, **MODS[mod](H))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("mod", list(MODS))
@pytest.mark.parametrize("lens,H,Hkv,Nq,d,page", [
    ([9000, 20, 3001], 4, 1, 1, 128, 64), ([5000] + [700 + 131 * i for i in range(40)], 8, 4, 2, 64, 128),
    ([2500, 2500, 1700], 32, 2, 4, 128, 64)])
def test_long_tables(lens, H, Hkv, Nq, d, page, mod, fp8):
    check(lens, H, Hkv, Nq, d, page, fp8, **MODS[mod](H))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("mod", list(MODS))
def test_windows_and_sinks(mod, fp8):
    check([3000, 100, 700], 8, 2, 3, 128, 32, fp8, window=250, sinks=37, **MODS[mod](8))
    check([3000, 100, 700], 4, 4, 1, 64, 16, fp8, window=1, **MODS[mod](4))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("cap", [2.0 ** 14, 2.0 ** 20, 2.0 ** 60])
def test_large_caps_leave_scores_as_they_are(cap, fp8):
    """x / cap below 2^-11: cap tanh(x / cap) is x within 2^-23 of it, as one fp32 rounding, of which the bounds
    without a cap give q.k's own sum d."""
    for lens, H, Hkv, Nq, d, page in (([130, 517, 33], 12, 12, 1, 64, 16), ([2500, 2500, 1700], 32, 2, 4, 128, 64)):
        c = pool(lens, Hkv, page, d, 5, fp8)
        q = torch.randn(len(lens), H, Nq, d, generator=c["gen"]).to(BF)
        a = dev({n: t for n, t in c.items() if n != "gen"})
        scales = {n: a[n] for n in ("k_scale", "v_scale") if n in a}
        o, lse = api.fwd_paged(q.to(DEV), a["k"], a["v"], a["table"], a["lens"], softcap=cap, **scales)
        eo, el, bo, bl = exact(c, q, d ** -0.5)
        within(o, eo, bo, "O")
        within(lse, el, bl, "LSE")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_slopes_of_positions_beyond_2_24(d, fp8):
    """16778217 keys of 64 pages that take turns: positions that fp32 does not hold, distances that it does.  Keys
    more than 8000 away weigh less than e^-380 of the rest (scores are below 10), so that the last 64 pages alone give
    the same."""
    page, pages, L = 128, 64, 2 ** 24 + 1001
    c = pool([page * pages], 2, page, d, 3, fp8)
    q = torch.randn(1, 4, 3, d, generator=c["gen"]).to(BF)
    slopes = torch.tensor([1.0, 0.7, 0.25, 0.05])
    c["table"] = (torch.arange(-(-L // page)) % pages).to(torch.int32)[None]
    c["lens"] = torch.tensor([L], dtype=torch.int32)
    o, lse = run(c, q, slopes=slopes)
    c["table"] = c["table"][:, -pages:].contiguous()
    c["lens"] = torch.tensor([(pages - 1) * page + L % page], dtype=torch.int32)
    eo, el, bo, bl = exact(c, q, d ** -0.5, slopes=slopes)
    within(o, eo, bo, "O")
    within(lse, el, bl, "LSE")


def test_all_fields_unset_is_the_plain_step():
    c = pool([100, 900], 2, 16, 64, 3, False)
    q = torch.randn(2, 4, 1, 64, generator=c["gen"]).to(BF).to(DEV)
    a = dev({n: t for n, t in c.items() if n != "gen"})
    o, lse = torch.empty_like(q), torch.empty(2, 4, 1, device=DEV)
    cache = _lib.PagedCache(a["k"].data_ptr(), a["v"].data_ptr(), None, None, a["table"].data_ptr(), a["lens"].data_ptr(), 2, 2,
                            64, a["k"].shape[0], 16, a["table"].shape[1])
    _lib.check(_lib.fa_fwd_paged_score(cache, q.data_ptr(), 256, 64, 64, o.data_ptr(), 256, 64, 64, lse.data_ptr(), 4, 1, 0.125, 0,
                                       0, _lib.Score(), None, 0, torch.cuda.current_stream().cuda_stream), "paged")
    eo, el, bo, bl = exact(c, q.cpu(), 0.125)
    within(o, eo, bo, "O")
    within(lse, el, bl, "LSE")


def test_bad_pages_are_hidden_and_reported():
    """A page number out of bounds hides its keys (FA_ERR_PAGE), with a bias as without."""
    c = pool([100], 2, 16, 64, 3, False)
    q = torch.randn(1, 4, 1, 64, generator=c["gen"]).to(BF)
    c["table"][0, 2] = 10 ** 6
    a = dev({n: t for n, t in c.items() if n != "gen"})
    kw = table_of(4, 32, 128, False, 4)
    o, lse = api.fwd_paged(q.to(DEV), a["k"], a["v"], a["table"], a["lens"], **dev(kw))
    torch.cuda.synchronize()
    assert api.last_device_error() == _lib.FA_ERR_PAGE
    keep = [j for j in range(100) if j // 16 != 2]
    full = _plain.gather(c["k"], torch.where(c["table"][0] > 99, 0, c["table"][0]), 100)
    vals = _plain.gather(c["v"], torch.where(c["table"][0] > 99, 0, c["table"][0]), 100)
    far = kw["buckets"].numel() // 2
    dist = 99 - torch.tensor(keep)
    add = kw["bias"].double()[kw["buckets"].long()[dist.clamp(max=far) + far]].T
    x = torch.einsum("hd,hkd->hk", q[0, :, 0].double(), full[:, keep].repeat_interleave(2, 0)) * 0.125 + add
    want = torch.einsum("hk,hkd->hd", torch.softmax(x, -1), vals[:, keep].repeat_interleave(2, 0))
    # three roundings of 2^-8 at most, of weights that sum to one and values below 5
    assert float((o[0, :, 0].cpu().double() - want).abs().max()) <= 3 * BF16_HALF * 5
    assert float((lse[0, :, 0].cpu().double() - torch.logsumexp(x, -1)).abs().max()) <= 2.0 ** -15


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("mod", ["cap-table", "cap-slopes"])
def test_prompt_append_and_decode_are_one_attention(mod, d):
    """A prompt through the forward, its keys into the cache, then steps of one and of three tokens, the last
    of them captured in a graph: row by row what the forward gives over the whole sequence."""
    B, H, Hkv, page, P, N = 2, 4, 2, 16, 150, 158
    g = torch.Generator().manual_seed(9)
    q, k, v = (torch.randn(B, h, N, d, generator=g).to(BF) for h in (H, Hkv, Hkv))
    kw = MODS[mod](H)
    e = Exact(q, k, v, True, 1 / math.sqrt(d), **kw)
    on = dev(kw)
    qd, kd, vd = q.to(DEV), k.to(DEV), v.to(DEV)
    o, lse = api.fwd(qd[:, :, :P].contiguous(), kd[:, :, :P].contiguous(), vd[:, :, :P].contiguous(), True, **on)
    within(o, e.o[:, :, :P], e.b_o[:, :, :P], "prompt")
    pages = -(-N // page)
    table = torch.randperm(B * pages, generator=g).to(torch.int32).view(B, pages).to(DEV)
    kc, vc = (torch.zeros(B * pages, Hkv, page, d, dtype=BF, device=DEV) for _ in range(2))
    lens = torch.zeros(B, dtype=torch.int32, device=DEV)

    def append(a, z):
        flat = lambda t: t[:, :, a:z].transpose(1, 2).reshape(B * (z - a), Hkv, d).contiguous()
        api.kv_append(flat(kd), flat(vd), kc, vc, table, lens)
        lens.add_(z - a)
    append(0, P)
    for a, z in ((P, P + 1), (P + 1, P + 2), (P + 2, P + 5)):
        append(a, z)
        so, sl = api.fwd_paged(qd[:, :, a:z], kc, vc, table, lens, **on)
        within(so, e.o[:, :, a:z], e.b_o[:, :, a:z], "step")
        within(sl, e.lse[:, :, a:z], e.b_lse[:, :, a:z], "step LSE")
    step = [t[:, :, :3].contiguous() for t in (qd, kd, vd)]

    def captured():
        flat = lambda t: t.transpose(1, 2).reshape(B * 3, Hkv, d).contiguous()
        api.kv_append(flat(step[1]), flat(step[2]), kc, vc, table, lens)
        lens.add_(3)
        return api.fwd_paged(step[0], kc, vc, table, lens, **on)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        so, sl = captured()
    for t, full in zip(step, (qd, kd, vd)):
        t.copy_(full[:, :, P + 5:N])
    graph.replay()
    torch.cuda.synchronize()
    within(so, e.o[:, :, P + 5:N], e.b_o[:, :, P + 5:N], "captured step")
    assert api.last_device_error() == _lib.FA_OK
