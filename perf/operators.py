"""Windowed attention with sinks, and serving from a paged key/value cache: the cases
that are timed, their plain forms and their exact values.

Five operators, in the order in which a model meets them:

  sinks     causal sliding-window attention in which the first few tokens stay visible,
            forward and backward (api.fwd / api.bwd with window= and sinks=)
  append    new keys and values into a bf16 paged cache, keys (and queries) rotated by
            their position on the way (api.kv_append)
  append8   the same into an e4m3 paged cache with one scale per page and head
  paged     attention of a step's new queries over the bf16 paged cache (api.fwd_paged)
  paged8    the same over the e4m3 paged cache

With ``own`` false, ``run`` computes each in elementary torch operations in 32 bits
(angles in 64), rounded once at the end; with ``own`` true it makes the framework's calls.
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0
SCALE_EXP_MIN, SCALE_EXP_MAX = -100, 121


def listed():
    return [
        # a long-context training step: 16 heads, 16384 tokens, the 4096-token window and four sink tokens
        {"name": "sinks_train_16k", "op": "sinks", "B": 1, "H": 16, "N": 16384, "d": 128, "window": 4096, "sinks": 4,
         "backward": True},
        # a short training batch with a narrow window, head size 64
        {"name": "sinks_train_1k", "op": "sinks", "B": 8, "H": 12, "N": 1024, "d": 64, "window": 256, "sinks": 16,
         "backward": True},
        # a prompt of odd length, forward alone, sinks longer than one key block
        {"name": "sinks_prompt_5001", "op": "sinks", "B": 2, "H": 8, "N": 5001, "d": 128, "window": 1000, "sinks": 130,
         "backward": False},
        # prompts of uneven length entering the cache together, queries rotated in the same call
        {"name": "append_prompts", "op": "append", "B": 6, "H": 32, "Hkv": 8, "d": 128, "rot": 128, "interleaved": False,
         "page": 64, "new": 8192, "even": False, "past": 0, "mix": 1},
        # one decode step of 64 sequences of uneven length
        {"name": "append_step", "op": "append", "B": 64, "H": 32, "Hkv": 8, "d": 128, "rot": 128, "interleaved": False,
         "page": 64, "new": 1, "even": True, "past": 8191, "mix": 2},
        # chunks of prompts continuing in half-filled 8-bit pages, half of each head rotated
        {"name": "append8_prompts", "op": "append8", "B": 6, "H": 32, "Hkv": 8, "d": 128, "rot": 64, "interleaved": False,
         "page": 64, "new": 8192, "even": False, "past": 4095, "mix": 3},
        # one decode step into 8-bit pages
        {"name": "append8_step", "op": "append8", "B": 64, "H": 32, "Hkv": 8, "d": 128, "rot": 128, "interleaved": True,
         "page": 32, "new": 1, "even": True, "past": 8191, "mix": 4},
        # the smallest decode step: one sequence of a few hundred tokens, 12 heads of 64, no head sharing
        {"name": "paged_one_short", "op": "paged", "B": 1, "H": 12, "Hkv": 12, "Nq": 1, "d": 64, "page": 16, "max": 517,
         "window": 0, "sinks": 0, "mix": 5},
        # a serving batch of uneven lengths, four query heads to a key head
        {"name": "paged_batch", "op": "paged", "B": 48, "H": 32, "Hkv": 8, "Nq": 1, "d": 128, "page": 64, "max": 16384,
         "window": 0, "sinks": 0, "mix": 6},
        # four draft tokens a sequence over very long caches, windowed with sinks
        {"name": "paged_draft_window", "op": "paged", "B": 16, "H": 32, "Hkv": 8, "Nq": 4, "d": 128, "page": 64,
         "max": 65536, "window": 4096, "sinks": 4, "mix": 7},
        # eight long sequences in 8 bits, 16 heads without sharing, 32768 tokens at most
        {"name": "paged8_long", "op": "paged8", "B": 8, "H": 16, "Hkv": 16, "Nq": 1, "d": 128, "page": 64, "max": 32768,
         "window": 0, "sinks": 0, "mix": 8},
        # a wide serving batch in 8 bits, eight query heads to a key head
        {"name": "paged8_batch", "op": "paged8", "B": 96, "H": 64, "Hkv": 8, "Nq": 1, "d": 128, "page": 64, "max": 12000,
         "window": 0, "sinks": 0, "mix": 9},
    ]


def _spread(rng, low, high):
    """A whole number between low and high, even over its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 1)))))))


def draw(rng):
    op = rng.choice(["sinks", "append", "append8", "paged", "paged8"])
    d = rng.choice([64, 128])
    if op == "sinks":
        B, H = rng.choice([(1, 1), (1, 16), (2, 8), (1, 5), (4, 12)])
        N = _spread(rng, 200, 12000 if B * H <= 16 else 4096)
        return {"op": op, "B": B, "H": H, "N": N, "d": d, "window": _spread(rng, 100, 4096), "sinks": rng.randint(1, 200),
                "backward": rng.random() < 0.6}
    page = rng.choice([16, 32, 64, 128])
    Hkv = rng.choice([1, 2, 4, 8, 16])
    G = rng.choice([1, 2, 3, 4, 8]) if Hkv <= 8 else 1
    if op in ("append", "append8"):
        step = rng.random() < 0.5
        B = _spread(rng, 1, 96) if step else rng.randint(1, 6)
        return {"op": op, "B": B, "H": Hkv * G if rng.random() < 0.7 else 0, "Hkv": Hkv, "d": d,
                "rot": rng.choice([d, d, d // 2]), "interleaved": rng.random() < 0.3, "page": page,
                "new": rng.randint(1, 4) if step else _spread(rng, 10, 8192), "even": step,
                "past": rng.choice([0, _spread(rng, 1, 16384)]), "mix": rng.randint(0, 10 ** 6)}
    B = _spread(rng, 1, 64)
    most = 2_000_000 // (B * Hkv) * (2 if op == "paged8" else 1)
    windowed = rng.random() < 0.3
    return {"op": op, "B": B, "H": Hkv * G, "Hkv": Hkv, "Nq": rng.choice([1, 1, 2, 4, 8]), "d": d, "page": page,
            "max": _spread(rng, 9, max(40, min(65536, most))), "window": _spread(rng, 64, 4096) if windowed else 0,
            "sinks": rng.randint(1, 70) if windowed else 0, "mix": rng.randint(0, 10 ** 6)}


# ---------------------------------------------------------------- inputs ----
def _lengths(case):
    """(keys in the cache before the call, new tokens) of each sequence of a paged case."""
    r = random.Random(case["mix"])
    B = case["B"]
    if case["op"] in ("append", "append8"):
        past = [case["past"]] + [r.randint(0, case["past"]) for _ in range(B - 1)]
        new = [case["new"]] + [case["new"] if case["even"] else r.randint(0, case["new"] // 2) for _ in range(B - 1)]
        return past, new
    return [case["max"]] + [r.randint(max(case["Nq"], case["max"] // 8), max(case["Nq"], case["max"]))
                            for _ in range(B - 1)], [0] * B


def _pool(case, g):
    """A paged cache: pages in random order, table entries behind a sequence's pages -1."""
    past, new = _lengths(case)
    page, B, Hkv, d = case["page"], case["B"], case["Hkv"], case["d"]
    pages = [-(-(p + n) // page) for p, n in zip(past, new)]
    total = sum(pages) + 3
    order = torch.randperm(total, generator=g, device="cuda")
    table = torch.full((B, max(1, max(pages))), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = order[at:at + n].to(torch.int32)
        at += n
    gain = torch.exp(0.4 * torch.randn(Hkv, 1, d, generator=g, device="cuda"))  # channels of uneven size
    s = {"table": table, "lens": torch.tensor(past, dtype=torch.int32, device="cuda"), "new": new}
    for name in ("k", "v"):
        x = torch.randn(total, Hkv, page, d, generator=g, device="cuda").mul_(gain if name == "k" else 1.0)
        if case["op"] in ("append", "paged"):
            s[name] = x.to(torch.bfloat16)
            continue
        scale = _scale_for(x.abs().amax(dim=(2, 3)))
        s[name] = (x / scale[:, :, None, None]).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        s[name + "_scale"] = scale
        del x
    return s, gain


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    bf = torch.bfloat16
    if case["op"] == "sinks":
        shape = (case["B"], case["H"], case["N"], case["d"])
        s = {n: torch.randn(shape, generator=g, device="cuda").to(bf) for n in ("q", "k", "v", "do")}
        s["ws"] = torch.empty(math.prod(shape) * 4 + math.prod(shape[:3]) * 4 + 512, dtype=torch.uint8, device="cuda")
        return {**s, "case": case}
    s, gain = _pool(case, g)
    s["case"] = case
    H, Hkv, d = case["H"], case["Hkv"], case["d"]
    if case["op"] in ("paged", "paged8"):
        s["q"] = torch.randn(case["B"], H, case["Nq"], d, generator=g, device="cuda").to(bf)
    else:
        T = sum(s["new"])
        # one projection's output holds a token's queries, keys and values side by side
        x = torch.randn(T, H + 2 * Hkv, d, generator=g, device="cuda")
        x[:, H:H + Hkv] *= gain[:, 0]
        x = x.to(bf)
        s["q_new"], s["k_new"], s["v_new"] = (x[:, :H] if H else None), x[:, H:H + Hkv], x[:, H + Hkv:]
        cu = [0]
        for n in s["new"]:
            cu.append(cu[-1] + n)
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
        i = torch.arange(case["rot"] // 2, dtype=torch.float64, device="cuda")
        s["inv_freq"] = 10000.0 ** (-2.0 * i / case["rot"])
    return s


# ----------------------------------------------------------- plain forms ----
def _visible(N, window, sinks):
    """[N, N]: query i sees key j when j <= i and j is in the window or a sink."""
    i, j = torch.arange(N, device="cuda")[:, None], torch.arange(N, device="cuda")[None, :]
    return (j <= i) & ((j > i - window) | (j < sinks))


def _plain_sinks(s):
    c = s["case"]
    q, k, v = (s[n].float() for n in ("q", "k", "v"))
    tau = 1.0 / math.sqrt(c["d"])
    x = (q @ k.mT).mul_(tau).masked_fill_(~_visible(c["N"], c["window"], c["sinks"]), -math.inf)
    m = x.amax(dim=-1, keepdim=True)
    p = x.sub_(m).exp_()
    total = p.sum(dim=-1, keepdim=True)
    p.div_(total)
    o, lse = p @ v, (m + total.log()).squeeze(-1)
    if not c["backward"]:
        return [o.bfloat16(), lse]
    do = s["do"].float()
    dv = p.mT @ do
    ds = (do @ v.mT).sub_((do * o).sum(dim=-1, keepdim=True)).mul_(p).mul_(tau)
    return [o.bfloat16(), lse, (ds @ k).bfloat16(), (ds.mT @ q).bfloat16(), dv.bfloat16()]


def _scale_for(bound):
    """The smallest power of two s with bound <= 448 s."""
    f, e = torch.frexp(bound)
    e = torch.where(bound > 0, e - 9 + (f > 0.875), SCALE_EXP_MIN).clamp(SCALE_EXP_MIN, SCALE_EXP_MAX)
    return torch.ldexp(torch.ones_like(bound), e)


def _rotate(x, angle, rot, interleaved):
    """x [T, H, d] in 32 bits, angle [T, rot / 2] in 64: pairs of the first rot columns turned by their angle."""
    if x.shape[-2] == 0:
        return x
    c, sn = angle.cos().float()[:, None], angle.sin().float()[:, None]
    r, rest = x[..., :rot], x[..., rot:]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :rot // 2], r[..., rot // 2:])
    a, b = a * c - b * sn, b * c + a * sn
    r = torch.stack((a, b), dim=-1).flatten(-2) if interleaved else torch.cat((a, b), dim=-1)
    return torch.cat((r, rest), dim=-1)


def _places(s):
    """For each new token its position, page and offset in the page."""
    T, page = s["k_new"].shape[0], s["case"]["page"]
    t = torch.arange(T, device="cuda", dtype=torch.int32)
    b = torch.searchsorted(s["cu"], t, right=True) - 1
    pos = (s["lens"][b] + t - s["cu"][b]).long()
    return pos, s["table"][b, pos // page].long(), pos % page


def _into_pages8(codes, scale, new, bound, pid, off, s):
    """new [T, Hkv, d] in 32 bits into e4m3 pages; bound [T, Hkv] sets the pages' scales."""
    page, lens = s["case"]["page"], s["lens"].long()
    need = torch.zeros_like(scale).index_reduce_(0, pid, bound, "amax")
    need = _scale_for(need)
    first = s["table"].gather(1, (lens // page).clamp(max=s["table"].shape[1] - 1)[:, None])[:, 0].long()
    held = (lens % page > 0) & (s["cu"][1:] > s["cu"][:-1])  # sequences that go on in a page begun earlier
    first = torch.where(held, first, first.clamp(min=0))
    old = scale[first]
    grown = torch.where(held[:, None], torch.maximum(old, need[first]), old)
    stays = held[:, None, None, None] & (torch.arange(page, device="cuda") < (lens % page)[:, None])[:, None, :, None]
    kept = codes[first].float()
    again = (kept * (old / grown)[:, :, None, None]).to(torch.float8_e4m3fn)
    keep = torch.where(stays, again.view(torch.uint8), codes[first].view(torch.uint8))
    # a sequence without a page begun earlier writes its rows back as they were: to a page of its own, or to none
    row = torch.where(held, first, codes.shape[0])
    wide = torch.cat((codes.view(torch.uint8), codes[:1].view(torch.uint8)))
    wide[row] = keep
    codes.view(torch.uint8).copy_(wide[:-1])
    scale_new = scale.index_copy(0, pid, need[pid])
    scale_new = torch.cat((scale_new, scale_new[:1])).index_copy(0, row, grown)[:-1]
    scale.copy_(scale_new)
    codes.view(torch.uint8)[pid, :, off] = (new / scale[pid][:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(
        torch.float8_e4m3fn).view(torch.uint8)


def _plain_append(s):
    c = s["case"]
    pos, pid, off = _places(s)
    angle = pos[:, None].double() * s["inv_freq"]
    k, v = _rotate(s["k_new"].float(), angle, c["rot"], c["interleaved"]), s["v_new"].float()
    q = None if s["q_new"] is None else _rotate(s["q_new"].float(), angle, c["rot"], c["interleaved"]).bfloat16()
    if c["op"] == "append":
        s["k"][pid, :, off], s["v"][pid, :, off] = k.bfloat16(), v.bfloat16()
        return [q, s["k"], s["v"]]
    # a turned pair is at most sqrt(2) times its larger half: the page's scale goes by 1.5 times the keys as they come
    _into_pages8(s["k"], s["k_scale"], k, s["k_new"].float().abs().amax(-1) * 1.5, pid, off, s)
    _into_pages8(s["v"], s["v_scale"], v, s["v_new"].float().abs().amax(-1), pid, off, s)
    return [q, s["k"], s["v"], s["k_scale"], s["v_scale"]]


def _plain_paged(s):
    c = s["case"]
    B, H, Hkv, Nq, d, page = (c[n] for n in ("B", "H", "Hkv", "Nq", "d", "page"))
    at = s["table"].long().clamp(min=0)
    k, v = s["k"][at].float(), s["v"][at].float()  # [B, pages, Hkv, page, d]
    if c["op"] == "paged8":
        k.mul_(s["k_scale"][at][..., None, None])
        v.mul_(s["v_scale"][at][..., None, None])
    k, v = (x.transpose(1, 2).reshape(B, Hkv, -1, d) for x in (k, v))
    q = s["q"].float().reshape(B, Hkv, H // Hkv * Nq, d)
    x = (q @ k.mT).mul_(1.0 / math.sqrt(d)).reshape(B, H, Nq, -1)
    j = torch.arange(x.shape[-1], device="cuda")
    last = (s["lens"].long()[:, None] - Nq + torch.arange(Nq, device="cuda"))[:, None, :, None]  # row i's own position
    seen = j <= last
    if c["window"]:
        seen = seen & ((j > last - c["window"]) | (j < c["sinks"]))
    x.masked_fill_(~seen, -math.inf)
    m = x.amax(dim=-1, keepdim=True).clamp(min=-3e38)  # a row that sees nothing: O = 0, LSE = -inf
    p = x.sub_(m).exp_()
    total = p.sum(dim=-1, keepdim=True)
    o = (p.reshape(B, Hkv, -1, p.shape[-1]) @ v).reshape(B, H, Nq, d) / total.clamp(min=1e-38)
    return [o.bfloat16(), (m + total.log()).squeeze(-1)]


def _run_own(s):
    from exact_io_aware_12_gb300 import api
    c = s["case"]
    if c["op"] == "sinks":
        o, lse = api.fwd(s["q"], s["k"], s["v"], True, window=c["window"], sinks=c["sinks"])
        if not c["backward"]:
            return [o, lse]
        return [o, lse, *api.bwd(s["q"], s["k"], s["v"], o, s["do"], lse, True, workspace=s["ws"], window=c["window"],
                                 sinks=c["sinks"])]
    if c["op"] in ("append", "append8"):
        q = api.kv_append(s["k_new"], s["v_new"], s["k"], s["v"], s["table"], s["lens"], cu_new=s["cu"], q=s["q_new"],
                          inv_freq=s["inv_freq"], interleaved=c["interleaved"], k_scale=s.get("k_scale"),
                          v_scale=s.get("v_scale"))
        return [q, s["k"], s["v"]] + ([s["k_scale"], s["v_scale"]] if c["op"] == "append8" else [])
    return list(api.fwd_paged(s["q"], s["k"], s["v"], s["table"], s["lens"], window=c["window"] or None,
                              sinks=c["sinks"], k_scale=s.get("k_scale"), v_scale=s.get("v_scale")))


def run(state):
    if own:
        return [x for x in _run_own(state) if x is not None]
    form = {"sinks": _plain_sinks, "append": _plain_append, "append8": _plain_append, "paged": _plain_paged,
            "paged8": _plain_paged}[state["case"]["op"]]
    return [x for x in form(state) if x is not None]


# ------------------------------------------------------------------ work ----
def _pairs(n, window, sinks, rows):
    """Visible (query, key) pairs of the last `rows` positions of n, and the distinct keys they see."""
    w = window or n
    pairs = 0
    for i in range(max(0, n - rows), n):
        low = max(0, i - w + 1)
        pairs += i + 1 - low + min(sinks, low)
    low = max(0, n - rows - w + 1)
    return pairs, n - low + min(sinks, low)


def work(case):
    c, d = case, case["d"]
    if c["op"] == "sinks":
        heads, rows = c["B"] * c["H"], c["B"] * c["H"] * c["N"]
        pairs = heads * _pairs(c["N"], c["window"], c["sinks"], c["N"])[0]
        tensors = 8 if c["backward"] else 4  # Q K V O, and dO dQ dK dV
        return {"bytes": rows * (tensors * d * 2 + 4), "flops": pairs * d * (14 if c["backward"] else 4)}
    past, new = _lengths(case)
    if c["op"] in ("append", "append8"):
        T, e = sum(new), 1 if c["op"] == "append8" else 2
        moved = T * d * (2 * c["Hkv"] * (2 + e) + c["H"] * 4) + c["B"] * 12
        if e == 1:  # scales of the pages reached, read and written
            moved += sum(-(-(p + n) // c["page"]) - p // c["page"] for p, n in zip(past, new) if n) * c["Hkv"] * 16
        return {"bytes": moved, "flops": T * (c["Hkv"] + c["H"]) * c["rot"] * 3}
    seen = [_pairs(n, c["window"], c["sinks"], c["Nq"]) for n in past]
    keys, pairs = sum(k for _, k in seen), sum(p for p, _ in seen)
    e = 1 if c["op"] == "paged8" else 2
    moved = keys * c["Hkv"] * d * 2 * e + keys // c["page"] * (4 + (8 * c["Hkv"] if e == 1 else 0))
    return {"bytes": moved + c["B"] * c["H"] * c["Nq"] * (d * 4 + 4), "flops": 4 * d * pairs * c["H"]}


# ----------------------------------------------------------------- exact ----
def _exact_sinks(s):
    """Row chunks against the keys that they see, head by head."""
    c = s["case"]
    N, w, S, tau = c["N"], c["window"], c["sinks"], 1.0 / math.sqrt(c["d"])
    q, k, v, do = (s[n].double().reshape(-1, N, c["d"]) for n in ("q", "k", "v", "do"))
    o, dq, dk, dv = (torch.zeros_like(q) for _ in range(4))
    lse = torch.empty(q.shape[:2], dtype=torch.float64, device="cuda")
    for h in range(q.shape[0]):
        for r0 in range(0, N, 2048):
            r1 = min(N, r0 + 2048)
            lo = max(0, r0 - w + 1)
            keys = torch.cat((torch.arange(0, min(S, lo), device="cuda"), torch.arange(lo, r1, device="cuda")))
            rows = torch.arange(r0, r1, device="cuda")[:, None]
            hidden = (keys > rows) | ((rows - keys >= w) & (keys >= S))
            x = torch.einsum("rd,kd->rk", q[h, r0:r1], k[h, keys]) * tau
            x[hidden] = -math.inf
            lse[h, r0:r1] = torch.logsumexp(x, dim=1)
            p = torch.exp(x - lse[h, r0:r1, None])
            o[h, r0:r1] = p @ v[h, keys]
            if c["backward"]:
                g = do[h, r0:r1]
                ds = p * (g @ v[h, keys].T - (g * o[h, r0:r1]).sum(1, keepdim=True))
                dq[h, r0:r1] = tau * (ds @ k[h, keys])
                dk[h].index_add_(0, keys, tau * (ds.T @ q[h, r0:r1]))
                dv[h].index_add_(0, keys, p.T @ g)
    shape = s["q"].shape
    out = [o.view(shape), lse.view(shape[:3])]
    return out + [dq.view(shape), dk.view(shape), dv.view(shape)] if c["backward"] else out


def _turned(x, pos, inv_freq, rot, interleaved):
    """Rotation of x [n, H, d] as a product of complex numbers."""
    turn = torch.polar(torch.ones_like(pos[:, None] * inv_freq), pos[:, None] * inv_freq)[:, None]
    x = x.clone()
    r = x[..., :rot]
    z = torch.complex(r[..., 0::2], r[..., 1::2]) if interleaved else torch.complex(r[..., :rot // 2], r[..., rot // 2:])
    z = z * turn
    if interleaved:
        x[..., 0:rot:2], x[..., 1:rot:2] = z.real, z.imag
    else:
        x[..., :rot // 2], x[..., rot // 2:rot] = z.real, z.imag
    return x


def _power(bound):
    """2^e with the least e that holds bound in 448 * 2^e; bound [Hkv] on the host."""
    out = []
    for b in bound.tolist():
        e = SCALE_EXP_MIN
        if b > 0:
            e = math.ceil(math.log2(b / E4M3_MAX)) - 1
            while b > E4M3_MAX * 2.0 ** e:
                e += 1
        out.append(2.0 ** max(SCALE_EXP_MIN, min(SCALE_EXP_MAX, e)))
    return torch.tensor(out, dtype=torch.float64, device="cuda")


def _exact_append(s):
    """Sequence by sequence and page by page; new entries of 8-bit pages before their rounding."""
    c = s["case"]
    page, rot, il = c["page"], c["rot"], c["interleaved"]
    K, V = s["k"].double(), s["v"].double()
    ks, vs = (s[n].double() if n in s else None for n in ("k_scale", "v_scale"))
    q = None if s["q_new"] is None else s["q_new"].double().clone()
    table, t0 = s["table"].tolist(), 0
    past, new = _lengths(c)
    for b, (p0, n) in enumerate(zip(past, new)):
        if n == 0:
            continue
        pos = torch.arange(p0, p0 + n, device="cuda", dtype=torch.float64)
        kn, vn = s["k_new"][t0:t0 + n].double(), s["v_new"][t0:t0 + n].double()
        kr = _turned(kn, pos, s["inv_freq"], rot, il)
        if q is not None:
            q[t0:t0 + n] = _turned(q[t0:t0 + n], pos, s["inv_freq"], rot, il)
        i = 0
        while i < n:
            at, off = table[b][(p0 + i) // page], (p0 + i) % page
            m = min(page - off, n - i)
            for cache, scales, rows, size in ((K, ks, kr, 1.5 * kn.abs()), (V, vs, vn, vn.abs())):
                x = rows[i:i + m].transpose(0, 1)
                if scales is not None:
                    to = _power(size[i:i + m].amax(dim=(0, 2)))
                    if off:
                        to = torch.maximum(to, scales[at])
                        held = cache[at, :, :off] * (scales[at] / to)[:, None, None]
                        cache[at, :, :off] = held.to(torch.float8_e4m3fn).double()
                    scales[at] = to
                    x = x / to[:, None, None]
                cache[at, :, off:off + m] = x
            i += m
        t0 += n
    return [x for x in (q, K, V, ks, vs) if x is not None]


def _exact_paged(s):
    """Sequence by sequence over its own keys in order."""
    c = s["case"]
    H, Hkv, Nq, d, page = (c[n] for n in ("H", "Hkv", "Nq", "d", "page"))
    o = torch.zeros(c["B"], H, Nq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((c["B"], H, Nq), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(_lengths(c)[0]):
        ids = s["table"][b, :-(-n // page)].long()
        keys = torch.arange(n, device="cuda")
        if c["window"]:
            keys = keys[(keys > n - Nq - c["window"]) | (keys < c["sinks"])]
        pid, off = ids[keys // page], keys % page
        k, v = s["k"][pid, :, off].double(), s["v"][pid, :, off].double()  # [keys, Hkv, d]
        if c["op"] == "paged8":
            k, v = k * s["k_scale"][pid].double()[..., None], v * s["v_scale"][pid].double()[..., None]
        for i in range(Nq):
            row = n - Nq + i
            see = keys <= row
            if c["window"]:
                see &= (row - keys < c["window"]) | (keys < c["sinks"])
            if row < 0:
                continue
            x = torch.einsum("hgd,khd->hgk", s["q"][b, :, i].double().view(Hkv, -1, d), k[see]) / math.sqrt(d)
            lse[b, :, i] = torch.logsumexp(x, dim=-1).view(H)
            o[b, :, i] = torch.einsum("hgk,khd->hgd", torch.softmax(x, dim=-1), v[see]).reshape(H, d)
    return [o, lse]


def exact(case, seed):
    s = prepare(case, seed)
    form = {"sinks": _exact_sinks, "append": _exact_append, "append8": _exact_append, "paged": _exact_paged,
            "paged8": _exact_paged}[case["op"]]
    return form(s)
