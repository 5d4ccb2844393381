"""Attention whose scores are capped, biased by distance or masked by documents and prefixes,
a learned bias by buckets of distance with its gradient, and decoding with either from a
paged key/value cache: the cases that are timed, their plain forms and their exact values.

Three operators:

  score     attention with scores capped by a tanh, or with a bias that falls with distance,
            within documents, behind a visible prefix or in a window, with grouped heads;
            forward and backward (api.fwd / api.bwd with softcap=, slopes=, docs=, prefix=)
  relative  attention with a learned bias per head and bucket of distance, forward and
            backward, with the gradient of the bias (api.fwd / api.bwd with bias= and buckets=)
  paged     a decode step over a paged cache, bf16 or e4m3, with scores capped or biased the
            same ways (api.fwd_paged with softcap=, slopes=, bias= and buckets=)

With ``own`` false, ``run`` computes each in elementary torch operations in 32 bits (the
bias's gradient, a long sum, in 64), rounded once at the end; with ``own`` true it makes
the framework's calls.
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0


def _score(name, B, H, Hkv, N, d, backward, causal=True, cap=0.0, slopes=False, docs="", prefix=0, window=0, mix=0):
    return {"name": name, "op": "score", "B": B, "H": H, "Hkv": Hkv, "N": N, "d": d, "backward": backward,
            "causal": causal, "cap": cap, "slopes": slopes, "docs": docs, "prefix": prefix, "window": window,
            "buckets": 0, "far": 0, "mix": mix}


def _relative(name, B, H, N, d, backward, causal, buckets, far, docs="", cap=0.0, mix=0):
    return {"name": name, "op": "relative", "B": B, "H": H, "Hkv": H, "N": N, "d": d, "backward": backward,
            "causal": causal, "cap": cap, "slopes": False, "docs": docs, "prefix": 0, "window": 0,
            "buckets": buckets, "far": far, "mix": mix}


def _paged(name, B, H, Hkv, Nq, d, page, most, fp8=False, cap=0.0, slopes=False, buckets=0, far=0, window=0, sinks=0,
           mix=0):
    return {"name": name, "op": "paged", "B": B, "H": H, "Hkv": Hkv, "Nq": Nq, "d": d, "page": page, "max": most,
            "fp8": fp8, "cap": cap, "slopes": slopes, "buckets": buckets, "far": far, "window": window, "sinks": sinks,
            "mix": mix}


def listed():
    return [
        # a training step's local layer: scores capped at 50, a 4096-token window, two query heads to a key head
        _score("cap_train_8k", 1, 16, 8, 8192, 128, True, cap=50.0, window=4096),
        # a short training batch whose positions enter as a bias that falls with distance, a slope per head
        _score("slopes_train_1k", 8, 12, 12, 1024, 64, True, slopes=True),
        # documents of uneven length packed into one row of 16384 tokens, its end padded
        _score("docs_train_16k", 1, 16, 16, 16384, 128, True, docs="packed", mix=1),
        # two prompts of odd length whose first 1500 tokens see one another, capped, four query heads to a key head
        _score("prefix_prompt_5001", 2, 8, 2, 5001, 128, False, cap=30.0, prefix=1500, mix=2),
        # the smallest call: one short prompt
        _score("slopes_prompt_77", 1, 12, 12, 77, 64, False, slopes=True),
        # an encoder's padded training batch, 32 buckets for both directions
        _relative("relative_encoder_2k", 4, 12, 2048, 64, True, False, 32, 128, docs="padded", mix=3),
        # a decoder's training step, 32 buckets of the past
        _relative("relative_decoder_4k", 1, 16, 4096, 128, True, True, 32, 128, mix=4),
        # a prompt of odd length, forward alone
        _relative("relative_prompt_901", 1, 16, 901, 64, False, True, 32, 128, mix=5),
        # a serving batch of uneven lengths with capped scores, four query heads to a key head
        _paged("paged_cap_batch", 48, 32, 8, 1, 128, 64, 16384, cap=50.0, mix=6),
        # the smallest decode step: one sequence of a few hundred tokens, a slope per head
        _paged("paged_slopes_short", 1, 12, 12, 1, 64, 16, 517, slopes=True, mix=7),
        # four draft tokens a sequence over long 8-bit caches, capped, windowed with sinks
        _paged("paged8_cap_draft", 16, 32, 8, 4, 128, 64, 32768, fp8=True, cap=30.0, window=4096, sinks=4, mix=8),
        # a decoder with a learned bias, 16 sequences of up to 4096 tokens
        _paged("paged_bias_batch", 16, 16, 16, 1, 64, 32, 4096, buckets=32, far=128, mix=9),
    ]


def _spread(rng, low, high):
    """A whole number between low and high, even over its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 1)))))))


def draw(rng):
    op = rng.choice(["score", "relative", "paged"])
    d = rng.choice([64, 128])
    mix = rng.randint(0, 10 ** 6)
    cap = rng.choice([5.0, 20.0, 30.0, 50.0])
    if op == "paged":
        Hkv = rng.choice([1, 2, 4, 8, 16])
        G = rng.choice([1, 2, 3, 4, 8]) if Hkv <= 8 else 1
        B = _spread(rng, 1, 64)
        fp8 = rng.random() < 0.4
        most = 2_000_000 // (B * Hkv) * (2 if fp8 else 1)
        windowed = rng.random() < 0.3
        kind = rng.choice(["cap", "slopes", "bias"])
        c = _paged("", B, Hkv * G, Hkv, rng.choice([1, 1, 2, 4, 8]), d, rng.choice([16, 32, 64, 128]),
                   _spread(rng, 9, max(40, min(65536, most))), fp8, cap if kind == "cap" else 0.0, kind == "slopes",
                   rng.choice([16, 32]) if kind == "bias" else 0, rng.choice([64, 128, 512]),
                   _spread(rng, 64, 4096) if windowed else 0, rng.randint(1, 70) if windowed else 0, mix)
    else:
        B, Hkv = rng.choice([(1, 1), (1, 8), (2, 4), (1, 5), (3, 6)])
        H = Hkv * (rng.choice([1, 1, 2, 3]) if op == "score" else 1)
        N = _spread(rng, 50, int(min(12000, math.sqrt(3e8 / (B * H)))))
        backward = rng.random() < 0.6
        causal = rng.random() < 0.6
        docs = rng.choice(["", "packed", "padded"])
        if op == "relative":
            c = _relative("", B, H, N, d, backward, causal, rng.choice([16, 32, 48]), rng.choice([64, 128, 500]), docs,
                          cap if rng.random() < 0.3 else 0.0, mix)
        else:
            kind = rng.choice(["cap", "slopes", "docs", "prefix"])
            causal = causal or kind == "prefix"
            if kind == "docs" and not docs:
                docs = "packed"
            c = _score("", B, H, Hkv, N, d, backward, causal, cap if kind == "cap" or rng.random() < 0.2 else 0.0,
                       kind == "slopes", docs, _spread(rng, 1, N) if kind == "prefix" else 0,
                       _spread(rng, 30, 4096) if causal and rng.random() < 0.25 else 0, mix)
    del c["name"]
    return c


# ---------------------------------------------------------------- inputs ----
def _runs(case):
    """For each sequence of the batch its documents, as (first token, end) in order; tokens in none are padding."""
    r = random.Random(case["mix"])
    out = []
    for _ in range(case["B"]):
        if case["docs"] == "packed":  # documents of uneven length, a few tokens of padding at the end
            end, at, runs = case["N"] - r.randint(0, min(100, case["N"] // 10)), 0, []
            while at < end:
                n = min(end - at, max(1, int(math.exp(r.uniform(math.log(30), math.log(4000))))))
                runs.append((at, at + n))
                at += n
        elif case["docs"] == "padded":  # one document, the rest padding
            runs = [(0, r.randint(max(1, case["N"] // 2), case["N"]))]
        else:
            runs = [(0, case["N"])]
        out.append(runs)
    return out


def _bucket_map(buckets, far, both):
    """Entry L + q - k (cut to 0 .. 2 L) holds the bucket of a query at q and a key at k: exact for near distances,
    even over the logarithm up to `far`, the last bucket beyond; with `both`, the later half of the buckets is for keys
    behind the query.  Distances from L on share a bucket."""
    n = buckets // 2 if both else buckets
    exact = n // 2

    def bucket(x):
        if x < exact:
            return x
        k = 0  # the largest k with (x / exact)^(n - exact) >= (far / exact)^k
        while k < n - 1 - exact and x ** (n - exact) * exact ** (k + 1) >= far ** (k + 1) * exact ** (n - exact):
            k += 1
        return exact + k

    L = 1
    while bucket(L) < n - 1:
        L += 1
    past = [bucket(x) for x in range(L + 1)]
    future = [n + b for b in past[:0:-1]] if both else [0] * L
    return torch.tensor(future + past, dtype=torch.int32, device="cuda")


def _lengths(case):
    r = random.Random(case["mix"])
    low, high = max(case["Nq"], case["max"] // 8), max(case["Nq"], case["max"])
    return [case["max"]] + [r.randint(low, high) for _ in range(case["B"] - 1)]


def _biases(case, s, g):
    if case["slopes"]:
        s["slopes"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / case["H"]) for h in range(case["H"])], device="cuda")
    if case["buckets"]:
        s["buckets"] = _bucket_map(case["buckets"], case["far"], not case.get("causal", True))
        s["bias"] = torch.randn(case["buckets"], case["H"], generator=g, device="cuda").to(torch.bfloat16)


def _pool(case, g):
    """A paged cache: pages in random order, table entries behind a sequence's pages -1."""
    page, B, Hkv, d = case["page"], case["B"], case["Hkv"], case["d"]
    lens = _lengths(case)
    pages = [-(-n // page) for n in lens]
    total = sum(pages) + 3
    order = torch.randperm(total, generator=g, device="cuda")
    table = torch.full((B, max(pages)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = order[at:at + n].to(torch.int32)
        at += n
    gain = torch.exp(0.4 * torch.randn(Hkv, 1, d, generator=g, device="cuda"))  # channels of uneven size
    s = {"table": table, "lens": torch.tensor(lens, dtype=torch.int32, device="cuda")}
    for name in ("k", "v"):
        x = torch.randn(total, Hkv, page, d, generator=g, device="cuda").mul_(gain if name == "k" else 1.0)
        if not case["fp8"]:
            s[name] = x.to(torch.bfloat16)
            continue
        scale = torch.exp2(torch.ceil(torch.log2(x.abs().amax(dim=(2, 3)) / E4M3_MAX)))
        s[name] = (x / scale[:, :, None, None]).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        s[name + "_scale"] = scale
        del x
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    bf = torch.bfloat16
    B, H, Hkv, d = case["B"], case["H"], case["Hkv"], case["d"]
    if case["op"] == "paged":
        s = _pool(case, g)
        s["q"] = torch.randn(B, H, case["Nq"], d, generator=g, device="cuda").mul_(3.0 if case["cap"] else 1.0).to(bf)
    else:
        N = case["N"]
        s = {}
        for n, heads in (("q", H), ("k", Hkv), ("v", Hkv), ("do", H)):
            x = torch.randn(B, heads, N, d, generator=g, device="cuda")
            # a model that caps its scores has some that come near the cap
            s[n] = x.mul_(2.0 if n in "qk" and case["cap"] else 1.0).to(bf)
        if case["docs"]:
            ids = torch.full((B, N), -1, dtype=torch.int32)
            for b, runs in enumerate(_runs(case)):
                for i, (first, end) in enumerate(runs):
                    ids[b, first:end] = i
            s["docs"] = ids.cuda()
        if case["prefix"]:
            r = random.Random(case["mix"])
            s["prefix"] = torch.tensor([case["prefix"]] + [r.randint(0, case["prefix"]) for _ in range(B - 1)],
                                       dtype=torch.int32, device="cuda")
    _biases(case, s, g)
    s["case"] = case
    return s


# ----------------------------------------------------------- plain forms ----
def _seen(s):
    """[B or 1, 1, N, N]: which keys a query sees."""
    c = s["case"]
    i, j = torch.arange(c["N"], device="cuda")[:, None], torch.arange(c["N"], device="cuda")[None, :]
    seen = torch.ones(1, 1, c["N"], c["N"], dtype=torch.bool, device="cuda")
    if c["causal"]:
        seen = (j <= i)[None, None]
        if c["prefix"]:
            seen = seen | (j < s["prefix"][:, None, None, None])
    if c["window"]:
        seen = seen & (j > i - c["window"])
    if c["docs"]:
        ids = s["docs"]
        seen = seen & ((ids[:, None, :, None] == ids[:, None, None, :]) & (ids >= 0)[:, None, :, None])
    return seen


def _distance_bias(s, distance):
    """The bias of each head at q - k = distance, 32 bits: [H, *distance.shape]."""
    c = s["case"]
    if c["slopes"]:
        return s["slopes"].view(-1, *[1] * distance.dim()) * -distance.abs().float()
    L = s["buckets"].numel() // 2
    return s["bias"].float()[s["buckets"][distance.clamp(-L, L) + L].long()].movedim(-1, 0)


def _plain_score(s):
    c = s["case"]
    B, H, Hkv, N, d = (c[n] for n in ("B", "H", "Hkv", "N", "d"))
    G, tau = H // Hkv, 1.0 / math.sqrt(d)
    q, k, v = (s[n].float().reshape(B, Hkv, -1, d) for n in ("q", "k", "v"))  # a key head's queries in a row
    x = (q @ k.mT).view(B, H, N, N).mul_(tau)
    slope = None
    if c["cap"]:
        x = x.div_(c["cap"]).tanh_()
        slope = 1.0 - x * x if c["backward"] else None
        x = x.mul_(c["cap"])
    if c["slopes"] or c["buckets"]:
        i = torch.arange(N, device="cuda")
        x += _distance_bias(s, i[:, None] - i[None, :])
    x.masked_fill_(~_seen(s), -math.inf)
    m = x.amax(dim=-1, keepdim=True).clamp(min=-3e38)  # a row that sees nothing: O = 0, LSE = -inf
    p = x.sub_(m).exp_()
    total = p.sum(dim=-1, keepdim=True)
    p.div_(total.clamp(min=1e-38))
    lse = (m + total.log()).squeeze(-1)
    o = (p.view(B, Hkv, G * N, N) @ v).view(B, H, N, d)
    if not c["backward"]:
        return [o.bfloat16(), lse]
    do = s["do"].float()
    D = (do * o).sum(dim=-1, keepdim=True)
    do = do.view(B, Hkv, G * N, d)
    dv = p.view(B, Hkv, G * N, N).mT @ do
    ds = (do @ v.mT).view(B, H, N, N).sub_(D).mul_(p)
    dbias = None
    if c["buckets"]:
        # rows of 2 N read as rows of 2 N + 1 start a place later each: the diagonals become columns
        wide = torch.zeros(H, N * (2 * N + 1), device="cuda")
        wide[:, :2 * N * N].view(H, N, 2 * N)[:, :, :N] = ds.sum(dim=0)
        by = wide.view(H, N, 2 * N + 1).sum(dim=1, dtype=torch.float64)
        # column t holds k - q = t, those from N on t - (2 N + 1)
        t = torch.arange(2 * N + 1, device="cuda")
        L = s["buckets"].numel() // 2
        at = s["buckets"][torch.where(t < N, -t, 2 * N + 1 - t).clamp(-L, L) + L].long()
        dbias = torch.zeros(c["buckets"], H, dtype=torch.float64, device="cuda").index_add_(0, at, by.T)
    if slope is not None:
        ds.mul_(slope)
    ds = ds.mul_(tau).view(B, Hkv, G * N, N)
    dq, dk = (ds @ k).view(B, H, N, d), ds.mT @ q
    return [o.bfloat16(), lse, dq.bfloat16(), dk.bfloat16(), dv.bfloat16(),
            None if dbias is None else dbias.to(s["bias"].dtype)]


def _plain_paged(s):
    c = s["case"]
    B, H, Hkv, Nq, d = (c[n] for n in ("B", "H", "Hkv", "Nq", "d"))
    at = s["table"].long().clamp(min=0)
    k, v = s["k"][at].float(), s["v"][at].float()  # [B, pages, Hkv, page, d]
    if c["fp8"]:
        k.mul_(s["k_scale"][at][..., None, None])
        v.mul_(s["v_scale"][at][..., None, None])
    k, v = (x.transpose(1, 2).reshape(B, Hkv, -1, d) for x in (k, v))
    q = s["q"].float().reshape(B, Hkv, H // Hkv * Nq, d)
    x = (q @ k.mT).mul_(1.0 / math.sqrt(d)).reshape(B, H, Nq, -1)
    if c["cap"]:
        x = x.div_(c["cap"]).tanh_().mul_(c["cap"])
    j = torch.arange(x.shape[-1], device="cuda")
    last = (s["lens"].long()[:, None] - Nq + torch.arange(Nq, device="cuda"))[:, :, None]  # row i's own position
    if c["slopes"] or c["buckets"]:
        x += _distance_bias(s, last - j).transpose(0, 1)
    last = last[:, None]
    seen = j <= last
    if c["window"]:
        seen = seen & ((j > last - c["window"]) | (j < c["sinks"]))
    x.masked_fill_(~seen, -math.inf)
    m = x.amax(dim=-1, keepdim=True).clamp(min=-3e38)
    p = x.sub_(m).exp_()
    total = p.sum(dim=-1, keepdim=True)
    o = (p.reshape(B, Hkv, -1, p.shape[-1]) @ v).reshape(B, H, Nq, d) / total.clamp(min=1e-38)
    return [o.bfloat16(), (m + total.log()).squeeze(-1)]


def _run_own(s):
    from exact_io_aware_12_gb300 import api
    c = s["case"]
    how = {"softcap": c["cap"] or None, "slopes": s.get("slopes"), "bias": s.get("bias"), "buckets": s.get("buckets"),
           "window": c["window"] or None}
    if c["op"] == "paged":
        return api.fwd_paged(s["q"], s["k"], s["v"], s["table"], s["lens"], sinks=c["sinks"], k_scale=s.get("k_scale"),
                             v_scale=s.get("v_scale"), **how)
    how.update(docs=s.get("docs"), prefix=s.get("prefix"))
    o, lse = api.fwd(s["q"], s["k"], s["v"], c["causal"], **how)
    if not c["backward"]:
        return [o, lse]
    return [o, lse, *api.bwd(s["q"], s["k"], s["v"], o, s["do"], lse, c["causal"], **how)]


def run(state):
    if own:
        return list(_run_own(state))
    out = _plain_paged(state) if state["case"]["op"] == "paged" else _plain_score(state)
    return [x for x in out if x is not None]


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
    c, d, H = case, case["d"], case["H"]
    if c["op"] == "paged":
        lens = _lengths(c)
        seen = [_pairs(n, c["window"], c["sinks"], c["Nq"]) for n in lens]
        keys, pairs = sum(k for _, k in seen), sum(p for p, _ in seen)
        e = 1 if c["fp8"] else 2
        moved = keys * c["Hkv"] * d * 2 * e + keys // c["page"] * (4 + (8 * c["Hkv"] if e == 1 else 0))
        return {"bytes": moved + c["B"] * H * c["Nq"] * (d * 4 + 4), "flops": 4 * d * pairs * H}
    pairs, r = 0, random.Random(c["mix"])
    prefixes = [c["prefix"]] + [r.randint(0, c["prefix"]) for _ in range(c["B"] - 1)]
    for runs, prefix in zip(_runs(c), prefixes):
        for first, end in runs:
            if not c["causal"]:
                pairs += (end - first) ** 2
                continue
            for i in range(first, end):
                pairs += max(i + 1, min(end, prefix)) - max(first, i - c["window"] + 1 if c["window"] else 0)
    rows, kv_rows = c["B"] * H * c["N"], c["B"] * c["Hkv"] * c["N"]
    both = 2 if c["backward"] else 1  # Q K V O, and dO dQ dK dV
    return {"bytes": (rows * 2 + kv_rows * 2) * both * d * 2 + rows * 4 + (c["B"] * c["N"] * 4 if c["docs"] else 0),
            "flops": pairs * H * d * (14 if c["backward"] else 4)}


# ----------------------------------------------------------------- exact ----
def _exact_bias(s, h, distance):
    """The bias of head h at q - k = distance, and the entry of the table that it comes from."""
    if "slopes" in s:
        return -s["slopes"][h].double() * distance.abs(), None
    if "buckets" in s:
        L = s["buckets"].numel() // 2
        entry = s["buckets"].long()[torch.clamp(distance, min=-L, max=L) + L]
        return s["bias"][:, h].double()[entry], entry
    return torch.zeros((), dtype=torch.float64, device="cuda"), None


def _exact_score(s):
    """Document by document and head by head, row chunks against the keys that they see."""
    c = s["case"]
    B, H, N, d = (c[n] for n in ("B", "H", "N", "d"))
    G, tau, cap = H // c["Hkv"], 1.0 / math.sqrt(d), c["cap"]
    q, k, v, do = (s[n].double() for n in ("q", "k", "v", "do"))
    o, dq, dk, dv = torch.zeros_like(q), torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    lse = torch.full((B, H, N), -math.inf, dtype=torch.float64, device="cuda")
    table = torch.zeros(H, max(1, c["buckets"]), dtype=torch.float64, device="cuda")
    for b, runs in enumerate(_runs(c)):
        prefix = int(s["prefix"][b]) if c["prefix"] else 0
        for first, end in runs:
            for r0 in range(first, end, 1024):
                r1 = min(end, r0 + 1024)
                lo = max(first, r0 - c["window"] + 1) if c["window"] else first
                hi = max(r1, min(end, prefix)) if c["causal"] else end
                dist = torch.arange(r0, r1, device="cuda")[:, None] - torch.arange(lo, hi, device="cuda")[None, :]
                hidden = torch.zeros_like(dist, dtype=torch.bool)
                if c["causal"]:
                    hidden |= (dist < 0) & (torch.arange(lo, hi, device="cuda") >= prefix)[None, :]
                if c["window"]:
                    hidden |= dist >= c["window"]
                for h in range(H):
                    kk, vv = k[b, h // G, lo:hi], v[b, h // G, lo:hi]
                    x = torch.einsum("rd,kd->rk", q[b, h, r0:r1], kk) * tau
                    turn = None
                    if cap:
                        turn = torch.cosh(x / cap).pow(-2)
                        x = cap * torch.tanh(x / cap)
                    bias, entry = _exact_bias(s, h, dist)
                    x = torch.where(hidden, -math.inf, x + bias)
                    lse[b, h, r0:r1] = torch.logsumexp(x, dim=1)
                    p = torch.exp(x - lse[b, h, r0:r1, None])
                    o[b, h, r0:r1] = p @ vv
                    if not c["backward"]:
                        continue
                    g = do[b, h, r0:r1]
                    ds = p * (g @ vv.T - (g * o[b, h, r0:r1]).sum(1, keepdim=True))
                    if entry is not None:
                        table[h] += torch.bincount(entry.flatten(), weights=ds.flatten(), minlength=c["buckets"])
                    if turn is not None:
                        ds = ds * turn
                    dq[b, h, r0:r1] = tau * (ds @ kk)
                    dk[b, h // G, lo:hi] += tau * (ds.T @ q[b, h, r0:r1])
                    dv[b, h // G, lo:hi] += p.T @ g
    out = [o, lse]
    if c["backward"]:
        out += [dq, dk, dv] + ([table.T.contiguous()] if c["buckets"] else [])
    return out


def _exact_paged(s):
    """Sequence by sequence over its own keys in order."""
    c = s["case"]
    H, Hkv, Nq, d, page = (c[n] for n in ("H", "Hkv", "Nq", "d", "page"))
    o = torch.zeros(c["B"], H, Nq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((c["B"], H, Nq), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(_lengths(c)):
        ids = s["table"][b, :-(-n // page)].long()
        keys = torch.arange(n, device="cuda")
        if c["window"]:
            keys = keys[(keys > n - Nq - c["window"]) | (keys < c["sinks"])]
        pid, off = ids[keys // page], keys % page
        k, v = s["k"][pid, :, off].double(), s["v"][pid, :, off].double()  # [keys, Hkv, d]
        if c["fp8"]:
            k, v = k * s["k_scale"][pid].double()[..., None], v * s["v_scale"][pid].double()[..., None]
        for i in range(Nq):
            row = n - Nq + i
            see = keys <= row
            if c["window"]:
                see &= (row - keys < c["window"]) | (keys < c["sinks"])
            if row < 0:
                continue
            x = torch.einsum("hgd,khd->hgk", s["q"][b, :, i].double().view(Hkv, -1, d), k[see]).reshape(H, -1)
            x = x / math.sqrt(d)
            if c["cap"]:
                x = c["cap"] * torch.tanh(x / c["cap"])
            if c["slopes"] or c["buckets"]:
                x = x + torch.stack([_exact_bias(s, h, row - keys[see])[0] for h in range(H)])
            lse[b, :, i] = torch.logsumexp(x, dim=-1)
            p = torch.softmax(x, dim=-1).view(Hkv, H // Hkv, -1)
            o[b, :, i] = torch.einsum("hgk,khd->hgd", p, v[see]).reshape(H, d)
    return [o, lse]


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_paged(s) if case["op"] == "paged" else _exact_score(s)
