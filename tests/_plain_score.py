"""Plain 64-bit forms of attention with capped, biased or masked scores and their bounds, for the
tests of the kernels that compute it.  Torch on the CPU, nothing of the library.

Bounds, element by element, from the roundings that the kernels make (each at most half a
step: bf16 2^-8, fp16 2^-11 relative), with P, dY and dX of the exact form:
  O      the weights enter the product as bf16 and are divided by the sum of the rounded ones
         (each off by at most 2 * 2^-8), and O is rounded to bf16
  LSE    fp32: q.k sums d products, |q|.|k| 2^-24 (d + 8) of it; the cap's tanh is off by
         4e-8 and 4 * 2^-24, times the cap; a bias is rounded with the score, 4 * 2^-24 of the
         largest; the exponential 2^-21, the sum of fewer than 2^13 rounded adds
         (in 128-key steps) 2^-17
  dV     P as bf16, the result rounded
  dQ dK  P as fp16 and dX as bf16, the result rounded; D is summed in fp32 from weights of fp32,
         whose relative error e times |dP| enters dY as P e
  dBias  P as fp16 (with a cap as bf16), P e, fp32 sums, the result rounded to its type
Where fp32 itself shows (a weight's exponent is off by the score's error), the relative
errors get LSE's bound on top.

Over many elements the errors add at random, each rounding's with a variance of at most h^2 / 3,
h its half step: the variances below (s_*, the root of their sum over all elements) give what
the whole may be off, with fp32's part at its bound (where a row sees one key, dP - D is 0 and
only that is left).
"""
import math

import torch

BF16_HALF, FP16_HALF, FP32_HALF = 2.0 ** -8, 2.0 ** -11, 2.0 ** -24


def runs_of(ids):
    """Each token's run of equal numbers, numbered; -1 for numbers below 0."""
    out, run = [], -1
    for i, x in enumerate(ids):
        if i == 0 or x != ids[i - 1]:
            run += 1
        out.append(run if x >= 0 else -1)
    return out


def seen(B, N, causal, docs=None, prefix=None, window=None):
    """[B, 1, N, N] bool."""
    i, j = torch.arange(N)[:, None], torch.arange(N)[None, :]
    see = torch.ones(B, 1, N, N, dtype=torch.bool)
    for b in range(B):
        if causal:
            ok = j <= i
            if prefix is not None:
                ok = ok | (j < int(prefix[b]))
            see[b, 0] &= ok
        if window is not None:
            see[b, 0] &= j > i - window
        if docs is not None:
            run = torch.tensor(runs_of(docs[b].tolist()))
            see[b, 0] &= (run[:, None] == run[None, :]) & (run >= 0)[:, None]
    return see


def bias_of(N, slopes=None, bias=None, buckets=None):
    """[H, N, N] in 64 bits, or 0."""
    dist = torch.arange(N)[:, None] - torch.arange(N)[None, :]
    if slopes is not None:
        return -slopes.double()[:, None, None] * dist.abs()
    if bias is not None:
        far = buckets.numel() // 2
        e = buckets.long()[dist.clamp(-far, far) + far]
        ok = (e >= 0) & (e < bias.shape[0])
        return torch.where(ok[..., None], bias.double()[e.clamp(0, bias.shape[0] - 1)], 0.0).permute(2, 0, 1)
    return 0.0


class Exact:
    """The forward and, with do, the backward; o, lse, dq, dk, dv, dbias and their bounds (b_*)."""

    def __init__(self, q, k, v, causal, tau, do=None, softcap=None, slopes=None, bias=None, buckets=None, docs=None,
                 prefix=None, window=None):
        B, H, N, d = q.shape
        G = H // k.shape[1]
        q, k, v = q.double(), k.double().repeat_interleave(G, 1), v.double().repeat_interleave(G, 1)
        see = seen(B, N, causal, docs, prefix, window)
        x = q @ k.mT * tau
        size = (q.abs() @ k.abs().mT * tau).amax() * FP32_HALF * (d + 8)  # of a score's error
        turn = torch.ones_like(x)
        if softcap:
            t = torch.tanh(x / softcap)
            turn, x = 1 - t * t, softcap * t
            size = size + softcap * (4e-8 + 4 * FP32_HALF)
        add = bias_of(N, slopes, bias, buckets)
        x = x + add
        top = x.abs().masked_fill(~see, 0).amax()
        size = float(size + 4 * FP32_HALF * top)
        x = x.masked_fill(~see, -math.inf)
        self.lse = torch.logsumexp(x, dim=-1)
        p = torch.exp(x - self.lse.clamp(min=-1e300)[..., None])
        p = torch.where(see, p, 0.0)
        self.p, self.see = p, see
        self.o = p @ v
        rel = 2 * size + 2.0 ** -20  # of a weight
        b_o = (2 * BF16_HALF + rel) * (p @ v.abs()) + BF16_HALF * self.o.abs() + 1e-9
        self.b_o = b_o
        h2 = BF16_HALF ** 2 / 3
        var_o = h2 * ((p * p) @ (v * v) + self.o ** 2)
        self.s_o = float(var_o.sum().sqrt())
        self.b_lse = size + 2.0 ** -16 + 2 * FP32_HALF * self.lse.clamp(min=-1e30).abs()
        if do is None:
            return
        do = do.double()
        D = (do * self.o).sum(-1, keepdim=True)
        dp = do @ v.mT
        dp_err = (do.abs() @ v.abs().mT) * FP32_HALF * (d + 2)
        e = (p * ((rel + 2.0 ** -20) * dp.abs() + dp_err)).sum(-1, keepdim=True)
        dy = p * (dp - D)
        dx = dy * turn * tau
        # an error of dY before dX's rounding, and of dX
        ey = (FP16_HALF + rel) * dy.abs() + p * (e + dp_err) + 2.0 ** -39 * (dp - D).abs() * see
        turn_err = 1e-6 * p * (dp - D).abs() if softcap else 0.0
        ex = tau * (ey * turn + turn_err) * (1 + BF16_HALF) + BF16_HALF * dx.abs()

        def shared(t):
            return t.view(B, H // G, G, N, -1).sum(2)
        var_x = (h2 + FP16_HALF ** 2 / 3) * dx * dx
        self.dq, self.b_dq = dx @ k, ex @ k.abs()
        e32 = tau * (rel * dy.abs() + p * (e + dp_err))
        self.s_dq = float((var_x @ (k * k) + h2 * self.dq ** 2).sum().sqrt() + (e32 @ k.abs()).norm())
        self.dk, self.b_dk = shared(dx.mT @ q), shared(ex.mT @ q.abs())
        self.dv, self.b_dv = shared(p.mT @ do), shared(((BF16_HALF + rel) * p).mT @ do.abs())
        self.s_dk = float((shared(var_x.mT @ (q * q)) + h2 * self.dk ** 2).sum().sqrt() + shared(e32.mT @ q.abs()).norm())
        self.s_dv = float((shared(h2 * (p * p).mT @ (do * do)) + h2 * self.dv ** 2).sum().sqrt())
        for n in ("dq", "dk", "dv"):
            b = getattr(self, "b_" + n)
            setattr(self, "b_" + n, b * (1 + 1e-3) + BF16_HALF * getattr(self, n).abs() + 1e-9)
        if bias is not None:
            far = buckets.numel() // 2
            dist = torch.arange(N)[:, None] - torch.arange(N)[None, :]
            at = buckets.long()[dist.clamp(-far, far) + far]
            nb = bias.shape[0]
            at = torch.where((at >= 0) & (at < nb), at, nb).flatten()

            def by(t):
                return torch.zeros(nb + 1, H, dtype=torch.float64).index_add_(0, at, t.sum(0).flatten(1).T)[:nb]
            self.dbias = by(dy)
            b = by(ey) + 2.0 ** -18 * by(dy.abs()) + (BF16_HALF * by(dy.abs()) if softcap else 0.0)
            half = BF16_HALF if softcap else FP16_HALF
            out = BF16_HALF if bias.dtype == torch.bfloat16 else FP32_HALF
            self.s_dbias = float(((half ** 2 * by(dy * dy) + out ** 2 * self.dbias ** 2) / 3).sum().sqrt()
                                 + by(e32 / tau).norm())
            self.b_dbias = b + (BF16_HALF if bias.dtype == torch.bfloat16 else FP32_HALF) * self.dbias.abs() + 1e-9


def within(got, want, bound, what):
    got = got.detach().cpu().double()
    assert got.shape == want.shape, what
    same = got == want  # (infinities)
    off = torch.where(same, torch.zeros_like(want), (got - want).abs() / bound)
    assert bool((off <= 1).all()), f"{what}: {float(off.nan_to_num(math.inf).max()):.3g} of its bound"
