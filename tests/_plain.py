"""Plain 64-bit forms of windowed attention with sinks and of the paged cache, for the
tests of the kernels that compute them.  Torch on the CPU, nothing of the library."""
import math

import torch

BF16_HALF = 2.0 ** -8    # a rounding to bf16 is off by at most this, relative
FP16_HALF = 2.0 ** -11
FP32_HALF = 2.0 ** -24
E4M3_HALF = 2.0 ** -4
E4M3_MAX = 448.0


def visible(nq, nk, window=0, sinks=0):
    """[nq, nk] bool: row i stands at position nk - nq + i."""
    i = torch.arange(nk - nq, nk)[:, None]
    j = torch.arange(nk)[None, :]
    see = j <= i
    if window:
        see = see & ((j > i - window) | (j < sinks))
    return see


def attention(q, k, v, tau, see):
    """(O, LSE, P) in 64 bits; rows without a visible key give 0 and -inf."""
    q, k, v = q.double(), k.double(), v.double()
    s = (q @ k.transpose(-1, -2) * tau).masked_fill(~see, -math.inf)
    lse = torch.logsumexp(s, dim=-1) if s.shape[-1] else torch.full(s.shape[:-1], -math.inf, dtype=torch.float64)
    p = torch.exp(s - lse.clamp(min=-1e300)[..., None])
    # (a hidden key's value does not count, whatever it is)
    v = torch.where(see.any(dim=-2)[..., :, None], v, torch.zeros_like(v))
    return p @ v, lse, p


def attention_bwd(q, k, v, do, tau, see):
    q, k, v, do = q.double(), k.double(), v.double(), do.double()
    o, _, p = attention(q, k, v, tau, see)
    dv = p.transpose(-1, -2) @ do
    ds = p * (do @ v.transpose(-1, -2) - (do * o).sum(-1, keepdim=True)) * tau
    return ds @ k, ds.transpose(-1, -2) @ q, dv


def rotate(x, pos, inv_freq, interleaved):
    """x [T, H, d] turned at positions pos [T] (64 bits)."""
    x = x.double().clone()
    rot = 2 * inv_freq.shape[0]
    a = pos.double()[:, None] * inv_freq
    c, s = a.cos()[:, None], a.sin()[:, None]
    r = x[..., :rot].clone()
    lo, hi = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :rot // 2], r[..., rot // 2:])
    lo2, hi2 = lo * c - hi * s, hi * c + lo * s
    if interleaved:
        x[..., 0:rot:2], x[..., 1:rot:2] = lo2, hi2
    else:
        x[..., :rot // 2], x[..., rot // 2:rot] = lo2, hi2
    return x


def scale_of(bound):
    """Smallest 2^e >= 2^-100 (and at most 2^121) with bound <= 448 * 2^e."""
    e = -100
    while e < 121 and bound > E4M3_MAX * 2.0 ** e:
        e += 1
    return 2.0 ** e


def to_e4m3(x):
    """Nearest e4m3 value (ties to even, saturating), as 64-bit values.  x: 64 bits."""
    x = x.clamp(-E4M3_MAX, E4M3_MAX)
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -30))).clamp(min=-6)
    # (log2 may be off next to a power of two: the quantum of the upper binade on a value
    # just below it would be too wide)
    e = torch.where(x.abs() < 2.0 ** e, e - 1, e).clamp(min=-6)
    e = torch.where(x.abs() >= 2.0 ** (e + 1), e + 1, e)
    quantum = 2.0 ** (e - 3)
    return torch.round(x / quantum) * quantum   # torch.round: ties to even


def make_pages(lens, page, gen, spare=2):
    """(num_pages, page_table int32 [B, max_pages] with -1 behind each sequence): pages in random order."""
    need = [-(-n // page) for n in lens]
    total = sum(need) + spare
    order = torch.randperm(total, generator=gen)
    table = torch.full((len(lens), max(1, max(need, default=1))), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n].to(torch.int32)
        at += n
    return total, table


def gather(cache, table_row, n, scale=None):
    """Keys 0 .. n - 1 of a sequence: [H_kv, n, d] in 64 bits."""
    page = cache.shape[2]
    ids = table_row[:-(-n // page)].long()
    if cache.dtype == torch.float8_e4m3fn:
        x = cache.view(torch.uint8)[ids].view(cache.dtype).double()
    else:
        x = cache[ids].double()
    if scale is not None:
        x = x * scale[ids].double()[:, :, None, None]
    return x.transpose(0, 1).reshape(cache.shape[1], -1, cache.shape[3])[:, :n]
