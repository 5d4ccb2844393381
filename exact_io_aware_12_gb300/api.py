"""Torch-facing helpers over the C ABI.

PyTorch only supplies device memory and the current stream; the tensors'
data pointers go straight to ``fa_fwd`` / ``fa_bwd``.  Inputs must be CUDA
bf16 tensors, contiguous, shaped [B, H, N, d].  The paged entry points
(``kv_append``, ``fwd_paged``), windows with sinks and attention with capped,
biased or masked scores check and call in a small extension module
(csrc/torch_binding.cpp), for their kernels can take less time than a call from
Python.
"""
from __future__ import annotations

import math
from typing import Optional, Tuple

import torch

from . import _lib


def _stream_handle(device: torch.device) -> int:
    if device.index is None:
        return torch.cuda.current_stream(device).cuda_stream
    return torch._C._cuda_getCurrentRawStream(device.index)  # without building a Stream object


def _check_inputs(*ts: torch.Tensor) -> Tuple[int, int, int, int]:
    ref = ts[0]
    if ref.dim() != 4:
        raise ValueError("expected [B, H, N, d] tensors")
    for t in ts:
        if not t.is_cuda or t.dtype != torch.bfloat16 or not t.is_contiguous():
            raise ValueError("inputs must be contiguous CUDA bf16 tensors")
        if t.shape != ref.shape or t.device != ref.device:
            raise ValueError("inputs must share shape and device")
    B, H, N, d = ref.shape
    return B, H, N, d


def _check_blocks(blocks: torch.Tensor, ref: torch.Tensor) -> int:
    """A block mask: CUDA uint8/bool, contiguous, shaped [nb, nb] (one mask) or
    [B, H, nb, nb] / [B*H, nb, nb] (one per head), nb = ceil(N / 128).
    Returns mask_heads."""
    B, H, N, _ = ref.shape
    nb = (N + _lib.BLOCK_MASK_EDGE - 1) // _lib.BLOCK_MASK_EDGE
    if not blocks.is_cuda or blocks.device != ref.device or not blocks.is_contiguous():
        raise ValueError("block mask must be a contiguous tensor on the inputs' device")
    if blocks.dtype not in (torch.uint8, torch.bool):
        raise ValueError("block mask must be uint8 or bool")
    if tuple(blocks.shape[-2:]) != (nb, nb):
        raise ValueError(f"block mask must end in ({nb}, {nb})")
    heads = blocks.numel() // (nb * nb)
    if blocks.dim() == 2:
        return 1
    if heads != B * H:
        raise ValueError(f"block mask has {heads} heads, expected 1 or {B * H}")
    return heads


def distance_buckets(num_buckets: int, max_distance: int, bidirectional: bool = False,
                     device=None) -> torch.Tensor:
    """The ``buckets`` of a learned relative position bias whose buckets widen with
    the distance: int32 [2 L + 1] on ``device``, entry L + i - j the bucket of a
    query at i and a key at j.  The first half of the buckets holds one distance
    each, the others grow evenly over the logarithm up to ``max_distance``, and the
    last holds all beyond.  ``bidirectional``: half of the buckets (num_buckets even)
    for keys at or before the query, half for keys behind it; else these share bucket 0.
    The borders are exact (whole numbers compared, no rounded logarithm).  L is the
    first distance of the last bucket."""
    n = num_buckets // 2 if bidirectional else num_buckets
    exact = n // 2
    if num_buckets < 2 or exact < 1 or max_distance <= exact or (bidirectional and num_buckets % 2):
        raise ValueError("need at least two buckets a side, evenly split, and max_distance beyond the exact ones")
    if num_buckets > _lib.SCORE_MAX_BUCKETS or max_distance > _lib.SCORE_MAX_DISTANCE:
        raise ValueError(f"at most {_lib.SCORE_MAX_BUCKETS} buckets and max_distance {_lib.SCORE_MAX_DISTANCE}")
    log_n = n - exact  # bucket exact + k begins at the first x with (x / exact)^log_n >= (max_distance / exact)^k
    past, b = [], 0
    while not past or past[-1] < n - 1:
        x = len(past)
        if x <= exact:
            b = x
        else:
            while b + 1 < n and (x ** log_n * exact ** (b + 1 - exact)
                                 >= max_distance ** (b + 1 - exact) * exact ** log_n):
                b += 1
        past.append(min(b, n - 1))
    future = [n + x for x in past[:0:-1]] if bidirectional else [0] * (len(past) - 1)
    return torch.tensor(future + past, dtype=torch.int32, device=device)


def fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, causal: bool,
        tau: Optional[float] = None, out: Optional[torch.Tensor] = None,
        lse: Optional[torch.Tensor] = None, o_fp32: bool = False, window: Optional[int] = None,
        blocks: Optional[torch.Tensor] = None, sinks: int = 0, softcap: Optional[float] = None,
        slopes: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
        buckets: Optional[torch.Tensor] = None, docs: Optional[torch.Tensor] = None,
        prefix: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """Forward pass.  Returns (O, LSE): O bf16 (fp32 with ``o_fp32``) and LSE
    fp32 [B, H, N].  ``window`` (with ``causal``): each query sees only its
    ``window`` most recent keys (fa_fwd_window), and with ``sinks`` also the
    first ``sinks`` keys of the sequence (fa_fwd_sinks).  ``blocks``: a block
    mask over 128 x 128 blocks (fa_fwd_blocks).

    Any of the following changes the scores or hides keys (fa_fwd_score); k and v
    may then have fewer heads, [B, H_kv, N, d]: query head h reads key head
    h // (H // H_kv).  A bf16 O, no sinks and no block mask go with them.
      softcap  scores become softcap * tanh(score / softcap)
      slopes   fp32 [H]: scores fall by slopes[h] for each position between
               query and key
      bias     bf16 or fp32 [num_buckets, H] with ``buckets``, int32
               [2 * max_distance + 1]: bias[buckets[max_distance + i - j], h] is
               added, the distance cut to +-max_distance (see distance_buckets;
               an entry outside [0, num_buckets) adds nothing)
      docs     int32 [B, N]: tokens see their own run of equal numbers only; a
               number below 0 is padding, which sees nothing and nothing sees
      prefix   int32 [B], with ``causal``: the first prefix[b] positions are
               visible from before them, too
    Values are finite, in padding and behind a mask, too.  The workspace (only
    documents take one) is allocated with torch when not given."""
    if (softcap is not None or slopes is not None or bias is not None or buckets is not None
            or docs is not None or prefix is not None):
        if o_fp32 or sinks or blocks is not None:
            raise ValueError("capped, biased or masked scores go with a bf16 O, no sinks and no block mask")
        return _lib.binding().fwd_score(q, k, v, causal, tau, softcap, slopes, bias, buckets, docs,
                                        prefix, window, out, lse, workspace)
    if workspace is not None:
        raise ValueError("this forward takes no workspace")
    if sinks and window is None:
        raise ValueError("sinks need a window")
    if window is not None and (not causal or o_fp32):
        raise ValueError("a window needs causal=True and a bf16 O")
    if blocks is not None and (o_fp32 or window is not None):
        raise ValueError("a block mask needs a bf16 O and no window")
    if sinks:
        return _lib.binding().fwd_sinks(q, k, v, tau, window, sinks, out, lse)
    B, H, N, d = _check_inputs(q, k, v)
    tau = 1.0 / math.sqrt(d) if tau is None else float(tau)
    o_dtype = torch.float32 if o_fp32 else torch.bfloat16
    if out is None:
        out = torch.empty(q.shape, dtype=o_dtype, device=q.device)
    if lse is None:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    if blocks is not None:
        heads = _check_blocks(blocks, q)
        code = _lib.fa_fwd_blocks(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                                  lse.data_ptr(), B, H, N, d, tau, int(bool(causal)),
                                  blocks.data_ptr(), heads, _stream_handle(q.device))
        _lib.check(code, "fa_fwd_blocks")
        return out, lse
    if window is not None:
        code = _lib.fa_fwd_window(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                                  lse.data_ptr(), B, H, N, d, tau, int(window),
                                  _stream_handle(q.device))
        _lib.check(code, "fa_fwd_window")
        return out, lse
    fn = _lib.fa_fwd_o32 if o_fp32 else _lib.fa_fwd
    code = fn(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(),
              B, H, N, d, tau, int(bool(causal)), _stream_handle(q.device))
    _lib.check(code, "fa_fwd_o32" if o_fp32 else "fa_fwd")
    return out, lse


def workspace_bytes(B: int, H: int, N: int, d: int) -> int:
    return _lib.fa_bwd_workspace_size(B, H, N, d)


def score_workspace_bytes(q: torch.Tensor, causal: bool, bias: Optional[torch.Tensor] = None,
                          buckets: Optional[torch.Tensor] = None, docs: Optional[torch.Tensor] = None,
                          prefix: Optional[torch.Tensor] = None, backward: bool = True,
                          bias_grad: bool = True) -> int:
    """Bytes of workspace that ``bwd`` (or ``fwd``) takes for queries of this size with
    these options (``bias_grad`` as in ``bwd``)."""
    B, H, N, d = q.shape
    at = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    s = _lib.Score(0.0, None, at(bias), at(buckets), int(bias is not None and bias.dtype == torch.float32),
                   0 if bias is None else bias.shape[0], 0 if buckets is None else buckets.shape[0] // 2,
                   at(docs), at(prefix), 0)
    if backward:
        size = _lib.fa_bwd_score_workspace_size if bias_grad else _lib.fa_bwd_score_frozen_workspace_size
        return size(B, H, N, d, int(bool(causal)), s)
    return _lib.fa_fwd_score_workspace_size(B, N, s)


def bwd(q, k, v, o, do, lse, causal: bool, tau: Optional[float] = None,
        dq: Optional[torch.Tensor] = None, dk: Optional[torch.Tensor] = None,
        dv: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
        window: Optional[int] = None, blocks: Optional[torch.Tensor] = None, sinks: int = 0,
        softcap: Optional[float] = None, slopes: Optional[torch.Tensor] = None,
        bias: Optional[torch.Tensor] = None, buckets: Optional[torch.Tensor] = None,
        docs: Optional[torch.Tensor] = None, prefix: Optional[torch.Tensor] = None,
        dbias: Optional[torch.Tensor] = None, bias_grad: bool = True):
    """Backward pass.  Returns (dQ, dK, dV), bf16.  ``workspace`` (a byte
    tensor of at least ``workspace_bytes`` bytes) is allocated with torch when
    not given, so the library itself allocates nothing.

    ``softcap`` to ``prefix`` as in ``fwd`` (fa_bwd_score; the workspace is then of
    ``score_workspace_bytes``): dK and dV have k's heads, summed over the query
    heads that share them.  With a ``bias`` its gradient, of its shape and type,
    comes fourth (in ``dbias`` where given), unless ``bias_grad`` is false."""
    if dbias is not None and bias is None:
        raise ValueError("dbias without a bias")
    if (softcap is not None or slopes is not None or bias is not None or buckets is not None
            or docs is not None or prefix is not None):
        if sinks or blocks is not None:
            raise ValueError("capped, biased or masked scores go with no sinks and no block mask")
        if not bias_grad and dbias is not None:
            raise ValueError("dbias without bias_grad")
        grads = _lib.binding().bwd_score(q, k, v, o, do, lse, causal, tau, softcap, slopes, bias, buckets,
                                         docs, prefix, window, dq, dk, dv, dbias if bias_grad else False,
                                         workspace)
        return grads if bias is not None and bias_grad else grads[:3]
    if sinks:
        if window is None:
            raise ValueError("sinks need a window")
        if not causal or blocks is not None:
            raise ValueError("a window needs causal=True and no block mask")
        return _lib.binding().bwd_sinks(q, k, v, o, do, lse, tau, window, sinks, dq, dk, dv, workspace)
    B, H, N, d = _check_inputs(q, k, v, o, do)
    if lse.dtype != torch.float32 or not lse.is_contiguous() or lse.shape != (B, H, N):
        raise ValueError("lse must be contiguous fp32 [B, H, N]")
    tau = 1.0 / math.sqrt(d) if tau is None else float(tau)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    need = workspace_bytes(B, H, N, d)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    if blocks is not None:
        if window is not None:
            raise ValueError("a block mask needs no window")
        heads = _check_blocks(blocks, q)
        code = _lib.fa_bwd_blocks(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                                  do.data_ptr(), lse.data_ptr(), dq.data_ptr(), dk.data_ptr(),
                                  dv.data_ptr(), workspace.data_ptr(), workspace.numel(), B, H, N,
                                  d, tau, int(bool(causal)), blocks.data_ptr(), heads,
                                  _stream_handle(q.device))
        _lib.check(code, "fa_bwd_blocks")
        return dq, dk, dv
    if window is not None:
        if not causal:
            raise ValueError("a window needs causal=True")
        code = _lib.fa_bwd_window(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                                  do.data_ptr(), lse.data_ptr(), dq.data_ptr(), dk.data_ptr(),
                                  dv.data_ptr(), workspace.data_ptr(), workspace.numel(), B, H, N,
                                  d, tau, int(window), _stream_handle(q.device))
        _lib.check(code, "fa_bwd_window")
        return dq, dk, dv
    code = _lib.fa_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), do.data_ptr(),
                       lse.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                       workspace.data_ptr(), workspace.numel(), B, H, N, d, tau,
                       int(bool(causal)), _stream_handle(q.device))
    _lib.check(code, "fa_bwd")
    return dq, dk, dv


def fwd_fp8(q8: torch.Tensor, k8: torch.Tensor, v8: torch.Tensor, q_scale: float, k_scale: float,
            v_scale: float, causal: bool, tau: Optional[float] = None,
            out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None):
    """FP8 forward (fa_fwd_fp8): q8, k8, v8 hold e4m3 bytes (uint8 or
    float8_e4m3fn tensors, contiguous, [B, H, N, 128]) whose values are
    byte * scale.  Returns (O bf16 [B, H, N, 128], LSE fp32 [B, H, N])."""
    ts = (q8, k8, v8)
    for t in ts:
        if not t.is_cuda or t.element_size() != 1 or not t.is_contiguous() or t.dim() != 4:
            raise ValueError("q8, k8, v8 must be contiguous CUDA [B, H, N, d] 1-byte tensors")
        if t.shape != q8.shape or t.device != q8.device:
            raise ValueError("q8, k8, v8 must share shape and device")
    B, H, N, d = q8.shape
    tau = 1.0 / math.sqrt(d) if tau is None else float(tau)
    if out is None:
        out = torch.empty((B, H, N, d), dtype=torch.bfloat16, device=q8.device)
    if lse is None:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q8.device)
    code = _lib.fa_fwd_fp8(q8.data_ptr(), k8.data_ptr(), v8.data_ptr(), out.data_ptr(),
                           lse.data_ptr(), B, H, N, d, tau, int(bool(causal)), float(q_scale),
                           float(k_scale), float(v_scale), _stream_handle(q8.device))
    _lib.check(code, "fa_fwd_fp8")
    return out, lse


def decode_workspace_bytes(B: int, H: int, Nq: int, Nk: int, d: int) -> int:
    return _lib.fa_decode_workspace_size(B, H, Nq, Nk, d)


def fwd_decode(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, causal: bool,
               tau: Optional[float] = None, out: Optional[torch.Tensor] = None,
               lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """Decode forward (fa_fwd_decode): q [B, H, Nq, d] (1 <= Nq <= 8) against
    the KV cache k, v [B, H, Nk, d]; with ``causal`` the queries are the last Nq
    positions.  Returns (O bf16 [B, H, Nq, d], LSE fp32 [B, H, Nq]).  The
    split workspace is allocated with torch when not given."""
    if q.dim() != 4:
        raise ValueError("expected [B, H, Nq, d] queries")
    B, H, Nq, d = q.shape
    _check_inputs(k, v)
    for t in (q, k, v):
        if not t.is_cuda or t.dtype != torch.bfloat16 or not t.is_contiguous():
            raise ValueError("inputs must be contiguous CUDA bf16 tensors")
    if k.shape[:2] != (B, H) or k.shape[3] != d or k.device != q.device:
        raise ValueError("k, v must be [B, H, Nk, d] on q's device")
    Nk = k.shape[2]
    tau = 1.0 / math.sqrt(d) if tau is None else float(tau)
    if out is None:
        out = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty((B, H, Nq), dtype=torch.float32, device=q.device)
    need = decode_workspace_bytes(B, H, Nq, Nk, d)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    wp, wn = (workspace.data_ptr(), workspace.numel()) if workspace is not None else (None, 0)
    code = _lib.fa_fwd_decode(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                              lse.data_ptr(), B, H, Nq, Nk, d, tau, int(bool(causal)), wp, wn,
                              _stream_handle(q.device))
    _lib.check(code, "fa_fwd_decode")
    return out, lse


def kv_append(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
              page_table: torch.Tensor, lens: torch.Tensor, cu_new: Optional[torch.Tensor] = None,
              q: Optional[torch.Tensor] = None, inv_freq: Optional[torch.Tensor] = None,
              interleaved: bool = False, k_scale: Optional[torch.Tensor] = None,
              v_scale: Optional[torch.Tensor] = None, q_out: Optional[torch.Tensor] = None):
    """Appends new tokens' k, v [T, H_kv, d] (any token and head strides that are
    multiples of 8) to the paged cache k_cache, v_cache [num_pages, H_kv,
    page_size, d] (fa_kv_append; with ``k_scale`` and ``v_scale`` [num_pages,
    H_kv] the cache is e4m3: fa_kv_append_fp8).  Sequence b's tokens are rows
    cu_new[b] .. cu_new[b + 1] - 1 (int32 [B + 1]; None: T / B each), placed
    behind the lens[b] keys that it has; add the new tokens to ``lens``
    afterwards.  ``inv_freq`` (float64 [rot / 2], radians per position) turns
    the first rot columns of the keys, and of ``q`` [T, H, d] where given, by
    their position; ``interleaved`` pairs neighbouring columns.  Returns the
    rotated queries (``q_out``, or a new tensor), or None without ``q``."""
    return _lib.binding().kv_append(k, v, k_cache, v_cache, page_table, lens, cu_new, q, inv_freq,
                                    interleaved, k_scale, v_scale, q_out)


def paged_workspace_bytes(q: torch.Tensor, k_cache: torch.Tensor, page_table: torch.Tensor,
                          window: Optional[int] = None, sinks: int = 0) -> int:
    """Bytes of workspace that ``fwd_paged`` takes for tensors of these sizes."""
    B, H, Nq, d = q.shape
    P, Hkv, page, _ = k_cache.shape
    fp8 = k_cache.dtype != torch.bfloat16
    c = _lib.PagedCache(None, None, 1 if fp8 else None, None, None, None, B, Hkv, d, P, page,
                        page_table.shape[1])
    return _lib.fa_paged_workspace_size(c, H, Nq, window or 0, sinks)


def fwd_paged(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
              page_table: torch.Tensor, lens: torch.Tensor, tau: Optional[float] = None,
              window: Optional[int] = None, sinks: int = 0, k_scale: Optional[torch.Tensor] = None,
              v_scale: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
              lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
              softcap: Optional[float] = None, slopes: Optional[torch.Tensor] = None,
              bias: Optional[torch.Tensor] = None, buckets: Optional[torch.Tensor] = None):
    """Attention of a decode step over a paged cache (fa_fwd_paged; with scales
    the cache is e4m3: fa_fwd_paged_fp8).  q [B, H, Nq, d] (1 <= Nq <= 8, any
    strides that are multiples of 8) holds each sequence's last Nq positions,
    which ``lens`` counts; query head h reads key head h // (H // H_kv).
    ``window`` and ``sinks`` as in ``fwd``.  Returns (O bf16 [B, H, Nq, d], LSE
    fp32 [B, H, Nq]); a row without keys gives 0 and -inf.  The workspace is
    allocated with torch when not given.  ``softcap``, ``slopes``, ``bias`` and
    ``buckets`` as in ``fwd`` (fa_fwd_paged_score): distances are between positions
    of the sequence."""
    if softcap is not None or slopes is not None or bias is not None or buckets is not None:
        return _lib.binding().fwd_paged(q, k_cache, v_cache, page_table, lens, tau, window, sinks, k_scale,
                                        v_scale, out, lse, workspace, softcap, slopes, bias, buckets)
    return _lib.binding().fwd_paged(q, k_cache, v_cache, page_table, lens, tau, window, sinks, k_scale,
                                    v_scale, out, lse, workspace)


def last_device_error(device: Optional[torch.device] = None) -> int:
    device = device or torch.device("cuda", torch.cuda.current_device())
    return _lib.fa_last_device_error(_stream_handle(device))


class _Once(torch.autograd.Function):
    """Gradients as they are, from what they depend on: differentiating them raises."""

    @staticmethod
    def forward(ctx, n, *ts):
        return tuple(t.view_as(t) for t in ts[:n])

    @staticmethod
    def backward(ctx, *gs):
        raise RuntimeError("attention's gradients have no derivative")


def _once(grads, *inputs):
    """With create_graph, gradients that the kernels wrote (autograd would take them for constants, and a second
    derivative would lack them without a word; torch's once_differentiable leaves them so where only saved tensors,
    not the incoming gradient, depend on the leaves)."""
    if not torch.is_grad_enabled():
        return grads
    return _Once.apply(len(grads), *grads, *inputs)


class _Attention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, causal, tau, window, sinks):
        o, lse = fwd(q, k, v, causal, tau, window=window, sinks=sinks)
        ctx.save_for_backward(q, k, v, o, lse)
        ctx.causal, ctx.tau, ctx.window, ctx.sinks = causal, tau, window, sinks
        return o

    @staticmethod
    def backward(ctx, do):
        q, k, v, o, lse = ctx.saved_tensors
        dq, dk, dv = _once(bwd(q, k, v, o, do.contiguous(), lse, ctx.causal, ctx.tau, window=ctx.window,
                               sinks=ctx.sinks), q, k, v, do)
        return dq, dk, dv, None, None, None, None


class _ScoredAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, bias, causal, tau, window, softcap, slopes, buckets, docs, prefix):
        o, lse = fwd(q, k, v, causal, tau, window=window, softcap=softcap, slopes=slopes, bias=bias,
                     buckets=buckets, docs=docs, prefix=prefix)
        ctx.save_for_backward(q, k, v, o, lse, bias, slopes, buckets, docs, prefix)
        ctx.how = causal, tau, window, softcap
        return o

    @staticmethod
    def backward(ctx, do):
        q, k, v, o, lse, bias, slopes, buckets, docs, prefix = ctx.saved_tensors
        causal, tau, window, softcap = ctx.how
        grads = _once(bwd(q, k, v, o, do.contiguous(), lse, causal, tau, window=window, softcap=softcap,
                          slopes=slopes, bias=bias, buckets=buckets, docs=docs, prefix=prefix,
                          bias_grad=ctx.needs_input_grad[3]), q, k, v, do, bias)
        dbias = grads[3] if len(grads) > 3 else None
        return (*grads[:3], dbias, None, None, None, None, None, None, None, None)


def attention(q, k, v, causal: bool = False, tau: Optional[float] = None,
              window: Optional[int] = None, sinks: int = 0, softcap: Optional[float] = None,
              slopes: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
              buckets: Optional[torch.Tensor] = None, docs: Optional[torch.Tensor] = None,
              prefix: Optional[torch.Tensor] = None) -> torch.Tensor:
    """O = softmax(tau Q K^T [causal]) V with autograd support; ``window`` and
    ``sinks``, and ``softcap`` to ``prefix``, as in ``fwd``.  Gradients flow to q, k, v and
    ``bias`` (not to ``slopes``), and have none of their own: with ``create_graph`` a second
    derivative through them raises RuntimeError.  A backward pass may be captured in a CUDA graph while no
    eager graph of the same leaves lives (torch ties a leaf to the stream that it was first
    used on)."""
    if (softcap is not None or slopes is not None or bias is not None or buckets is not None
            or docs is not None or prefix is not None):
        if sinks:
            raise ValueError("capped, biased or masked scores go with no sinks")
        if slopes is not None and slopes.requires_grad:
            raise ValueError("slopes take no gradient")
        return _ScoredAttention.apply(q, k, v, bias, causal, tau, window, softcap, slopes, buckets, docs, prefix)
    return _Attention.apply(q, k, v, causal, tau, window, sinks)


class HostPipeline:
    """Forward + backward steps on tensors that live in pinned host memory,
    through the library's native host pipeline (fa_host_pipeline_* in
    include/fa.h).

    Each step copies its Q, K, V, dO in, runs fwd and bwd, and copies O, LSE,
    dQ, dK, dV back out.  The library owns ``depth`` device buffer sets
    (default 2) and one stream per copy direction; the kernels run on the
    caller's current stream.  The copies of neighbouring steps overlap each
    other's kernels, as a training or serving loop overlaps the next batch's
    transfer with the current step.  ``step`` only enqueues work;
    ``synchronize`` waits for all of it.  Host tensors must be pinned,
    contiguous, of the configured shape (bf16; LSE fp32), and must not be
    touched until the step has finished."""

    def __init__(self, B: int, H: int, N: int, d: int, causal: bool, tau: Optional[float] = None,
                 device: Optional[torch.device] = None, depth: int = 2):
        self.shape = (B, H, N, d)
        self.tau = 1.0 / math.sqrt(d) if tau is None else float(tau)
        self.device = device or torch.device("cuda", torch.cuda.current_device())
        self.stream = torch.cuda.current_stream(self.device)
        with torch.cuda.device(self.device):
            code, self._p = _lib.fa_host_pipeline_create(B, H, N, d, self.tau, int(bool(causal)),
                                                         int(depth), self.stream.cuda_stream)
        _lib.check(code, "fa_host_pipeline_create")

    def _check(self, ts, dtype, shape):
        for t in ts:
            if t.is_cuda or t.dtype != dtype or tuple(t.shape) != shape or not t.is_contiguous():
                raise ValueError(f"host tensors must be contiguous CPU {dtype} of shape {shape}")

    def step(self, q, k, v, do, o_out, lse_out, dq_out, dk_out, dv_out) -> None:
        self._check((q, k, v, do, o_out, dq_out, dk_out, dv_out), torch.bfloat16, self.shape)
        self._check((lse_out,), torch.float32, self.shape[:3])
        code = _lib.fa_host_pipeline_step(self._p, q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                          do.data_ptr(), o_out.data_ptr(), lse_out.data_ptr(),
                                          dq_out.data_ptr(), dk_out.data_ptr(), dv_out.data_ptr())
        _lib.check(code, "fa_host_pipeline_step")

    def mark(self) -> torch.cuda.Event:
        """A timing event on the kernels' stream after every step enqueued so
        far, copies included; copies enqueued later start after it."""
        e = torch.cuda.Event(enable_timing=True)
        e.record(self.stream)  # materialise the handle
        _lib.check(_lib.fa_host_pipeline_mark(self._p, e.cuda_event), "fa_host_pipeline_mark")
        return e

    def finish_event(self) -> torch.cuda.Event:
        return self.mark()

    def synchronize(self) -> None:
        _lib.check(_lib.fa_host_pipeline_sync(self._p), "fa_host_pipeline_sync")

    def close(self) -> None:
        if getattr(self, "_p", None) is not None and self._p.value:
            code = _lib.fa_host_pipeline_destroy(self._p)
            self._p = None
            _lib.check(code, "fa_host_pipeline_destroy")

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
