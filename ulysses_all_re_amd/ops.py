"""PyTorch operator over the exchange: autograd, the 4-D all-to-all API, torch.compile.

The FastVideo ``ulysses_a2a`` API page exposes the exchange as
``try_all_to_all_4D(x, scatter_dim, gather_dim)`` and wraps it in an
autograd function.  Here the same entry point works on the rank-stacked
tensors of this library (all ``w`` virtual ranks in one tensor, rank axis
first), and the dims name axes of one rank's 4-D tensor ``[B, S, H, D]``:

    scatter_dim=2, gather_dim=1  -> mode 0 (scatter heads, gather sequence)
    scatter_dim=1, gather_dim=2  -> mode 1 (the inverse)

The exchange is a permutation of elements, so its gradient is the inverse
permutation: the backward of mode m is the exchange in mode 1 - m, run by
the same HIP kernels.  The operator is registered with ``torch.library`` and
has a shape-only fake implementation, so ``torch.compile`` traces it as one
opaque call (where the page has to decline inside compiled regions, this
operator needs no decline).  Every call runs the HIP library; there is no
other implementation.

``chunked=True`` runs the page's chunked form: one batch plane at a time
through a window sized for one plane of every rank.  As the page's
communicator keeps one registered window and rebuilds it larger when a call
needs more (and says so in its log), the operator keeps one window per device
and stream, grows it (never shrinks it) when a larger shape arrives, logs the
growth, and rebuilds the chunked plans that borrowed the old one.  Calls on
one stream share its window in stream order; other streams get windows of
their own.

``norm_all_to_all_4D`` is the same entry point with an RMS norm on the
head-complete side: before the exchange in mode 0 (query and key norms), after
it in mode 1 (a sub-layer norm, with the residual's addition), each in one
launch forward and one or two backward.  ``checkpoint`` keeps what the backward
pass needs of the activations in 8 bits, a little over half a 2-byte type.

``rope_all_to_all_4D`` is the same entry point with rotary positions, in one
launch either way, and ``window_attention`` the attention of what mode 0
gathers, over a sliding window and sinks; both have gradients.

Both caches are bounded: at most ``MAX_PLANS`` plans and ``MAX_WINDOWS``
windows are kept, the least recently used going first (a window's plans go
with it).  A dropped window returns to torch's allocator in its own stream's
order, after the work already queued there.  One lock covers the lookup and
the enqueue of each call, so a plan is never closed while another thread is
between finding it and launching on it.
"""
from __future__ import annotations

import logging
import threading
from collections import OrderedDict
from typing import Optional, Tuple

import torch

from . import Plan, Rotary

MAX_PLANS = 64
MAX_WINDOWS = 8

_log = logging.getLogger(__name__)
_plans: "OrderedDict" = OrderedDict()     # key -> Plan, least recently used first
_windows: "OrderedDict" = OrderedDict()   # (device, stream id) -> uint8 window of chunked exchanges
_lock = threading.Lock()


def _drop_plans_of(win) -> None:
    for k in [k for k, p in _plans.items() if p.window is win]:
        _plans.pop(k).close()


def _window_for(device, stream, nbytes: int):
    """The stream's window, grown to at least nbytes; growing closes the plans
    that borrowed the old one (caller holds _lock)."""
    key = (device, stream.stream_id)
    win = _windows.get(key)
    if win is not None and win.numel() >= nbytes:
        _windows.move_to_end(key)
        return win
    if win is not None:
        _drop_plans_of(win)
        _log.info("ua2a: chunked window of %s stream %d grown from %d to %d bytes",
                  device, stream.stream_id, win.numel(), nbytes)
    else:
        _log.info("ua2a: chunked window of %s stream %d created with %d bytes",
                  device, stream.stream_id, nbytes)
    # the old window is released to torch's allocator in this stream's order
    win = torch.empty(nbytes, dtype=torch.uint8, device=device)
    _windows[key] = win
    _windows.move_to_end(key)
    while len(_windows) > MAX_WINDOWS:
        _, old = _windows.popitem(last=False)
        _drop_plans_of(old)
    return win


def _plan_for(w: int, B: int, S_local: int, H: int, D: int, dtype, device,
              chunked: bool = False) -> Plan:
    """One cached plan per shape, dtype and device (plans are small host
    objects); chunked plans per stream too, each borrowing its stream's
    window (caller holds _lock)."""
    window = None
    key = (w, B, S_local, H, D, dtype, device)
    if chunked:
        stream = torch.cuda.current_stream(device)
        e = torch.empty((), dtype=dtype).element_size()
        need = Plan.window_bytes(w, B, S_local, H, D, e)
        window = _window_for(device, stream, need)
        key += (stream.stream_id,)
    plan = _plans.get(key)
    if plan is None:
        plan = Plan(w, B, S_local, H, D, dtype, window=window, device=device)
        _plans[key] = plan
        while len(_plans) > MAX_PLANS:
            _plans.popitem(last=False)[1].close()
    else:
        _plans.move_to_end(key)
    return plan


def _local_shape(shape, w: int, mode: int):
    """(B, S_local, H, D) of a rank-stacked input of the given mode."""
    if len(shape) != 5 or shape[0] != w:
        raise ValueError(f"expected a rank-stacked [w={w}, B, S, H, D] tensor, got {tuple(shape)}")
    _, B, S, Hx, D = shape
    if mode == 0:
        return B, S, Hx, D
    if S % w:
        raise ValueError(f"mode 1 needs S_global = {S} divisible by w = {w}")
    return B, S // w, Hx * w, D


def _out_shape(shape, w: int, mode: int):
    B, S, H, D = _local_shape(shape, w, mode)
    if H % w:
        raise ValueError(f"H = {H} is not divisible by w = {w}")
    return (w, B, S * w, H // w, D) if mode == 0 else (w, B, S, H, D)


@torch.library.custom_op("ua2a::exchange", mutates_args=())
def exchange(x: torch.Tensor, w: int, mode: int, chunked: bool = False) -> torch.Tensor:
    """Rank-stacked Ulysses exchange on the GPU (mode 0 or 1); returns a new tensor."""
    if mode not in (0, 1):
        raise ValueError("mode must be 0 or 1")
    if x.device.type != "cuda":
        raise RuntimeError(f"the exchange runs on the GPU only (got a {x.device.type} tensor)")
    B, S, H, D = _local_shape(x.shape, w, mode)
    x = x.contiguous()
    with _lock:
        plan = _plan_for(w, B, S, H, D, x.dtype, x.device, chunked)
        return plan.exchange(x, mode, chunked)


@exchange.register_fake
def _exchange_fake(x: torch.Tensor, w: int, mode: int, chunked: bool = False) -> torch.Tensor:
    return x.new_empty(_out_shape(x.shape, w, mode))


def _setup_context(ctx, inputs, output):
    _, w, mode, chunked = inputs
    ctx.w = w
    ctx.mode = mode
    ctx.chunked = chunked


def _backward(ctx, grad):
    # d(out)/d(in) is a permutation matrix; its transpose is the inverse exchange
    return exchange(grad.contiguous(), ctx.w, 1 - ctx.mode, ctx.chunked), None, None, None


exchange.register_autograd(_backward, setup_context=_setup_context)


def all_to_all_4D(x: torch.Tensor, scatter_dim: int, gather_dim: int, w: int,
                  chunked: bool = False) -> torch.Tensor:
    """The page's 4-D all-to-all on rank-stacked tensors ``[w, B, S, H, D]``.

    ``scatter_dim`` / ``gather_dim`` index one rank's ``[B, S, H, D]``: (2, 1)
    scatters heads and gathers the sequence (mode 0), (1, 2) is the inverse
    (mode 1).  Other pairs are not an exchange this operator implements.
    ``chunked`` moves one batch plane at a time through the stream's window.
    """
    if (scatter_dim, gather_dim) == (2, 1):
        mode = 0
    elif (scatter_dim, gather_dim) == (1, 2):
        mode = 1
    else:
        raise ValueError(f"unsupported (scatter_dim, gather_dim) = ({scatter_dim}, {gather_dim}); "
                         "use (2, 1) for heads -> sequence or (1, 2) for the inverse")
    return exchange(x, w, mode, chunked)


# ------------------------------------------------------- norms with the exchange

_FORMATS = {0: None, 1: torch.float8_e4m3fn, 2: torch.float8_e5m2}


def _format_code(dtype, what: str) -> int:
    for code, d in _FORMATS.items():
        if d == dtype:
            return code
    raise TypeError(f"{what} must be torch.float8_e4m3fn, torch.float8_e5m2 or None, not {dtype}")


def _norm_shapes(shape, w: int, mode: int, per_head: bool):
    """(P shape, out shape, rstd shape, blocks per head) of a norm's input shape."""
    out = _out_shape(shape, w, mode)
    p = tuple(shape) if mode == 0 else out
    return p, out, p[:4] if per_head else p[:3], -(-p[4] // 32)


@torch.library.custom_op("ua2a::norm_exchange", mutates_args=())
def norm_exchange(x: torch.Tensor, weight: Optional[torch.Tensor], residual: Optional[torch.Tensor], w: int, mode: int,
                  per_head: bool, eps: float, out_format: int, saved_format: int) -> Tuple[
                      torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor]:
    """RMS norm joined with the rank-stacked exchange on the GPU: (out, scales,
    sum, saved, saved_scales, rstd) as ``Plan.norm_exchange`` returns them,
    empty tensors for what the call does not have; formats 0 none, 1 e4m3, 2 e5m2."""
    if mode not in (0, 1):
        raise ValueError("mode must be 0 or 1")
    if x.device.type != "cuda":
        raise RuntimeError(f"the exchange runs on the GPU only (got a {x.device.type} tensor)")
    B, S, H, D = _local_shape(x.shape, w, mode)
    if residual is not None:
        residual = residual.contiguous()
    if weight is not None:
        weight = weight.contiguous()
    with _lock:
        plan = _plan_for(w, B, S, H, D, x.dtype, x.device)
        r = plan.norm_exchange(x.contiguous(), weight, mode, residual=residual, per_head=per_head, eps=eps,
                               out_dtype=_FORMATS[out_format], checkpoint=_FORMATS[saved_format], rstd=True)
    none = x.new_empty(0)
    return tuple(none.clone() if t is None else t for t in r)


@norm_exchange.register_fake
def _norm_exchange_fake(x, weight, residual, w, mode, per_head, eps, out_format, saved_format):
    p, out, stat, nb = _norm_shapes(x.shape, w, mode, per_head)
    e8 = torch.float8_e8m0fnu
    return (x.new_empty(out, dtype=_FORMATS[out_format] or x.dtype),
            x.new_empty(out[:-1] + (nb,), dtype=e8) if out_format else x.new_empty(0),
            x.new_empty(p) if residual is not None else x.new_empty(0),
            x.new_empty(p, dtype=_FORMATS[saved_format]) if saved_format else x.new_empty(0),
            x.new_empty(p[:-1] + (nb,), dtype=e8) if saved_format else x.new_empty(0),
            x.new_empty(stat, dtype=torch.float32))


@torch.library.custom_op("ua2a::norm_exchange_backward", mutates_args=())
def norm_exchange_backward(dy: torch.Tensor, weight: Optional[torch.Tensor], saved: torch.Tensor,
                           saved_scales: Optional[torch.Tensor], rstd: torch.Tensor, dsum: Optional[torch.Tensor], w: int,
                           mode: int, per_head: bool, residual: bool, dweight: bool) -> Tuple[
                               torch.Tensor, torch.Tensor, torch.Tensor]:
    """(dx, dresidual, dweight) as ``Plan.norm_exchange_backward`` returns them;
    dresidual is empty where it is dx (mode 0) or there is no residual."""
    B, S, H, D = _local_shape(dy.shape, w, 1 - mode)
    if dsum is not None:
        dsum = dsum.contiguous()
    if weight is not None:
        weight = weight.contiguous()
    with _lock:
        plan = _plan_for(w, B, S, H, D, dy.dtype, dy.device)
        r = plan.norm_exchange_backward(dy.contiguous(), weight, mode, saved.contiguous(), rstd,
                                        saved_scales=saved_scales, dsum=dsum, residual=residual, per_head=per_head,
                                        dweight=dweight)
    none = dy.new_empty(0)
    return (r.dx, r.dresidual if residual and mode == 1 else none, none.clone() if r.dweight is None else r.dweight)


@norm_exchange_backward.register_fake
def _norm_exchange_backward_fake(dy, weight, saved, saved_scales, rstd, dsum, w, mode, per_head, residual, dweight):
    x = _out_shape(dy.shape, w, 1 - mode)
    return (dy.new_empty(x), dy.new_empty(tuple(dy.shape)) if residual and mode == 1 else dy.new_empty(0),
            dy.new_empty(weight.shape, dtype=torch.float32) if weight is not None and dweight else dy.new_empty(0))


def _norm_setup_context(ctx, inputs, output):
    x, weight, residual, w, mode, per_head, eps, out_format, saved_format = inputs
    out, scales, total, saved, saved_scales, rstd = output
    ctx.mark_non_differentiable(scales, saved, saved_scales, rstd)
    ctx.set_materialize_grads(False)
    ctx.args = (w, mode, per_head, residual is not None)
    ctx.weight = weight is not None
    if saved_format:
        kept = (saved, saved_scales)
    else:
        kept = (x if residual is None else total, None)
    ctx.save_for_backward(weight, *kept, rstd)


def _norm_backward(ctx, g_out, g_scales, g_sum, g_saved, g_saved_scales, g_rstd):
    weight, saved, saved_scales, rstd = ctx.saved_tensors
    w, mode, per_head, residual = ctx.args
    if g_out is None:
        if g_sum is None:
            return (None,) * 9
        # only the sum is used: the norm adds nothing, whatever its values are
        needs = ctx.needs_input_grad
        dx = None if not needs[0] else g_sum if mode == 0 else exchange(g_sum.contiguous(), w, 0)
        dw = torch.zeros_like(weight) if ctx.weight and needs[1] else None
        return dx, dw, g_sum if needs[2] else None, None, None, None, None, None, None
    dx, dres, dw = norm_exchange_backward(g_out, weight, saved, saved_scales, rstd, g_sum, w, mode, per_head, residual,
                                          ctx.weight and ctx.needs_input_grad[1])
    dres = (dx if mode == 0 else dres) if residual and ctx.needs_input_grad[2] else None
    dw = dw.to(weight.dtype) if ctx.weight and ctx.needs_input_grad[1] else None
    return dx, dw, dres, None, None, None, None, None, None


norm_exchange.register_autograd(_norm_backward, setup_context=_norm_setup_context)


def norm_all_to_all_4D(x: torch.Tensor, weight: Optional[torch.Tensor], scatter_dim: int, gather_dim: int, w: int,
                       residual: Optional[torch.Tensor] = None, per_head: bool = False, eps: float = 1e-6,
                       checkpoint=None, out_dtype=None):
    """``all_to_all_4D`` with an RMS norm on the head-complete side, in one launch.

    (2, 1): the norm of ``x`` (+ ``residual``), then heads scattered and the
    sequence gathered; (1, 2): the inverse exchange of ``x`` (+ ``residual``),
    then the norm.  ``weight``: one value per head value, [H*D], or with
    ``per_head`` one norm per head and [D]; of x's dtype or float32, None for
    ones.  ``residual`` is head-complete, ``[w, B, S_local, H, D]``.

    Returns out, with a residual (out, sum): the sum that was normed, in x's
    dtype.  ``out_dtype`` (torch.float8_e4m3fn or e5m2) makes out a pair (codes,
    scales) with one power-of-two scale per 32 values along D; such a call has
    no gradient.  ``checkpoint`` (the same dtypes) keeps 8 bits of what was
    normed for the backward pass in place of the values: its gradients are those
    of the norm at the values that the 8 bits stand for, with the exact rstd.
    """
    if (scatter_dim, gather_dim) == (2, 1):
        mode = 0
    elif (scatter_dim, gather_dim) == (1, 2):
        mode = 1
    else:
        raise ValueError(f"unsupported (scatter_dim, gather_dim) = ({scatter_dim}, {gather_dim}); "
                         "use (2, 1) for heads -> sequence or (1, 2) for the inverse")
    out_format, saved_format = _format_code(out_dtype, "out_dtype"), _format_code(checkpoint, "checkpoint")
    wants = torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in (x, weight, residual))
    if out_format and wants:
        raise ValueError("an 8-bit result has no gradient: call it under torch.no_grad()")
    if not wants:
        saved_format = 0                                   # nothing to keep
    p, _, _, _ = _norm_shapes(x.shape, w, mode, per_head)
    if residual is not None and tuple(residual.shape) != p:
        raise ValueError(f"residual has shape {tuple(residual.shape)}, expected {p}")
    if residual is not None and residual.dtype != x.dtype:
        raise TypeError(f"residual has dtype {residual.dtype}, x has {x.dtype}")
    n = p[4] if per_head else p[3] * p[4]
    if weight is not None and tuple(weight.shape) != (n,):
        raise ValueError(f"weight has shape {tuple(weight.shape)}, expected {(n,)}")
    out, scales, total, _, _, _ = norm_exchange(x, weight, residual, w, mode, per_head, eps, out_format, saved_format)
    if out_format:
        out = (out, scales)
    return out if residual is None else (out, total)


# ------------------------------------------------- rotary positions, attention


def _rotary(D: int, turns, axes, naxes: int, halves: bool) -> Rotary:
    """The Rotary that an operator's tensors are of."""
    r = Rotary.__new__(Rotary)
    r.D, r.pairs, r.naxes, r.halves = D, turns.numel(), naxes, halves
    r.turns, r.axes, r.device = turns, axes, turns.device
    return r


@torch.library.custom_op("ua2a::rope_exchange", mutates_args=())
def rope_exchange(x: torch.Tensor, positions: torch.Tensor, turns: torch.Tensor, axes: torch.Tensor, w: int, mode: int,
                  naxes: int, halves: bool, inverse: bool) -> torch.Tensor:
    """Rotary positions joined with the rank-stacked exchange on the GPU, as
    ``Plan.rope_exchange``; turns, axes, naxes and halves are a Rotary's."""
    if mode not in (0, 1):
        raise ValueError("mode must be 0 or 1")
    if x.device.type != "cuda":
        raise RuntimeError(f"the exchange runs on the GPU only (got a {x.device.type} tensor)")
    B, S, H, D = _local_shape(x.shape, w, mode)
    with _lock:
        plan = _plan_for(w, B, S, H, D, x.dtype, x.device)
        return plan.rope_exchange(x.contiguous(), _rotary(D, turns, axes, naxes, halves), positions.contiguous(), mode, inverse)


@rope_exchange.register_fake
def _rope_exchange_fake(x, positions, turns, axes, w, mode, naxes, halves, inverse):
    return x.new_empty(_out_shape(x.shape, w, mode))


def _rope_setup_context(ctx, inputs, output):
    _, positions, turns, axes, w, mode, naxes, halves, inverse = inputs
    ctx.save_for_backward(positions, turns, axes)
    ctx.args = (w, mode, naxes, halves, inverse)


def _rope_backward(ctx, grad):
    # a rotation's transpose turns the other way, an exchange's is its inverse
    positions, turns, axes = ctx.saved_tensors
    w, mode, naxes, halves, inverse = ctx.args
    dx = rope_exchange(grad.contiguous(), positions, turns, axes, w, 1 - mode, naxes, halves, not inverse)
    return dx, None, None, None, None, None, None, None, None


rope_exchange.register_autograd(_rope_backward, setup_context=_rope_setup_context)


def rope_all_to_all_4D(x: torch.Tensor, rotary: Rotary, positions: torch.Tensor, scatter_dim: int, gather_dim: int, w: int,
                       inverse: bool = False) -> torch.Tensor:
    """``all_to_all_4D`` with rotary positions, in one launch.

    ``rotary``: a :class:`Rotary`.  ``positions``: int32 ``[axes, S_local*w]``
    or ``[axes, B, S_local*w]``, tokens in gathered order.  ``inverse`` turns
    the other way.  The gradient of x is the same call the other way round.
    """
    if (scatter_dim, gather_dim) == (2, 1):
        mode = 0
    elif (scatter_dim, gather_dim) == (1, 2):
        mode = 1
    else:
        raise ValueError(f"unsupported (scatter_dim, gather_dim) = ({scatter_dim}, {gather_dim}); "
                         "use (2, 1) for heads -> sequence or (1, 2) for the inverse")
    if rotary.D != x.shape[-1]:
        raise ValueError(f"rotary is for heads of {rotary.D}, x has {x.shape[-1]}")
    return rope_exchange(x, positions, rotary.turns, rotary.axes, w, mode, rotary.naxes, rotary.halves, inverse)


def _attention_plan(q, k, w: int) -> Plan:
    """The plan of gathered queries ``[w, B, S, heads, D]`` (caller holds _lock)."""
    if q.device.type != "cuda":
        raise RuntimeError(f"attention runs on the GPU only (got a {q.device.type} tensor)")
    B, S, H, D = _local_shape(q.shape, w, 1)
    return _plan_for(w, B, S, H, D, q.dtype, q.device)


@torch.library.custom_op("ua2a::window_attention", mutates_args=())
def _window_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, counts: Optional[torch.Tensor], w: int,
                      left: Optional[int], right: Optional[int], sinks: int, chunk: int, scale: Optional[float],
                      lse: bool) -> Tuple[torch.Tensor, torch.Tensor]:
    """(out, lse) of ``Plan.window_attention``; lse is empty where it is not asked for."""
    with _lock:
        plan = _attention_plan(q, k, w)
        r = plan.window_attention(q.contiguous(), k.contiguous(), v.contiguous(), left=left, right=right, sinks=sinks,
                                  chunk=chunk, counts=None if counts is None else counts.contiguous(), scale=scale, lse=lse)
    return r.out, r.lse if lse else q.new_empty(0, dtype=torch.float32)


@_window_attention.register_fake
def _window_attention_fake(q, k, v, counts, w, left, right, sinks, chunk, scale, lse):
    _, B, SG, hl, _ = q.shape
    return (torch.empty_like(q, memory_format=torch.contiguous_format),
            q.new_empty((w, B, hl, SG) if lse else (0,), dtype=torch.float32))


@torch.library.custom_op("ua2a::window_attention_backward", mutates_args=())
def _window_attention_grads(dout: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: torch.Tensor,
                            lse: torch.Tensor, counts: Optional[torch.Tensor], w: int, left: Optional[int],
                            right: Optional[int], sinks: int, chunk: int, scale: Optional[float]) -> Tuple[
                                torch.Tensor, torch.Tensor, torch.Tensor]:
    """(dq, dk, dv) of ``Plan.window_attention_backward``."""
    with _lock:
        plan = _attention_plan(q, k, w)
        r = plan.window_attention_backward(dout.contiguous(), q.contiguous(), k.contiguous(), v.contiguous(), out, lse,
                                           left=left, right=right, sinks=sinks, chunk=chunk, scale=scale,
                                           counts=None if counts is None else counts.contiguous())
    return r.dq, r.dk, r.dv


@_window_attention_grads.register_fake
def _window_attention_grads_fake(dout, q, k, v, out, lse, counts, w, left, right, sinks, chunk, scale):
    return tuple(torch.empty_like(t, memory_format=torch.contiguous_format) for t in (q, k, v))


def _attention_setup_context(ctx, inputs, output):
    q, k, v, counts, w, left, right, sinks, chunk, scale, lse = inputs
    out, stats = output
    ctx.mark_non_differentiable(stats)
    ctx.set_materialize_grads(False)
    ctx.args = (w, left, right, sinks, chunk, scale)
    ctx.has = lse
    ctx.save_for_backward(q, k, v, out, stats, counts)


def _attention_backward(ctx, g_out, g_stats):
    if g_out is None:
        return (None,) * 11
    if not ctx.has:
        raise RuntimeError("a call without lse has no gradient")
    q, k, v, out, stats, counts = ctx.saved_tensors
    dq, dk, dv = _window_attention_grads(g_out, q, k, v, out, stats, counts, *ctx.args)
    needs = ctx.needs_input_grad
    return (dq if needs[0] else None, dk if needs[1] else None, dv if needs[2] else None) + (None,) * 8


_window_attention.register_autograd(_attention_backward, setup_context=_attention_setup_context)


def window_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, w: int, left: Optional[int] = None,
                     right: Optional[int] = None, sinks: int = 0, chunk: int = 1, counts: Optional[torch.Tensor] = None,
                     scale: Optional[float] = None) -> torch.Tensor:
    """softmax(scale q k^T) v of gathered heads ``[w, B, S, heads, D]`` (what mode 0
    gives), over a sliding window and sinks; k and v may have fewer heads.

    A query at position p sees, with c(x) = x // chunk, the positions j with
    ``c(p) - left <= c(j) <= c(p) + right`` (None: no bound) and the first
    ``sinks``; with ``right=0`` nothing past its own chunk.  ``counts``: int32
    ``[B]`` on the device, the tokens of each plane's sequences; the rest is
    padding, whose rows and gradients are zeros.  bfloat16 and float16, D a
    multiple of 8 up to 128.  q, k and v have gradients.
    """
    wants = torch.is_grad_enabled() and any(t.requires_grad for t in (q, k, v))
    out, _ = _window_attention(q, k, v, counts, w, left, right, sinks, chunk, scale, wants)
    return out
