"""Python binding of the activation operators (include/ua2a_act.h): RMS norms
joined with the exchange, forward and backward, and the 8-bit key/value cache.

Argument marshalling only, like the package's binding of the exchange: the
HIP kernels in libua2a.so do the work.  The calls are methods of ``Plan``.

8-bit tensors come as two: codes (``torch.float8_e4m3fn`` or
``torch.float8_e5m2``), shaped like the values, and scales
(``torch.float8_e8m0fnu``, powers of two), one per block of 32 values along
the last axis -- the same shape with D replaced by ceil(D / 32), so both are
tensors of the exchange's layouts themselves.
"""
from __future__ import annotations

import ctypes
import sys
from typing import NamedTuple, Optional

from . import UA2A_ERR_DEVICE, UA2A_OK, UA2AError

_pkg = sys.modules[__package__]      # its functions are looked up when they are called

UA2A_BLOCK = 32          # values that share a scale

EXPORTED = (
    "ua2a_norm_exchange", "ua2a_norm_exchange_backward", "ua2a_norm_workspace",
    "ua2a_cache_write", "ua2a_cache_read",
)


class ua2a_norm_t(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_void_p) for n in (
        "x", "residual", "weight", "out", "out_scales", "sum", "saved", "saved_scales", "rstd")]
        + [("eps", ctypes.c_float)]
        + [(n, ctypes.c_int32) for n in ("type", "weight_type", "per_head", "out_format", "saved_format")])


class ua2a_norm_grad_t(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_void_p) for n in (
        "dy", "dsum", "saved", "saved_scales", "weight", "rstd", "dx", "dresidual", "dweight", "workspace")]
        + [("workspace_bytes", ctypes.c_int64)]
        + [(n, ctypes.c_int32) for n in ("type", "weight_type", "per_head", "saved_format", "saved_gathered")])


class ua2a_cache_t(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("sequences", ctypes.c_int64),
                ("capacity", ctypes.c_int64), ("format", ctypes.c_int32)]


def declare_activation_signatures(lib: ctypes.CDLL) -> ctypes.CDLL:
    """Set ctypes argument/return types of the activation operators on a loaded library."""
    i32, i64, vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p
    sig = {
        "ua2a_norm_exchange": [vp, i32, ctypes.POINTER(ua2a_norm_t), vp],
        "ua2a_norm_exchange_backward": [vp, i32, ctypes.POINTER(ua2a_norm_grad_t), vp],
        "ua2a_norm_workspace": [vp, i32, ctypes.POINTER(i64)],
        "ua2a_cache_write": [vp, ctypes.POINTER(ua2a_cache_t), i32, vp, vp, vp, vp, vp],
        "ua2a_cache_read": [vp, ctypes.POINTER(ua2a_cache_t), i32, i64, vp, vp, vp, vp, vp],
    }
    for name, argtypes in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = argtypes
        fn.restype = ctypes.c_int
    return lib


class NormExchange(NamedTuple):
    """Results of ``Plan.norm_exchange``; what was not asked for is None."""
    out: object                       # in the type, or codes
    scales: Optional[object] = None   # of out's codes
    sum: Optional[object] = None      # x + residual, P layout
    saved: Optional[object] = None    # checkpoint: codes of what was normed, P layout
    saved_scales: Optional[object] = None
    rstd: Optional[object] = None     # [w, B, S_local], per head [w, B, S_local, H]


class NormGradients(NamedTuple):
    """Results of ``Plan.norm_exchange_backward``."""
    dx: object
    dresidual: Optional[object] = None   # mode 0: dx itself
    dweight: Optional[object] = None     # fp32


_tables = None


def _types():
    """(element type codes, 8-bit format codes) by torch dtype."""
    global _tables
    if _tables is None:
        import torch
        _tables = ({torch.bfloat16: 0, torch.float16: 1, torch.float32: 2},
                   {torch.float8_e4m3fn: 1, torch.float8_e5m2: 2})
    return _tables


def _format_of(dtype, what: str) -> int:
    """The 8-bit format code of a torch dtype (0 for None)."""
    if dtype is None:
        return 0
    f = _types()[1].get(dtype)
    if f is None:
        raise TypeError(f"{what} must be torch.float8_e4m3fn or torch.float8_e5m2, not {dtype}")
    return f


def _ptr(t):
    return None if t is None else t.data_ptr()


def _blocks(D: int) -> int:
    return -(-D // UA2A_BLOCK)


class Cache:
    """An 8-bit key/value cache of sequence-gathered heads.

    ``codes`` ``[2, w, sequences, capacity, H/w, D]`` and ``scales``
    ``[2, w, sequences, capacity, H/w, ceil(D/32)]``, keys first, then values.
    A new cache holds zeros.  ``Plan.cache_write`` fills it and
    ``Plan.cache_read`` reads it back; ``Cache.of`` takes tensors that the
    caller has.
    """

    def __init__(self, w: int, H: int, D: int, sequences: int, capacity: int, dtype=None, device=None):
        import torch
        dtype = torch.float8_e4m3fn if dtype is None else dtype
        _format_of(dtype, "a cache's dtype")
        if min(w, H, D, sequences, capacity) < 1 or H % w:
            raise ValueError("a cache needs sizes of at least 1 and H divisible by w")
        lead = (2, w, sequences, capacity, H // w)
        device = torch.device("cuda") if device is None else device
        self._set(torch.zeros(lead + (D,), dtype=torch.uint8, device=device).view(dtype),
                  torch.zeros(lead + (_blocks(D),), dtype=torch.uint8, device=device).view(torch.float8_e8m0fnu))

    @classmethod
    def of(cls, codes, scales) -> "Cache":
        """A cache over the caller's tensors (contiguous, shaped as above)."""
        cache = cls.__new__(cls)
        cache._set(codes, scales)
        return cache

    @staticmethod
    def _check(codes, scales) -> None:
        import torch
        _format_of(codes.dtype, "a cache's codes")
        if scales.dtype not in (torch.float8_e8m0fnu, torch.uint8):
            raise TypeError(f"a cache's scales must be torch.float8_e8m0fnu (or uint8), not {scales.dtype}")
        if codes.dim() != 6 or codes.shape[0] != 2:
            raise ValueError(f"codes must be [2, w, sequences, capacity, H/w, D], got {tuple(codes.shape)}")
        if tuple(scales.shape) != tuple(codes.shape[:-1]) + (_blocks(codes.shape[-1]),):
            raise ValueError(f"scales have shape {tuple(scales.shape)}, codes {tuple(codes.shape)}")
        if scales.device != codes.device:
            raise ValueError(f"scales are on {scales.device}, codes are on {codes.device}")
        if not (codes.is_contiguous() and scales.is_contiguous()):
            raise ValueError("codes and scales must be contiguous")
        for t, what in ((codes, "codes"), (scales, "scales")):
            if t.untyped_storage().nbytes() < t.storage_offset() + t.numel():
                raise ValueError(f"{what} have lost their memory")

    @property
    def codes(self):
        return self._codes

    @property
    def scales(self):
        return self._scales

    def _set(self, codes, scales) -> None:
        import torch
        self._check(codes, scales)
        self._codes, self._scales = codes, scales
        self.device, self.int32 = codes.device, torch.int32
        _, self.w, self.sequences, self.capacity, self.heads, self.D = codes.shape
        self.per_sequence = (self.sequences,)
        self.heads_of = (self.w, self.heads * self.w, self.D)
        self._codes_at, self._scales_at = codes.data_ptr(), scales.data_ptr()
        self._ref = ctypes.byref(ua2a_cache_t(self._codes_at, self._scales_at, self.sequences, self.capacity,
                                              _format_of(codes.dtype, "codes")))


class ActivationCalls:
    """The activation operators as methods of ``Plan`` (its shape, type and device)."""

    def _type(self) -> int:
        t = _types()[0].get(self.dtype)
        if t is None:
            raise TypeError(f"norms and caches take bfloat16, float16 and float32 plans, not {self.dtype}")
        return t

    def _expect(self, t, dtype, shape, what):
        """An argument or a reused buffer of the given type and shape on the plan's device."""
        if t is None:
            raise ValueError(f"{what} is missing")
        if t.dtype != dtype:
            raise TypeError(f"{what} has dtype {t.dtype}, expected {dtype}")
        if t.device != self.device:
            raise ValueError(f"{what} is on {t.device}, plan is on {self.device}")
        if t.shape != shape:
            raise ValueError(f"{what} has shape {tuple(t.shape)}, expected {tuple(shape)}")
        if not t.is_contiguous():
            raise ValueError(f"{what} must be contiguous")
        return t

    def _weight(self, weight, per_head: bool) -> int:
        """Checks a norm's weight and returns its type code."""
        if weight is None:
            return 0
        n = self.D if per_head else self.H * self.D
        code = _types()[0].get(weight.dtype)
        if code is None or (code != 2 and weight.dtype is not self.dtype):
            raise TypeError(f"weight has dtype {weight.dtype}, expected {self.dtype} or float32")
        if not self._fits(weight, weight.dtype, (n,)):
            self._expect(weight, weight.dtype, (n,), "weight")
        return code

    def _rstd_shape(self, per_head: bool):
        lead = (self.w, self.B, self.S_local)
        return lead + (self.H,) if per_head else lead

    def _fits(self, t, dtype, shape) -> bool:
        """Whether t is a contiguous tensor of the given type and shape on the plan's device."""
        return t.shape == shape and t.dtype is dtype and t.device == self.device and t.is_contiguous()

    def _issue(self, name: str, stream, *args) -> None:
        """The library's `name`(handle, *args, stream) on `stream` (None: torch's
        current one), with the plan's device current."""
        sptr = (_pkg._current_raw_stream(self.device) if stream is None else stream.cuda_stream) or None
        handle = self.handle
        fn = getattr(_pkg._lib or _pkg.load_library(), name)
        rc = fn(handle, *args, sptr)
        if rc == UA2A_OK:
            return
        if rc == UA2A_ERR_DEVICE and handle:
            # another device is current: the library changed nothing; retry on the plan's
            import torch
            with torch.cuda.device(self.device):
                rc = fn(handle, *args, sptr)
        if rc != UA2A_OK:
            raise UA2AError(rc, name, _pkg.ua2a_plan_last_error(handle) if handle else "")

    def _norm_spec(self, mode, per_head, out_dtype, checkpoint, rstd, residual):
        """What a kind of norm_exchange call takes and gives, worked out once:
        (type code, format codes, x's shape, P shape, ((dtype, shape) or None)
        of each result)."""
        specs = self.__dict__.setdefault("_norm_specs", {})
        key = (mode, per_head, out_dtype, checkpoint, rstd, residual)
        spec = specs.get(key)
        if spec is None:
            import torch
            code = self._type()
            if mode not in (0, 1):
                raise ValueError("mode must be 0 or 1")
            ofmt, sfmt = _format_of(out_dtype, "out_dtype"), _format_of(checkpoint, "checkpoint")
            p, oshape, nb = self.in_shape(0), self.out_shape(mode), (_blocks(self.D),)
            e8 = torch.float8_e8m0fnu
            want = ((self.dtype if out_dtype is None else out_dtype, oshape),
                    (e8, oshape[:-1] + nb) if ofmt else None,
                    (self.dtype, p) if residual else None,
                    (checkpoint, p) if sfmt else None,
                    (e8, p[:-1] + nb) if sfmt else None,
                    (torch.float32, self._rstd_shape(per_head)) if rstd or sfmt else None)
            spec = specs[key] = (code, ofmt, sfmt, self.in_shape(mode), p, want)
        return spec

    def _on_stream(self, stream):
        """Allocations inside belong to `stream`, so that torch reuses their memory
        only in its order."""
        import contextlib
        import torch
        return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)

    def norm_exchange(self, x, weight, mode: int, *, residual=None, per_head: bool = False, eps: float = 1e-6,
                      out_dtype=None, checkpoint=None, rstd: bool = False, out: Optional[NormExchange] = None,
                      stream=None) -> NormExchange:
        """RMS norm joined with the exchange, in one launch.

        mode 0: ``x`` in P layout; the norm of ``x`` (+ ``residual``), exchanged to A layout.
        mode 1: ``x`` in A layout; exchanged to P layout (+ ``residual``), then normed.

        The norm covers a token's H*D values, or each head's D with ``per_head``;
        ``weight`` has as many (the plan's dtype or float32; None: ones).
        With a ``residual`` (P layout) the sum, rounded to the plan's dtype, is
        what is normed, and is returned.  ``out_dtype`` (a float8 dtype) gives
        the result as codes and scales.  ``checkpoint`` (a float8 dtype) also
        returns what was normed in 8 bits, and rstd: all that
        ``norm_exchange_backward`` needs; ``rstd=True`` returns rstd alone.
        ``out``: an earlier result whose tensors are written again.
        """
        per_head = bool(per_head)
        code, ofmt, sfmt, xshape, p, want = self._norm_spec(mode, per_head, out_dtype, checkpoint, bool(rstd),
                                                            residual is not None)
        if not self._fits(x, self.dtype, xshape):
            self._check(x, xshape, "input")
        if residual is not None and not self._fits(residual, self.dtype, p):
            self._check(residual, p, "residual")
        wcode = self._weight(weight, per_head) if weight is not None else 0
        if out is None:
            import torch
            with self._on_stream(stream):
                out = NormExchange(*(None if q is None else torch.empty(q[1], dtype=q[0], device=self.device)
                                     for q in want))
        else:
            for name, t, q in zip(NormExchange._fields, out, want):
                if q is not None and (t is None or not self._fits(t, q[0], q[1])):
                    self._expect(t, q[0], q[1], f"out.{name}")
            out = NormExchange(*[t if q is not None else None for t, q in zip(out, want)])
        args = ua2a_norm_t(x.data_ptr(), _ptr(residual), _ptr(weight), *[None if t is None else t.data_ptr() for t in out],
                           eps, code, wcode, per_head, ofmt, sfmt)
        self._issue("ua2a_norm_exchange", stream, mode, ctypes.byref(args))
        return out

    def norm_exchange_backward(self, dy, weight, mode: int, saved, rstd, *, saved_scales=None, dsum=None,
                               residual: bool = False, per_head: bool = False, dweight: bool = True,
                               out: Optional[NormGradients] = None, stream=None) -> NormGradients:
        """Gradients of ``norm_exchange(mode)``.

        ``dy``: gradient of its out.  ``saved``: the checkpoint's codes with
        ``saved_scales``, or what was normed itself: the forward call's
        ``sum`` with a residual (``residual=True``), else its ``x``.  ``dsum``:
        gradient of the sum, with a residual.  Returns dx in x's layout, the
        residual's gradient in P layout (mode 0: dx itself) and the weight's in
        float32 (summed in a fixed order; None without a weight or with
        ``dweight=False``).  ``out``: an earlier result to write again.
        """
        import torch
        per_head = bool(per_head)
        code = self._type()
        if mode not in (0, 1):
            raise ValueError("mode must be 0 or 1")
        self._check(dy, self.out_shape(mode), "dy")
        p, xshape = self.in_shape(0), self.in_shape(mode)
        wcode = self._weight(weight, per_head)
        if dsum is not None:
            if not residual:
                raise ValueError("dsum is the gradient of a residual's sum: pass residual=True")
            self._check(dsum, p, "dsum")
        fmt = 0
        if saved_scales is not None:
            fmt = _format_of(saved.dtype, "saved")
            self._expect(saved, saved.dtype, p, "saved")
            if saved_scales.dtype not in (torch.float8_e8m0fnu, torch.uint8):
                raise TypeError(f"saved_scales must be torch.float8_e8m0fnu (or uint8), not {saved_scales.dtype}")
            self._expect(saved_scales, saved_scales.dtype, p[:-1] + (_blocks(self.D),), "saved_scales")
        else:
            self._check(saved, p if residual else xshape, "saved")
        self._expect(rstd, torch.float32, self._rstd_shape(per_head), "rstd")
        dweight = bool(dweight) and weight is not None
        wshape = (self.D if per_head else self.H * self.D,)
        apart = residual and mode == 1
        space, nspace = None, 0
        if dweight:
            spaces = self.__dict__.setdefault("_norm_workspace", {})
            nspace = spaces.get(per_head)
            if nspace is None:
                n = ctypes.c_int64()
                rc = _pkg.load_library().ua2a_norm_workspace(self.handle, per_head, ctypes.byref(n))
                if rc != UA2A_OK:
                    raise UA2AError(rc, "ua2a_norm_workspace")
                nspace = spaces[per_head] = n.value
        with self._on_stream(stream):
            if dweight:
                space = torch.empty(nspace, dtype=torch.uint8, device=self.device)
            if out is None:
                dx = torch.empty(xshape, dtype=self.dtype, device=self.device)
                dres = torch.empty(p, dtype=self.dtype, device=self.device) if apart else None
                dw = torch.empty(wshape, dtype=torch.float32, device=self.device) if dweight else None
            else:
                dx = self._expect(out.dx, self.dtype, xshape, "out.dx")
                dres = self._expect(out.dresidual, self.dtype, p, "out.dresidual") if apart else None
                dw = self._expect(out.dweight, torch.float32, wshape, "out.dweight") if dweight else None
        args = ua2a_norm_grad_t(dy.data_ptr(), _ptr(dsum), saved.data_ptr(), _ptr(saved_scales), _ptr(weight),
                                rstd.data_ptr(), dx.data_ptr(), _ptr(dres), _ptr(dw), _ptr(space), nspace, code, wcode,
                                per_head, fmt, int(mode == 1 and not residual and fmt == 0))
        self._issue("ua2a_norm_exchange_backward", stream, mode, ctypes.byref(args))
        return NormGradients(dx, dres if apart else dx if residual else None, dw)

    def _check_cache(self, cache: Cache, starts, counts) -> None:
        codes, scales = cache._codes, cache._scales
        if codes.data_ptr() != cache._codes_at or scales.data_ptr() != cache._scales_at:
            cache._set(codes, scales)                          # a tensor has been given other memory
        if cache.heads_of != (self.w, self.H, self.D):
            raise ValueError(f"cache has w = {cache.w}, {cache.heads} heads of {cache.D} per rank; "
                             f"the plan w = {self.w}, {self.H // self.w} of {self.D}")
        if cache.device != self.device:
            raise ValueError(f"cache is on {cache.device}, plan is on {self.device}")
        for t, what in ((starts, "starts"), (counts, "counts")):
            if t is not None and not self._fits(t, cache.int32, cache.per_sequence):
                self._expect(t, cache.int32, cache.per_sequence, what)

    def cache_write(self, cache: Cache, k, v, starts, counts=None, stream=None) -> Cache:
        """The mode-0 exchange of new keys and values (P layout; one may be
        None) straight into the cache, in 8 bits, one launch.

        The B * S_local*w gathered tokens are taken in order, n = B * S_local*w
        / sequences for each sequence; token t of sequence i goes to position
        ``starts[i] + t`` where ``t < counts[i]`` (None: all) and the position
        lies in the cache; other tokens are dropped, other positions keep what
        they hold.  ``starts``, ``counts``: int32 device tensors.
        """
        code = self._type()
        self._check_cache(cache, starts, counts)
        if k is None and v is None:
            raise ValueError("nothing to write: k and v are both None")
        if starts is None:
            raise ValueError("starts is missing")
        shape = (self.w, self.B, self.S_local, self.H, self.D)
        for t, what in ((k, "k"), (v, "v")):
            if t is not None and not self._fits(t, self.dtype, shape):
                self._check(t, shape, what)
        self._issue("ua2a_cache_write", stream, cache._ref, code, _ptr(k), _ptr(v), starts.data_ptr(), _ptr(counts))
        return cache

    def cache_read(self, cache: Cache, tokens: int, starts=None, counts=None, out=None, stream=None):
        """Positions ``starts[i] + t`` (None: from 0), t < ``tokens`` and
        ``counts[i]`` (None: all), of every sequence, back in the plan's dtype:
        (k, v), each ``[w, sequences, tokens, H/w, D]``, one launch.  Rows
        without a position are left as they were; without ``out`` they are
        zeros, which fills both results first (two launches more).  An entry
        of ``out`` that is None is not read.
        """
        code = self._type()
        self._check_cache(cache, starts, counts)
        if tokens < 1:
            raise ValueError(f"tokens must be at least 1, not {tokens}")
        shape = (self.w, cache.sequences, tokens, self.H // self.w, self.D)
        if out is None:
            import torch
            with self._on_stream(stream):
                out = tuple(torch.zeros(shape, dtype=self.dtype, device=self.device) for _ in range(2))
        else:
            if len(out) != 2 or (out[0] is None and out[1] is None):
                raise ValueError("out must be (k, v), one of which may be None")
            for t, what in zip(out, ("out[0]", "out[1]")):
                if t is not None and not self._fits(t, self.dtype, shape):
                    self._check(t, shape, what)
            out = tuple(out)
        self._issue("ua2a_cache_read", stream, cache._ref, code, tokens, _ptr(starts), _ptr(counts), _ptr(out[0]),
                    _ptr(out[1]))
        return out
