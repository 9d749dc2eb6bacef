"""Python binding of the attention block's operators (include/ua2a_attn.h):
rotary positions joined with the exchange, and attention with a sliding window
and sinks, of gathered heads, forward and backward, and over the 8-bit cache.

Argument marshalling only: the HIP kernels in libua2a.so do the work.  The
calls are methods of ``Plan``.

What a query at position p sees, with c(x) = x // chunk: the positions j with
``c(p) - left <= c(j) <= c(p) + right``, and the first ``sinks`` positions.
``None`` for left or right: no bound on that side.  With ``right=0`` (causal)
nothing past p's own chunk is seen, sinks or not.  ``chunk=1`` counts tokens;
a video's frames are chunks of as many tokens as a frame has.
"""
from __future__ import annotations

import ctypes
import sys
from typing import NamedTuple, Optional

from . import UA2A_OK, UA2AError
from .activations import _ptr, ua2a_cache_t

_pkg = sys.modules[__package__]      # its functions are looked up when they are called

EXPORTED = (
    "ua2a_rope", "ua2a_attention", "ua2a_attention_workspace", "ua2a_attention_backward",
    "ua2a_attention_backward_workspace", "ua2a_cache_attention", "ua2a_cache_attention_workspace",
)


class ua2a_rope_t(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_void_p) for n in ("x", "out", "positions", "turns", "axes")]
                + [(n, ctypes.c_int32) for n in (
                    "pairs", "naxes", "halves", "inverse", "per_plane", "from_", "to", "type")])


class ua2a_window_t(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("left", "right", "sinks", "chunk")]


_TAIL = [("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_int64), ("window", ua2a_window_t)]


class ua2a_attention_t(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_void_p) for n in ("q", "k", "v", "out", "lse", "counts")] + _TAIL
                + [("kv_heads", ctypes.c_int64), ("scale", ctypes.c_float), ("type", ctypes.c_int32)])


class ua2a_attention_grad_t(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_void_p) for n in (
        "dout", "q", "k", "v", "out", "lse", "dq", "dk", "dv", "counts")] + _TAIL
        + [("kv_heads", ctypes.c_int64), ("scale", ctypes.c_float), ("type", ctypes.c_int32)])


class ua2a_cache_attention_t(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_void_p) for n in ("q", "out", "starts", "counts")] + _TAIL
                + [("n", ctypes.c_int64), ("kv_heads", ctypes.c_int64), ("scale", ctypes.c_float),
                   ("type", ctypes.c_int32)])


def declare_attention_signatures(lib: ctypes.CDLL) -> ctypes.CDLL:
    """Set ctypes argument/return types of the attention operators on a loaded library."""
    vp, out, ptr = ctypes.c_void_p, ctypes.POINTER(ctypes.c_int64), ctypes.POINTER
    sig = {
        "ua2a_rope": [vp, ptr(ua2a_rope_t), vp],
        "ua2a_attention": [vp, ptr(ua2a_attention_t), vp],
        "ua2a_attention_workspace": [vp, ptr(ua2a_attention_t), out],
        "ua2a_attention_backward": [vp, ptr(ua2a_attention_grad_t), vp],
        "ua2a_attention_backward_workspace": [vp, ptr(ua2a_attention_grad_t), out],
        "ua2a_cache_attention": [vp, ptr(ua2a_cache_t), ptr(ua2a_cache_attention_t), vp],
        "ua2a_cache_attention_workspace": [vp, ptr(ua2a_cache_t), ptr(ua2a_cache_attention_t), out],
    }
    for name, argtypes in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = argtypes
        fn.restype = ctypes.c_int
    return lib


class Attention(NamedTuple):
    """Results of ``Plan.window_attention``."""
    out: object
    lse: Optional[object] = None      # [w, B, H/w, S_local*w], fp32, natural; -inf where a row sees nothing


class AttentionGradients(NamedTuple):
    """Results of ``Plan.window_attention_backward``."""
    dq: object
    dk: object
    dv: object


class Rotary:
    """Which values of a head turn with a token's position, and how fast.

    ``dims``: for each axis (time, height, width, ...) how many values of a head
    turn with its positions (even numbers, D together at most; the others stay
    as they are).  Axis a's pairs, in order, turn by ``theta ** (-2 i / dims[a])``
    radians per position.  Pairs are neighbours (2i, 2i + 1), or with ``halves``
    (i, i + sum(dims) / 2).  ``Rotary.of`` takes frequencies of the caller's own.

    Frequencies are held as 64-bit fractions of a turn, so an angle modulo a
    turn is good to 32 bits at any int32 position.  ``turns`` and ``axes`` are
    device tensors, made once.
    """

    def __init__(self, D: int, dims, theta: float = 10000.0, halves: bool = False, device=None):
        dims = tuple(int(d) for d in dims)
        if not dims or any(d < 0 or d % 2 for d in dims) or sum(dims) < 2 or sum(dims) > D:
            raise ValueError(f"dims must be even and {D} together at most (and some), got {dims}")
        if not (0.0 < theta < float("inf")):
            raise ValueError(f"theta must be positive and finite, not {theta}")
        freqs = [theta ** (-2.0 * i / d) for d in dims for i in range(d // 2)]
        axes = [a for a, d in enumerate(dims) for _ in range(d // 2)]
        self._set(D, freqs, axes, len(dims), halves, device)

    @classmethod
    def of(cls, D: int, frequencies, axes, halves: bool = False, device=None) -> "Rotary":
        """Pair i turns by ``frequencies[i]`` radians per position of axis
        ``axes[i]`` (sequences of numbers, read in double precision)."""
        rotary = cls.__new__(cls)
        freqs, axes = [float(f) for f in frequencies], [int(a) for a in axes]
        if not freqs or len(freqs) != len(axes) or 2 * len(freqs) > D:
            raise ValueError(f"expected as many axes as frequencies, at most {D // 2} (and some), got {len(freqs)} "
                             f"frequencies and {len(axes)} axes")
        if any(f != f or f in (float("inf"), float("-inf")) for f in freqs):
            raise ValueError("frequencies must be finite")
        if min(axes) < 0:
            raise ValueError("axes must be at least 0")
        rotary._set(D, freqs, axes, max(axes) + 1, halves, device)
        return rotary

    def _set(self, D, freqs, axes, naxes, halves, device):
        from fractions import Fraction
        import torch
        # 1 / (2 pi) to 2^-120: the quotient by 2 pi in integers, so that a turn's
        # fraction has the 53 bits that its frequency has
        inverse = Fraction(211553206025302378997855913028439351, 1 << 120)
        turns = [round(Fraction(f) * inverse * (1 << 64)) % (1 << 64) for f in freqs]
        turns = [t - (1 << 64) if t >= 1 << 63 else t for t in turns]     # the bits, as int64
        self.D, self.pairs, self.naxes, self.halves = D, len(freqs), naxes, bool(halves)
        device = torch.device("cuda") if device is None else torch.device(device)
        self.turns = torch.tensor(turns, dtype=torch.int64).to(device)
        self.axes = torch.tensor(axes, dtype=torch.int32).to(device)
        self.device = self.turns.device


def _bound(x, what: str) -> int:
    if x is None:
        return -1
    if x < 0:
        raise ValueError(f"{what} must be at least 0, or None for no bound, not {x}")
    return x


class AttentionCalls:
    """The attention block's operators as methods of ``Plan``."""

    # ------------------------------------------------------------------ rotary

    def _rope(self, x, rotary, positions, from_a, to_a, inverse, out, stream):
        specs = self.__dict__.setdefault("_rope_specs", {})
        spec = specs.get(rotary.naxes)
        if spec is None:
            import torch
            SG, a = self.S_local * self.w, rotary.naxes
            spec = specs[a] = (self._type(), (self.in_shape(0), self.out_shape(0)), (a, SG), (a, self.B, SG), torch.int32,
                               torch.int64)
        code, shapes, one, each, int32, int64 = spec
        if not self._fits(x, self.dtype, shapes[from_a]):
            self._check(x, shapes[from_a], "input")
        if rotary.D != self.D:
            raise ValueError(f"rotary is for heads of {rotary.D}, the plan has {self.D}")
        turns, axes, pairs = rotary.turns, rotary.axes, (rotary.pairs,)
        if not (self._fits(turns, int64, pairs) and self._fits(axes, int32, pairs)):
            self._expect(turns, int64, pairs, "rotary.turns")
            self._expect(axes, int32, pairs, "rotary.axes")
        planes = positions.dim() == 3
        if planes and positions.shape[1] == 1:
            positions, planes = positions[:, 0], False            # one plane for all
        if not self._fits(positions, int32, each if planes else one):
            self._expect(positions, int32, each if planes else one, "positions")
        if out is None:
            import torch
            with self._on_stream(stream):
                out = torch.empty(shapes[to_a], dtype=self.dtype, device=self.device)
        elif not self._fits(out, self.dtype, shapes[to_a]):
            self._check(out, shapes[to_a], "output")
        args = ua2a_rope_t(x.data_ptr(), out.data_ptr(), positions.data_ptr(), turns.data_ptr(), axes.data_ptr(),
                           rotary.pairs, rotary.naxes, rotary.halves, bool(inverse), planes, from_a, to_a, code)
        self._issue("ua2a_rope", stream, ctypes.byref(args))
        return out

    def rope_exchange(self, x, rotary: Rotary, positions, mode: int, inverse: bool = False, out=None, stream=None):
        """Rotary positions joined with the exchange, in one launch: ``x`` in P
        layout (mode 0) or A layout (mode 1), the result in the other.

        ``positions``: int32, ``[axes, S_local*w]`` for all planes or ``[axes,
        B, S_local*w]``, tokens in gathered order, any values.  ``inverse``
        turns the other way: ``rope_exchange(dy, rotary, positions, 1 - mode,
        inverse=True)`` is the gradient.
        """
        if mode not in (0, 1):
            raise ValueError("mode must be 0 or 1")
        return self._rope(x, rotary, positions, mode, 1 - mode, inverse, out, stream)

    def rope(self, x, rotary: Rotary, positions, gathered: bool = False, inverse: bool = False, out=None, stream=None):
        """The same within a layout: P, or A with ``gathered``.  ``out`` may be
        ``x`` itself (new keys before ``cache_write``)."""
        side = 1 if gathered else 0
        return self._rope(x, rotary, positions, side, side, inverse, out, stream)

    # --------------------------------------------------------------- attention

    def _attention_spec(self, kind, heads, sizes, left, right, sinks, chunk, scale):
        """What a kind of call needs, worked out once: (type code, window, scale, key
        heads on all ranks, bytes of scratch).  heads: key heads of a rank; sizes:
        (sequences, capacity, n) of a cache's call, else None."""
        specs = self.__dict__.setdefault("_attention_specs", {})
        if scale is not None:
            scale = float(scale)                               # a tensor's value may change from call to call
        left, right = (x if x is None else int(x) for x in (left, right))
        sinks, chunk = int(sinks), int(chunk)
        key = (kind, heads, sizes, left, right, sinks, chunk, scale)
        spec = specs.get(key)
        if spec is not None:
            return spec
        code = self._type()
        if code == 2:
            raise TypeError("attention takes bfloat16 and float16 plans, not float32")
        if self.D % 8 or self.D > 128:
            raise ValueError(f"attention takes heads of a multiple of 8 values up to 128, not {self.D}")
        if sinks < 0 or chunk < 1:
            raise ValueError(f"sinks must be at least 0 and chunk at least 1, not {sinks} and {chunk}")
        bounds = (_bound(left, "left"), _bound(right, "right"), sinks, chunk)
        if max(bounds) >= 1 << 31:
            raise ValueError(f"a window's sizes must be below 2^31, got {bounds}")
        scale = self.D ** -0.5 if scale is None else scale
        if not 1e-37 < scale < 1e38:
            raise ValueError(f"scale must be positive and finite (within 1e-37 and 1e38), not {scale}")
        if heads < 1 or (self.H // self.w) % heads:
            raise ValueError(f"{heads} key heads per rank do not divide the plan's {self.H // self.w}")
        window, kv, need = ua2a_window_t(*bounds), heads * self.w, ctypes.c_int64()
        lib = _pkg._lib or _pkg.load_library()
        if kind == "cache":
            cache = ua2a_cache_t(None, None, sizes[0], sizes[1], 1)
            args = ua2a_cache_attention_t(window=window, n=sizes[2], kv_heads=kv, scale=scale, type=code)
            rc = lib.ua2a_cache_attention_workspace(self.handle, ctypes.byref(cache), ctypes.byref(args), ctypes.byref(need))
        elif kind == "backward":
            args = ua2a_attention_grad_t(window=window, kv_heads=kv, scale=scale, type=code)
            rc = lib.ua2a_attention_backward_workspace(self.handle, ctypes.byref(args), ctypes.byref(need))
        else:
            args = ua2a_attention_t(window=window, kv_heads=kv, scale=scale, type=code)
            rc = lib.ua2a_attention_workspace(self.handle, ctypes.byref(args), ctypes.byref(need))
        if rc != UA2A_OK:
            raise UA2AError(rc, "ua2a_attention_workspace")
        if len(specs) >= 1024:
            specs.clear()
        spec = specs[key] = (code, window, scale, kv, need.value)
        return spec

    def _check_heads(self, q, k, v, counts):
        """Checks a call's tensors and returns the key heads of a rank."""
        gathered = self.__dict__.get("_gathered")
        if gathered is None:
            import torch
            gathered = self._gathered = (self.out_shape(0), torch.int32)
        shape, int32 = gathered
        if not self._fits(q, self.dtype, shape):
            self._check(q, shape, "q")
        if k.dim() != 5:
            raise ValueError(f"k must be [w, B, S_local*w, heads, D], got {tuple(k.shape)}")
        heads = k.shape[3]
        kshape = shape[:3] + (heads, shape[4])
        for t, what in ((k, "k"), (v, "v")):
            if not self._fits(t, self.dtype, kshape):
                self._check(t, kshape, what)
        if counts is not None and not self._fits(counts, int32, (self.B,)):
            self._expect(counts, int32, (self.B,), "counts")
        return heads

    def _space(self, need, stream):
        """Scratch of `need` bytes for a call, None for 0."""
        if need == 0:
            return None
        import torch
        with self._on_stream(stream):
            return torch.empty(need, dtype=torch.uint8, device=self.device)

    def window_attention(self, q, k, v, *, left=None, right=None, sinks: int = 0, chunk: int = 1, counts=None,
                         scale=None, lse: bool = False, out: Optional[Attention] = None, stream=None) -> Attention:
        """softmax(scale q k^T) v of gathered heads, over what the window shows.

        ``q``: A layout, ``[w, B, S_local*w, H/w, D]`` (what mode 0 gives);
        ``k``, ``v``: the same with any number of heads that divides H/w.
        ``counts``: int32 ``[B]`` on the device, the tokens of each plane's
        sequences; the rest is padding, which no query sees and whose rows are
        zeros.  ``scale``: default D ** -0.5.  ``lse``: also the rows'
        log-sum-exp, which ``window_attention_backward`` takes.  ``out``: an
        earlier result to write again.  bfloat16 and float16, D a multiple of 8
        up to 128.
        """
        heads = self._check_heads(q, k, v, counts)
        code, window, scale, kv, need = self._attention_spec("forward", heads, None, left, right, sinks, chunk, scale)
        if out is None or lse:
            import torch
            w, B, SG, hl, _ = self.out_shape(0)
            stats = (w, B, hl, SG)
        if out is None:
            with self._on_stream(stream):
                out = Attention(torch.empty(q.shape, dtype=self.dtype, device=self.device),
                                torch.empty(stats, dtype=torch.float32, device=self.device) if lse else None)
        else:
            if not self._fits(out.out, self.dtype, q.shape):
                self._check(out.out, q.shape, "out.out")
            if lse:
                self._expect(out.lse, torch.float32, stats, "out.lse")
            out = Attention(out.out, out.lse if lse else None)
        space = self._space(need, stream)
        args = ua2a_attention_t(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.out.data_ptr(), _ptr(out.lse), _ptr(counts),
                                _ptr(space), need, window, kv, scale, code)
        self._issue("ua2a_attention", stream, ctypes.byref(args))
        return out

    def window_attention_backward(self, dout, q, k, v, out, lse, *, left=None, right=None, sinks: int = 0,
                                  chunk: int = 1, counts=None, scale=None,
                                  grads: Optional[AttentionGradients] = None, stream=None) -> AttentionGradients:
        """Gradients of ``window_attention`` (same window, counts and scale):
        ``dout`` is the gradient of its ``out``; ``out`` and ``lse`` are its
        results.  Sums run in a fixed order, so equal inputs give equal bits.
        ``grads``: an earlier result to write again."""
        import torch
        heads = self._check_heads(q, k, v, counts)
        code, window, scale, kv, need = self._attention_spec("backward", heads, None, left, right, sinks, chunk, scale)
        w, B, SG, hl, _ = shape = self.out_shape(0)
        self._check(dout, shape, "dout")
        self._check(out, shape, "out")
        self._expect(lse, torch.float32, (w, B, hl, SG), "lse")
        if grads is None:
            with self._on_stream(stream):
                grads = AttentionGradients(*(torch.empty(t.shape, dtype=self.dtype, device=self.device)
                                             for t in (q, k, v)))
        else:
            for t, like, what in zip(grads, (q, k, v), AttentionGradients._fields):
                self._check(t, like.shape, f"grads.{what}")
            grads = AttentionGradients(*grads)
        space = self._space(need, stream)
        args = ua2a_attention_grad_t(dout.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                                     lse.data_ptr(), *[t.data_ptr() for t in grads], _ptr(counts), _ptr(space), need, window,
                                     kv, scale, code)
        self._issue("ua2a_attention_backward", stream, ctypes.byref(args))
        return grads

    def cache_attention(self, cache, q, starts, counts=None, *, left=None, right=0, sinks: int = 0, chunk: int = 1,
                        scale=None, out=None, stream=None):
        """The same attention of new tokens over a ``Cache`` that holds their
        keys and values already (``cache_write`` with the same ``starts`` and
        ``counts``).

        ``q``: ``[w, sequences, n, H/w, D]`` in the plan's dtype, n new tokens
        of each sequence (mode 0's result holds them in this order); the
        cache's heads divide H/w.  Token t < ``counts[i]`` (None: all) of
        sequence i has position ``starts[i] + t``, where that lies in the
        cache, and the positions up to the last of them hold keys.  Rows
        without a position are left as they were; without ``out`` they are
        zeros (the result is filled first).
        """
        self._check_cache_of(cache, None, starts, counts)
        if starts is None:
            raise ValueError("starts is missing")
        n = q.shape[2] if q.dim() == 5 else 0
        shape = (self.w, cache.sequences, n, self.H // self.w, self.D)
        if not self._fits(q, self.dtype, shape):
            self._check(q, shape, "q")
        if n < 1:
            raise ValueError("q has no tokens")
        code, window, scale, kv, need = self._attention_spec("cache", cache.heads, (cache.sequences, cache.capacity, n), left,
                                                             right, sinks, chunk, scale)
        if out is None:
            import torch
            with self._on_stream(stream):
                out = torch.zeros(shape, dtype=self.dtype, device=self.device)
        elif not self._fits(out, self.dtype, shape):
            self._check(out, shape, "out")
        space = self._space(need, stream)
        args = ua2a_cache_attention_t(q.data_ptr(), out.data_ptr(), starts.data_ptr(), _ptr(counts), _ptr(space), need, window,
                                      n, kv, scale, code)
        self._issue("ua2a_cache_attention", stream, cache._ref, ctypes.byref(args))
        return out
