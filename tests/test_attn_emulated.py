"""The attention operators' host side and walks, without a GPU: the library's own
argument checks, shapes, tiles, parts and places, carried out on host memory."""
from __future__ import annotations

import ctypes

import pytest
import torch

import ulysses_all_re_amd as ua
from tests import act_reference as act
from tests import attn_reference as ref
from tests.emu import attn_build
from ulysses_all_re_amd.activations import ua2a_cache_t
from ulysses_all_re_amd.attention import (ua2a_attention_grad_t, ua2a_attention_t, ua2a_cache_attention_t, ua2a_rope_t,
                                          ua2a_window_t)

INVALID, SHAPE, ALIGN, ALIAS, CAPACITY, DEVICE = -1, -2, -3, -4, -5, -6


@pytest.fixture(scope="module")
def lib():
    so = ctypes.CDLL(attn_build.build())
    i32, i64, vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p
    so.ua2a_plan.argtypes = [ctypes.POINTER(vp), i32, i64, i64, i64, i64, i32, i32, vp, i64, i32]
    so.ua2a_destroy.argtypes = [vp]
    so.ua2a_attn_emu_errors.restype = so.ua2a_attn_emu_last.restype = i64
    return ua.declare_attention_signatures(so)


@pytest.fixture
def dry(lib):
    lib.ua2a_attn_emu_dry(1)
    yield lib
    lib.ua2a_attn_emu_dry(0)


def make_plan(lib, w, B, S, H, D, e=2, device=0):
    h = ctypes.c_void_p()
    assert lib.ua2a_plan(ctypes.byref(h), w, B, S, H, D, e, 0, None, 0, device) == 0
    return h


def values(shape, dtype, seed, size=1.0):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * size).to(dtype)


def aligned(shape, dtype):
    """Uninitialised memory that starts at a multiple of 16 bytes."""
    n = 1
    for s in shape:
        n *= s
    raw = torch.empty(n + 16, dtype=dtype)
    off = (-raw.data_ptr() % 16) // raw.element_size()
    return raw[off:off + n].view(shape)


def keep(t):
    out = aligned(t.shape, t.dtype)
    out.copy_(t)
    return out


def window_of(window):
    left, right, sinks, chunk = window
    return ua2a_window_t(-1 if left is None else left, -1 if right is None else right, sinks, chunk)


WINDOWS = [(None, None, 0, 1), (None, 0, 0, 1), (0, 0, 0, 1), (5, 0, 3, 1), (30, 9, 2, 1), (0, 0, 0, 7), (1, 0, 5, 16),
           (2, 1, 40, 33), (0, 0, 70, 1), (0, None, 500, 1), (1, 0, 150, 64)]
# (w, B, S, H, D), key heads
SHAPES = [((1, 1, 1, 1, 8), 1), ((2, 1, 17, 4, 16), 2), ((3, 2, 13, 6, 8), 3), ((1, 1, 140, 7, 8), 1), ((1, 2, 300, 2, 8), 2),
          ((1, 1, 40, 2, 104), 1)]


@pytest.mark.parametrize("shape,kv", SHAPES, ids=lambda v: "x".join(map(str, v)) if isinstance(v, tuple) else str(v))
def test_attention_walks(lib, shape, kv):
    """Forward and backward: every key that a row sees, once; every value written once."""
    w, B, S, H, D = shape
    plan = make_plan(lib, *shape)
    a = (w, B, S * w, H // w, D)
    ka = a[:3] + (kv // w, D)
    q, k, v = keep(values(a, torch.bfloat16, 1)), keep(values(ka, torch.bfloat16, 2)), keep(values(ka, torch.bfloat16, 3))
    dout = keep(values(a, torch.bfloat16, 4, 0.1))
    for i, window in enumerate(WINDOWS):
        counts = None if i % 2 else [max(0, S * w - 5 * b - i) for b in range(B)]
        n = None if counts is None else torch.tensor(counts, dtype=torch.int32)
        out, lse = aligned(a, torch.bfloat16), torch.empty(w, B, H // w, S * w)
        args = ua2a_attention_t(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(),
                                None if n is None else n.data_ptr(), None, 0, window_of(window), kv, D ** -0.5, 0)
        need = ctypes.c_int64()
        assert lib.ua2a_attention_workspace(plan, ctypes.byref(args), ctypes.byref(need)) == 0
        space = aligned((max(1, need.value // 4),), torch.float32)
        args.workspace, args.workspace_bytes = space.data_ptr(), need.value
        assert lib.ua2a_attention(plan, ctypes.byref(args), None) == 0
        assert lib.ua2a_attn_emu_errors() == 0, window
        ref.check_forward(out, lse, q, k, v, window, D ** -0.5, counts, f"{window}")
        grads = [aligned(a, torch.bfloat16), aligned(ka, torch.bfloat16), aligned(ka, torch.bfloat16)]
        args = ua2a_attention_grad_t(dout.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                                     lse.data_ptr(), *[t.data_ptr() for t in grads], None if n is None else n.data_ptr(),
                                     None, 0, window_of(window), kv, D ** -0.5, 0)
        assert lib.ua2a_attention_backward_workspace(plan, ctypes.byref(args), ctypes.byref(need)) == 0
        space = aligned((need.value // 4,), torch.float32)
        args.workspace, args.workspace_bytes = space.data_ptr(), need.value
        assert lib.ua2a_attention_backward(plan, ctypes.byref(args), None) == 0
        assert lib.ua2a_attn_emu_errors() == 0, window
        ref.check_backward(grads, dout, q, k, v, out, lse, window, D ** -0.5, counts, f"{window}")
    lib.ua2a_destroy(plan)


@pytest.mark.parametrize("H,kv,D,seqs,cap,n", [(1, 1, 8, 1, 1, 1), (8, 2, 8, 3, 150, 1), (14, 2, 16, 2, 300, 2), (4, 4, 40, 2, 200, 20),
                                               (2, 2, 8, 1, 1500, 140), (2, 1, 8, 1, 4000, 1)])
def test_cache_walks(lib, H, kv, D, seqs, cap, n):
    fmt = torch.float8_e4m3fn
    plan = make_plan(lib, 1, 1, 1, H, D)
    g = torch.Generator().manual_seed(5)
    codes, scales = act.quantise(torch.randn((2, 1, seqs, cap, kv, D), generator=g), fmt)
    codes = keep(codes)
    held = act.dequantise(codes, scales, fmt).to(torch.bfloat16)
    q = keep(values((1, seqs, n, H, D), torch.bfloat16, 6))
    for i, window in enumerate(WINDOWS):
        starts = torch.randint(-2, cap + 1, (seqs,), generator=g).to(torch.int32)
        starts[0] = cap - n
        counts = torch.randint(0, n + 2, (seqs,), generator=g).to(torch.int32) if i % 2 else None
        out = keep(torch.full(q.shape, 7.0, dtype=torch.bfloat16))
        cache = ua2a_cache_t(codes.data_ptr(), scales.data_ptr(), seqs, cap, 1)
        args = ua2a_cache_attention_t(q.data_ptr(), out.data_ptr(), starts.data_ptr(),
                                      None if counts is None else counts.data_ptr(), None, 0, window_of(window), n, kv, 0.3, 0)
        need = ctypes.c_int64()
        assert lib.ua2a_cache_attention_workspace(plan, ctypes.byref(cache), ctypes.byref(args), ctypes.byref(need)) == 0
        space = aligned((max(1, need.value // 4),), torch.float32)
        args.workspace, args.workspace_bytes = space.data_ptr(), need.value
        assert lib.ua2a_cache_attention(plan, ctypes.byref(cache), ctypes.byref(args), None) == 0
        assert lib.ua2a_attn_emu_errors() == 0, window
        for s in range(seqs):
            start, count = int(starts[s]), n if counts is None else int(counts[s])
            live = [t for t in range(n) if t < count and 0 <= start + t < cap]
            assert bool((out[:, s, [t for t in range(n) if t not in live]] == 7).all())
            if not live:
                continue
            end = start + live[-1] + 1
            seen = ref.visible(start + torch.tensor(live), torch.arange(end), *window)
            for h in range(H):
                row = ref.Row(q[0, s, live, h], held[0, 0, s, :end, h * kv // H], held[1, 0, s, :end, h * kv // H], seen, 0.3)
                want = row.out()
                act.assert_close(out[0, s, live, h], want, ref.forward_bound(row, torch.bfloat16, want), f"{window} {s} {h}")
    lib.ua2a_destroy(plan)


@pytest.mark.parametrize("t", ["bf16", "fp32"])
@pytest.mark.parametrize("shape,dims,halves", [((1, 1, 1, 1, 2), (2,), False), ((2, 1, 5, 4, 16), (16,), True),
                                               ((3, 2, 7, 6, 40), (12, 14, 10), False), ((2, 1, 3, 2, 7), (4,), False),
                                               ((2, 2, 3, 4, 7), (2, 4), True), ((1, 2, 5, 3, 264), (130, 128), False),
                                               ((1, 1, 3, 2, 1030), (1030,), True), ((2, 1, 900, 16, 64), (32, 32), True),
                                               ((1, 1, 2, 1, 4104), (4096,), True)],
                         ids=lambda v: "x".join(map(str, v)) if isinstance(v, tuple) else str(v))
def test_rope_walks(lib, shape, dims, halves, t):
    w, B, S, H, D = shape
    dtype, code = (torch.bfloat16, 0) if t == "bf16" else (torch.float32, 2)
    plan = make_plan(lib, *shape, e=2 if t == "bf16" else 4)
    r = ua.Rotary(D, dims, halves=halves, device="cpu")
    freqs = [10000.0 ** (-2.0 * i / d) for d in dims for i in range(d // 2)]
    axes = [a for a, d in enumerate(dims) for _ in range(d // 2)]
    g = torch.Generator().manual_seed(1)
    for planes in (0, 1):
        pos = torch.randint(-2 ** 31, 2 ** 31, (len(dims),) + ((B,) if planes else ()) + (S * w,), generator=g).to(torch.int32)
        for from_a, to_a in ((0, 1), (1, 0), (0, 0), (1, 1)):
            p, a = shape, (w, B, S * w, H // w, D)
            x, out = keep(values(a if from_a else p, dtype, 3)), aligned(a if to_a else p, dtype)
            args = ua2a_rope_t(x.data_ptr(), out.data_ptr(), pos.data_ptr(), r.turns.data_ptr(), r.axes.data_ptr(), r.pairs,
                               r.naxes, halves, to_a, planes, from_a, to_a, code)
            assert lib.ua2a_rope(plan, ctypes.byref(args), None) == 0
            assert lib.ua2a_attn_emu_errors() == 0
            if D > 300 or S > 100:
                continue                                          # places alone: the definition is exact and slow
            want, size = ref.rope(x, pos, freqs, axes, halves, w, from_a, to_a, bool(to_a))
            ref.check_rope(out, want, size, dtype, f"{shape} {from_a}->{to_a}")
    lib.ua2a_destroy(plan)


def test_windows_by_their_definition():
    """What a query sees and which queries see a key, over small sizes (the same rules
    that the walks above take, here against each other)."""
    t = torch.arange(40)
    for window in [(l, r, s, c) for l in (None, 0, 2) for r in (None, 0, 3) for s in (0, 1, 7, 50) for c in (1, 3, 16)]:
        left, right, sinks, chunk = window
        seen = ref.visible(t, t, *window)
        for p in range(40):
            for j in range(40):
                near = (left is None or j // chunk >= p // chunk - left) and (right is None or j // chunk <= p // chunk + right)
                sink = j < sinks and (right != 0 or j // chunk <= p // chunk)
                assert bool(seen[p, j]) == (near or sink), (window, p, j)


# ---------------------------------------------------------------- refusals

def attention_args(**kw):
    base = dict(q=1 << 40, k=1 << 42, v=1 << 43, out=1 << 44, workspace=1 << 45, workspace_bytes=1 << 40,
                window=ua2a_window_t(-1, 0, 0, 1), kv_heads=4, scale=0.5, type=0)
    base.update(kw)
    return ua2a_attention_t(**base)


@pytest.mark.parametrize("change,code", [
    (dict(), 0), (dict(q=None), INVALID), (dict(out=None), INVALID), (dict(type=2), INVALID), (dict(type=9), INVALID),
    (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(window=ua2a_window_t(-2, 0, 0, 1)), INVALID),
    (dict(window=ua2a_window_t(0, -2, 0, 1)), INVALID), (dict(window=ua2a_window_t(0, 0, -1, 1)), INVALID),
    (dict(window=ua2a_window_t(0, 0, 0, 0)), INVALID), (dict(window=ua2a_window_t(1 << 31, 0, 0, 1)), INVALID),
    (dict(window=ua2a_window_t(0, 0, 0, 1 << 31)), INVALID),
    (dict(window=ua2a_window_t((1 << 31) - 1, (1 << 31) - 1, (1 << 31) - 1, (1 << 31) - 1)), 0),
    (dict(kv_heads=0), SHAPE), (dict(kv_heads=3), SHAPE), (dict(kv_heads=6), SHAPE), (dict(kv_heads=8), 0),
    (dict(q=(1 << 40) + 8), ALIGN), (dict(lse=(1 << 46) + 2), ALIGN), (dict(counts=(1 << 46) + 1), ALIGN),
    (dict(out=1 << 40), ALIAS), (dict(lse=1 << 40), ALIAS), (dict(lse=1 << 44), ALIAS), (dict(counts=1 << 44), ALIAS)])
def test_attention_refusals(dry, change, code):
    plan = make_plan(dry, 2, 1, 8, 8, 16)
    args = attention_args(**change)
    assert dry.ua2a_attention(plan, ctypes.byref(args), None) == code
    dry.ua2a_destroy(plan)


def test_attention_shapes_and_workspaces(dry):
    for shape, code in (((1, 1, 8, 4, 12), SHAPE), ((1, 1, 8, 4, 136), SHAPE), ((1, 1, 8, 4, 128), 0), ((1, 1, 8, 32768, 128), 0),
                        ((1, 1, 8, 65536, 128), SHAPE), ((1, 63, 1 << 23, 4, 8), 0),
                        ((1, 64, 1 << 23, 4, 8), SHAPE)):
        plan = make_plan(dry, *shape)
        args = attention_args(kv_heads=shape[3], k=1 << 46, v=1 << 48, out=1 << 50, workspace=1 << 52)
        assert dry.ua2a_attention(plan, ctypes.byref(args), None) == code, shape
        dry.ua2a_destroy(plan)
    plan = make_plan(dry, 1, 1, 4000, 1, 64)
    args = attention_args(kv_heads=1)
    need = ctypes.c_int64()
    assert dry.ua2a_attention_workspace(plan, ctypes.byref(args), ctypes.byref(need)) == 0 and need.value > 0
    for change, code in ((dict(workspace_bytes=need.value), 0), (dict(workspace_bytes=need.value - 1), CAPACITY),
                         (dict(workspace=None), INVALID), (dict(workspace=(1 << 45) + 8), ALIGN),
                         (dict(workspace=1 << 40), ALIAS)):
        assert dry.ua2a_attention(plan, ctypes.byref(attention_args(kv_heads=1, **change)), None) == code, change
    assert dry.ua2a_attention_workspace(plan, ctypes.byref(args), None) == INVALID
    assert dry.ua2a_attention(plan, None, None) == INVALID and dry.ua2a_attention(None, ctypes.byref(args), None) == INVALID
    other = make_plan(dry, 2, 1, 8, 8, 16, device=1)
    assert dry.ua2a_attention(other, ctypes.byref(attention_args()), None) == DEVICE
    four = make_plan(dry, 2, 1, 8, 8, 16, e=4)
    assert dry.ua2a_attention(four, ctypes.byref(attention_args(type=2)), None) == INVALID


def grad_args(**kw):
    base = {n: (40 << 36) + (i << 33) for i, n in enumerate(("dout", "q", "k", "v", "out", "lse", "dq", "dk", "dv"))}
    base.update(workspace=1 << 45, workspace_bytes=1 << 40, window=ua2a_window_t(-1, 0, 0, 1), kv_heads=4, scale=0.5, type=0)
    base.update(kw)
    return ua2a_attention_grad_t(**base)


@pytest.mark.parametrize("change,code", [
    (dict(), 0), (dict(dk=None), INVALID), (dict(lse=None), INVALID), (dict(workspace=None), INVALID),
    (dict(type=2), INVALID), (dict(scale=0.0), INVALID), (dict(kv_heads=3), SHAPE), (dict(dout=8), ALIGN), (dict(dv=8), ALIGN),
    (dict(workspace=8), ALIGN), (dict(lse=2), ALIGN), (dict(workspace_bytes=4), CAPACITY),
    (dict(dk=(40 << 36) + (6 << 33)), ALIAS), (dict(dq=40 << 36), ALIAS), (dict(workspace=40 << 36), ALIAS)])
def test_backward_refusals(dry, change, code):
    plan = make_plan(dry, 2, 1, 8, 8, 16)
    assert dry.ua2a_attention_backward(plan, ctypes.byref(grad_args(**change)), None) == code
    dry.ua2a_destroy(plan)


@pytest.mark.parametrize("args,cache,code", [
    (dict(), dict(), 0), (dict(q=None), {}, INVALID), (dict(starts=None), {}, INVALID), ({}, dict(codes=None), INVALID),
    ({}, dict(scales=None), INVALID), ({}, dict(format=0), INVALID), ({}, dict(sequences=0), SHAPE),
    ({}, dict(capacity=0), SHAPE), ({}, dict(capacity=1 << 31), SHAPE), (dict(n=0), {}, SHAPE), (dict(n=1 << 31), {}, SHAPE),
    (dict(kv_heads=5), {}, SHAPE), ({}, dict(codes=4), ALIGN), (dict(q=8), {}, ALIGN), (dict(starts=2), {}, ALIGN),
    (dict(out=1 << 41), {}, ALIAS), (dict(out=1 << 40), {}, ALIAS), (dict(n=1 << 24), dict(sequences=1 << 8), SHAPE)])
def test_cache_refusals(dry, args, cache, code):
    plan = make_plan(dry, 1, 1, 1, 8, 64)
    c = dict(codes=1 << 41, scales=1 << 42, sequences=3, capacity=100, format=1)
    c.update(cache)
    a = dict(q=1 << 40, out=1 << 43, starts=1 << 44, workspace=1 << 45, workspace_bytes=1 << 40,
             window=ua2a_window_t(-1, 0, 0, 1), n=2, kv_heads=4, scale=0.5, type=0)
    a.update(args)
    assert dry.ua2a_cache_attention(plan, ctypes.byref(ua2a_cache_t(**c)), ctypes.byref(ua2a_cache_attention_t(**a)), None) == code
    dry.ua2a_destroy(plan)


@pytest.mark.parametrize("change,code", [
    (dict(), 0), (dict(x=None), INVALID), (dict(turns=None), INVALID), (dict(to=2), INVALID), (dict(halves=2), INVALID),
    (dict(type=2), INVALID), (dict(pairs=0), SHAPE), (dict(pairs=9), SHAPE), (dict(naxes=0), SHAPE),
    (dict(naxes=1 << 30), SHAPE), (dict(turns=(1 << 43) + 4), ALIGN), (dict(x=(1 << 40) + 1), ALIGN),
    (dict(positions=(1 << 42) + 2), ALIGN), (dict(out=1 << 40), ALIAS), (dict(out=1 << 40, to=0), 0),
    (dict(out=(1 << 40) + 2, to=0), ALIAS), (dict(out=1 << 42), ALIAS)])
def test_rope_refusals(dry, change, code):
    plan = make_plan(dry, 2, 1, 8, 8, 16)
    a = dict(x=1 << 40, out=1 << 41, positions=1 << 42, turns=1 << 43, axes=1 << 44, pairs=8, naxes=1, halves=0, inverse=0,
             per_plane=0, from_=0, to=1, type=0)
    a.update(change)
    assert dry.ua2a_rope(plan, ctypes.byref(ua2a_rope_t(**a)), None) == code
    dry.ua2a_destroy(plan)


def test_parts_fit_their_workspace(dry):
    """Over many shapes: a call's parts are within what it states, and a small one."""
    g = torch.Generator().manual_seed(0)
    pick = lambda lo, hi: int(torch.randint(lo, hi + 1, (1,), generator=g))  # noqa: E731
    for _ in range(300):
        w, group, D = pick(1, 4), pick(1, 5), 8 * pick(1, 16)
        kv = w * pick(1, 6)
        B, S = pick(1, 3), pick(1, 20000 // w)
        plan = make_plan(dry, w, B, S, kv * group, D)
        window = ua2a_window_t(pick(-1, 3000), pick(-1, 3) * pick(0, 500), pick(0, 3000), pick(1, 2000))
        if window.right < -1:
            window.right = -1
        need = ctypes.c_int64()
        args = attention_args(window=window, kv_heads=kv, k=1 << 46, v=1 << 48, out=1 << 50, workspace=1 << 52)
        assert dry.ua2a_attention_workspace(plan, ctypes.byref(args), ctypes.byref(need)) == 0
        assert need.value <= 512 * 128 * (D + 2) * 4
        assert dry.ua2a_attention(plan, ctypes.byref(args), None) == 0
        args = grad_args(window=window, kv_heads=kv, **{n: (i + 1) << 46 for i, n in enumerate(
            ("dout", "q", "k", "v", "out", "lse", "dq", "dk", "dv", "workspace"))})
        assert dry.ua2a_attention_backward_workspace(plan, ctypes.byref(args), ctypes.byref(need)) == 0
        assert need.value <= (256 << 20) + w * B * S * w * kv * group // w * 4 + 16
        assert dry.ua2a_attention_backward(plan, ctypes.byref(args), None) == 0
        assert dry.ua2a_attn_emu_errors() == 0
        dry.ua2a_destroy(plan)


def test_a_scale_past_the_range_in_powers_of_two(dry):
    plan = make_plan(dry, 2, 1, 8, 8, 16)
    assert dry.ua2a_attention(plan, ctypes.byref(attention_args(scale=3e38)), None) == INVALID
    assert dry.ua2a_attention(plan, ctypes.byref(attention_args(scale=2e38)), None) == 0
    assert dry.ua2a_attention_backward(plan, ctypes.byref(grad_args(scale=3e38)), None) == INVALID
    dry.ua2a_destroy(plan)


@pytest.mark.parametrize("end", [(1 << 31) - 1, (1 << 31) - 2, (1 << 31) - 64, (1 << 31) - 128, 1000])
def test_tiles_at_the_end_of_the_largest_cache(lib, end):
    """A tile that reaches 2^31: what the kernels take as seen by all rows, by none, and by a
    row, against the definition in Python's integers."""
    flags = (ctypes.c_uint8 * 128)()
    for left, right, sinks, chunk in [(0, 0, 0, 1), (None, 0, 0, 1), (40, 0, 5, 1), (None, None, 0, 1), (0, 0, (1 << 31) - 1, 1),
                                      (1, 0, 4, 50), (3, 7, 0, 1), (0, None, 9, 16), (200, 0, 0, 1)]:
        window = window_of((left, right, sinks, chunk))

        def sees(p, j):
            c = j // chunk - p // chunk
            near = (left is None or c >= -left) and (right is None or c <= right)
            return j < end and (near or (j < sinks and (right != 0 or c <= 0)))

        for size in (32, 64, 128):
            last = (end - 1) // size * size
            for k0 in (0, last - size, last):
                for p0, p1 in ((end - 1, end - 1), (end - 31, end - 1), (end - 128, end - 60)):
                    got = lib.ua2a_attn_emu_tile(ctypes.byref(window), p0, p1, end, k0, size, flags)
                    at = (end, left, right, sinks, chunk, size, k0, p0, p1)
                    rows = [[sees(p, j) for j in range(k0, k0 + size)] for p in range(p0, p1 + 1)]
                    assert list(map(bool, flags[:size])) == rows[0], at
                    if got & 1:
                        assert all(map(all, rows)), at
                    if got & 2:
                        assert not any(map(any, rows)), at
                    # a tile that one row sees whole, or not at all, is known as such
                    if p0 == p1:
                        assert bool(got & 1) == all(rows[0]) or sinks, at
                        assert bool(got & 2) == (not any(rows[0])), at
