"""GPU: rotary positions, and windowed attention forward, backward and over the
8-bit cache, against their definitions in 64 bits."""
from __future__ import annotations

import sys

import pytest
import torch

import ulysses_all_re_amd as ua
from tests import act_reference as act
from tests import attn_reference as ref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2


def note(msg):
    print(f"[gpu-case] {msg}", flush=True)
    sys.stdout.flush()


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ua.load_library()
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()


def values(shape, dtype, seed, size=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * size).to(dtype).to(DEV)


def ints(xs):
    return torch.tensor(xs, dtype=torch.int32, device=DEV)


# ------------------------------------------------------------------- rotary

# (w, B, S, H, D), dims, halves
ROPES = [((1, 1, 1, 1, 2), (2,), False), ((2, 1, 5, 4, 16), (16,), True), ((3, 2, 7, 6, 40), (12, 14, 10), False),
         ((2, 1, 9, 8, 128), (44, 42, 42), False), ((4, 2, 3, 8, 64), (16, 24, 24), True), ((2, 1, 3, 2, 7), (4,), False),
         ((2, 2, 3, 4, 7), (2, 4), True), ((5, 1, 4, 10, 72), (22, 22, 22), True), ((1, 3, 5, 3, 260), (130, 128), False),
         ((1, 1, 3, 2, 1030), (1030,), True), ((8, 1, 2, 8, 96), (0, 48, 40), False)]


@pytest.mark.parametrize("t", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("shape,dims,halves", ROPES, ids=lambda v: "x".join(map(str, v)) if isinstance(v, tuple) else str(v))
def test_rope(shape, dims, halves, t):
    w, B, S, H, D = shape
    dtype = TYPES[t]
    note(f"rope {shape} {dims} {halves} {t}")
    plan = ua.Plan(*shape, dtype, device=DEV)
    rotary = ua.Rotary(D, dims, halves=halves, device=DEV)
    freqs = [10000.0 ** (-2.0 * i / d) for d in dims for i in range(d // 2)]
    axes = [a for a, d in enumerate(dims) for _ in range(d // 2)]
    g = torch.Generator().manual_seed(1)
    for per_plane in (False, True):
        lead = (len(dims), B, S * w) if per_plane else (len(dims), S * w)
        pos = torch.randint(-2 ** 31, 2 ** 31, lead, generator=g).to(torch.int32)
        pos[..., :1] = 0
        for from_a, to_a in ((0, 1), (1, 0), (0, 0), (1, 1)):
            inverse = bool(from_a) != per_plane
            x = values(plan.in_shape(from_a), dtype, 3, 2.0)
            x.view(-1)[0] = 0.0
            if from_a == to_a:
                got = plan.rope(x, rotary, pos.to(DEV), gathered=bool(from_a), inverse=inverse)
                kept = x.clone()
                assert plan.rope(kept, rotary, pos.to(DEV), gathered=bool(from_a), inverse=inverse, out=kept) is kept
                assert torch.equal(kept, got)
            else:
                got = plan.rope_exchange(x, rotary, pos.to(DEV), from_a, inverse=inverse)
            want, size = ref.rope(x.cpu(), pos, freqs, axes, halves, w, from_a, to_a, inverse)
            ref.check_rope(got.cpu(), want, size, dtype, f"{shape} {from_a}->{to_a}")


def test_rope_copies_what_does_not_turn():
    """Values past the pairs keep their bits, infinities, NaN and -0 too, at any place."""
    for D, dims, halves in ((16, (10,), False), (16, (8,), True), (9, (4,), True), (24, (4, 2), False)):
        plan = ua.Plan(2, 1, 3, 4, D, torch.bfloat16, device=DEV)
        x = values(plan.in_shape(0), torch.bfloat16, 5)
        odd = torch.tensor([float("inf"), float("-inf"), float("nan"), -0.0], dtype=torch.bfloat16, device=DEV)
        R = sum(dims)
        x[..., R:] = odd[torch.arange(D - R, device=DEV) % 4]
        y = plan.rope(x, ua.Rotary(D, dims, halves=halves, device=DEV), ints([list(range(6))] * len(dims)))
        assert torch.equal(y[..., R:].contiguous().view(torch.int16), x[..., R:].contiguous().view(torch.int16))
        assert bool(torch.isfinite(y[..., :R]).all())


def test_rope_own_frequencies_and_axes():
    """Frequencies and axes in any order; the exchange alone where nothing moves."""
    D, w = 32, 2
    plan = ua.Plan(w, 2, 5, 4, D, torch.float32, device=DEV)
    freqs, axes = [3.0, 0.25, 1e-3, 7.5, 0.5, 2.0, 1.0], [2, 0, 1, 1, 0, 2, 2]
    rotary = ua.Rotary.of(D, freqs, axes, device=DEV)
    pos = torch.randint(0, 99999, (3, 2, 10), generator=torch.Generator().manual_seed(2)).to(torch.int32)
    x = values(plan.in_shape(0), torch.float32, 6)
    want, size = ref.rope(x.cpu(), pos, freqs, axes, False, w, 0, 1)
    ref.check_rope(plan.rope_exchange(x, rotary, pos.to(DEV), 0).cpu(), want, size, torch.float32, "own")
    still = plan.rope_exchange(x, rotary, torch.zeros_like(pos).to(DEV), 0)
    assert torch.equal(still, plan.exchange(x, 0))


def test_rope_off_a_vector_and_many_tokens():
    """Tensors off a 16-byte boundary; more tokens than one workgroup takes."""
    shape = (2, 1, 700, 4, 64)
    plan = ua.Plan(*shape, torch.float16, device=DEV)
    rotary = ua.Rotary(64, (32, 32), device=DEV)
    pos = torch.stack([torch.arange(1400) // 40, torch.arange(1400) % 40]).to(torch.int32).to(DEV)
    n = plan.layout["tensor_elems"]
    flat = values((n + 3,), torch.float16, 7)
    x, out = flat[3:].view(plan.in_shape(0)), torch.empty(n + 1, dtype=torch.float16, device=DEV)[1:].view(plan.out_shape(0))
    a = plan.rope_exchange(x.contiguous().clone(), rotary, pos, 0)
    assert torch.equal(plan.rope_exchange(x, rotary, pos, 0, out=out), a)
    back = plan.rope_exchange(a, rotary, pos, 1, inverse=True)
    assert bool(((back - x).abs() <= 2.0 ** -9 * (x.abs() + 4)).all())


# ---------------------------------------------------------------- attention

# left, right, sinks, chunk
WINDOWS = [(None, None, 0, 1), (None, 0, 0, 1), (0, 0, 0, 1), (5, 0, 3, 1), (40, 0, 0, 1), (70, 9, 2, 1), (3, 200, 0, 1),
           (0, 0, 0, 7), (1, 0, 5, 16), (2, 1, 40, 33), (None, 0, 9, 50), (0, 0, 70, 1), (0, None, 500, 1), (1, 0, 200, 64)]

# (w, B, S, H, D), key heads
SHAPES = [((1, 1, 1, 1, 8), 1), ((2, 1, 33, 4, 80), 4), ((3, 2, 43, 6, 64), 3), ((1, 1, 129, 7, 32), 1),
          ((2, 2, 70, 8, 128), 2), ((1, 1, 300, 2, 96), 2), ((2, 1, 64, 2, 16), 2), ((1, 2, 257, 4, 72), 2)]


def inputs(shape, kv, dtype, seed=0, size=1.5):
    w, B, S, H, D = shape
    q = values((w, B, S * w, H // w, D), dtype, 10 + seed, size)
    k = values((w, B, S * w, kv // w, D), dtype, 20 + seed, size)
    v = values((w, B, S * w, kv // w, D), dtype, 30 + seed)
    return q, k, v


def as_args(window):
    return dict(zip(("left", "right", "sinks", "chunk"), window))


@pytest.mark.parametrize("t", ["bf16", "fp16"])
@pytest.mark.parametrize("shape,kv", SHAPES, ids=lambda v: "x".join(map(str, v)) if isinstance(v, tuple) else str(v))
def test_attention(shape, kv, t):
    w, B, S, H, D = shape
    dtype = TYPES[t]
    plan = ua.Plan(*shape, dtype, device=DEV)
    q, k, v = inputs(shape, kv, dtype)
    dout = values(q.shape, dtype, 40, 0.1)
    for i, window in enumerate(WINDOWS):
        counts = None if i % 2 else [max(0, S * w - 7 * b - i) for b in range(B)]
        note(f"attention {shape} {kv} {t} {window} {counts}")
        n = None if counts is None else ints(counts)
        r = plan.window_attention(q, k, v, counts=n, lse=True, **as_args(window))
        ref.check_forward(r.out, r.lse, q, k, v, window, D ** -0.5, counts, f"{window}")
        g = plan.window_attention_backward(dout, q, k, v, r.out, r.lse, counts=n, **as_args(window))
        ref.check_backward(g, dout, q, k, v, r.out, r.lse, window, D ** -0.5, counts, f"{window}")


def test_attention_scales_and_far_scores():
    """Other factors, and scores that are hundreds apart (the maximum moves often)."""
    shape = (1, 1, 200, 2, 64)
    plan = ua.Plan(*shape, torch.bfloat16, device=DEV)
    q, k, v = inputs(shape, 2, torch.bfloat16, 1, 4.0)
    k *= torch.linspace(0.1, 4.0, 200, device=DEV).view(1, 1, -1, 1, 1).to(k.dtype)
    dout = values(q.shape, q.dtype, 41)
    for scale in (1.0, 1e-3, 0.37):
        for window in ((None, None, 0, 1), (20, 0, 2, 1)):
            r = plan.window_attention(q, k, v, scale=scale, lse=True, **as_args(window))
            ref.check_forward(r.out, r.lse, q, k, v, window, scale, None, f"scale {scale}")
            g = plan.window_attention_backward(dout, q, k, v, r.out, r.lse, scale=scale, **as_args(window))
            ref.check_backward(g, dout, q, k, v, r.out, r.lse, window, scale, None, f"scale {scale}")


@pytest.mark.parametrize("t", ["bf16", "fp16"])
def test_attention_infinities_and_nan(t):
    """Infinities and NaN reach the rows that see them, with their sign, and no others."""
    dtype = TYPES[t]
    shape = (1, 1, 300, 2, 64)
    plan = ua.Plan(*shape, dtype, device=DEV)
    q, k, v = inputs(shape, 2, dtype, 2)
    v[0, 0, 100, 0, 5] = float("inf")
    v[0, 0, 100, 0, 6] = float("-inf")
    v[0, 0, 130, 0, 5] = float("-inf")
    v[0, 0, 131, 1, 63] = float("nan")
    v[0, 0, 299, 1, 0] = float("nan")
    k[0, 0, 210, 1] = float("nan")
    for window in ((20, 0, 0, 1), (None, 0, 3, 1), (10, 10, 2, 1), (1, 0, 0, 32), (0, 0, 101, 1)):
        note(f"infinities {window}")
        r = plan.window_attention(q, k, v, **as_args(window)).out[0, 0].float()
        t_ = torch.arange(300, device=DEV)
        seen = ref.visible(t_, t_, *window)
        clean = torch.where(torch.isfinite(v), v, torch.zeros_like(v))
        kk = torch.where(torch.isfinite(k), k, torch.zeros_like(k))
        base = plan.window_attention(q, kk, clean, **as_args(window)).out[0, 0].float()
        want = base.clone()
        for j, h, d, x in ((100, 0, 5, float("inf")), (100, 0, 6, float("-inf")), (130, 0, 5, float("-inf")),
                           (131, 1, 63, float("nan")), (299, 1, 0, float("nan"))):
            want[:, h, d] += torch.where(seen[:, j], x, 0.0)
        want[:, 1] = torch.where(seen[:, 210, None], float("nan"), want[:, 1])
        assert torch.equal(torch.isnan(r), torch.isnan(want)), window
        ok = ~torch.isnan(want)
        # rows apart from the NaN key's are the same bits: the others' weights are untouched
        assert torch.equal(r[ok], want[ok]), window


@pytest.mark.parametrize("t", ["bf16", "fp16"])
def test_padding_may_hold_anything(t):
    """Rows and keys past counts: whatever they hold, forward and backward."""
    dtype = TYPES[t]
    shape, counts = (2, 3, 60, 4, 64), [97, 0, 500]
    plan = ua.Plan(*shape, dtype, device=DEV)
    q, k, v = inputs(shape, 2, dtype, 3)
    dout = values(q.shape, dtype, 42)
    n = ints(counts)
    window = (30, 2, 4, 1)
    r = plan.window_attention(q, k, v, counts=n, lse=True, **as_args(window))
    g = plan.window_attention_backward(dout, q, k, v, r.out, r.lse, counts=n, **as_args(window))
    ref.check_forward(r.out, r.lse, q, k, v, window, 64 ** -0.5, counts, "padding")
    for bad in (float("nan"), float("inf"), torch.finfo(dtype).min):
        q2, k2, v2, d2 = (x.clone() for x in (q, k, v, dout))
        for b, c in enumerate(counts):
            for x in (q2, k2, v2, d2):
                x[:, b, c:] = bad
        r2 = plan.window_attention(q2, k2, v2, counts=n, lse=True, **as_args(window))
        assert torch.equal(r2.out, r.out) and torch.equal(r2.lse, r.lse)
        g2 = plan.window_attention_backward(d2, q2, k2, v2, r2.out, r2.lse, counts=n, **as_args(window))
        assert all(torch.equal(a, b) for a, b in zip(g, g2))
    for some in ([-5, 1, 2 ** 31 - 1],):
        r = plan.window_attention(q, k, v, counts=ints(some), lse=True, **as_args(window))
        ref.check_forward(r.out, r.lse, q, k, v, window, 64 ** -0.5, some, "odd counts")


def test_long_walks_in_parts():
    """Few heads and many keys: a tile's keys, or a key's rows, go to several
    workgroups; sinks' rows do so where the window is short."""
    for shape, kv, window, counts in (((1, 1, 3000, 1, 64), 1, (None, 0, 0, 1), None),
                                      ((1, 2, 2500, 2, 128), 1, (None, None, 0, 1), [1700, 2500]),
                                      ((2, 1, 2000, 4, 32), 4, (64, 0, 5, 1), None),
                                      ((1, 1, 5000, 8, 32), 8, (1, 1, 200, 50), [4321])):
        note(f"parts {shape} {window}")
        plan = ua.Plan(*shape, torch.bfloat16, device=DEV)
        q, k, v = inputs(shape, kv, torch.bfloat16, 4)
        dout = values(q.shape, q.dtype, 43, 0.1)
        n = None if counts is None else ints(counts)
        r = plan.window_attention(q, k, v, counts=n, lse=True, **as_args(window))
        ref.check_forward(r.out, r.lse, q, k, v, window, q.shape[-1] ** -0.5, counts, f"{shape}")
        g = plan.window_attention_backward(dout, q, k, v, r.out, r.lse, counts=n, **as_args(window))
        ref.check_backward(g, dout, q, k, v, r.out, r.lse, window, q.shape[-1] ** -0.5, counts, f"{shape}")
        again = plan.window_attention_backward(dout, q, k, v, r.out, r.lse, counts=n, **as_args(window))
        assert all(torch.equal(a, b) for a, b in zip(g, again))


def test_gradients_against_differences():
    """The backward pass against differences of the definition's forward pass."""
    shape = (1, 1, 24, 4, 16)
    plan = ua.Plan(*shape, torch.float16, device=DEV)
    q, k, v = inputs(shape, 2, torch.float16, 5, 1.0)
    dout = values(q.shape, q.dtype, 44)
    window = (6, 0, 2, 1)
    r = plan.window_attention(q, k, v, lse=True, **as_args(window))
    grads = plan.window_attention_backward(dout, q, k, v, r.out, r.lse, **as_args(window))

    def loss(*x):
        return sum((row.out() * dout[a, b, :n, h].double()).sum() for (a, b, h, n), row in ref.rows_of(*x, window, 0.25))

    g = torch.Generator().manual_seed(9)
    for i, x in enumerate((q, k, v)):
        for _ in range(4):
            way = torch.randn(x.shape, generator=g).double().to(DEV)
            args = [t.double() for t in (q, k, v)]
            args[i] = args[i] + 1e-4 * way
            up = loss(*args)
            args[i] = args[i] - 2e-4 * way
            slope = float(up - loss(*args)) / 2e-4
            got = float((grads[i].double() * way).sum())
            size = float((grads[i].double().abs() * way.abs()).sum())
            # a gradient's values are within 2^-9 of the fp16 pass's sizes; differences add 1e-7
            assert abs(got - slope) <= 2.0 ** -8 * size, (i, got, slope)


# --------------------------------------------------------------------- cache

def make_cache(w, seqs, cap, heads, D, fmt, seed):
    """A cache of random codes, and what it holds in float64."""
    g = torch.Generator().manual_seed(seed)
    codes, scales = act.quantise(torch.randn((2, w, seqs, cap, heads, D), generator=g) * 1.3, fmt)
    cache = ua.Cache.of(codes.to(DEV).view(fmt), scales.to(DEV).view(torch.float8_e8m0fnu))
    return cache, act.dequantise(codes, scales, fmt)


def as_type(x, dtype):
    """float64 rounded to the type as a cache read does."""
    most = torch.finfo(dtype).max
    return torch.where(torch.isfinite(x), x.clamp(-most, most), x).to(dtype)


def check_cache(plan, cache, held, q, starts, counts, window, what, scale=None):
    dtype = plan.dtype
    w, seqs, n, hl, D = q.shape
    group = hl // cache.heads
    before = values(q.shape, dtype, 77)
    out = before.clone()
    got = plan.cache_attention(cache, q, ints(starts), None if counts is None else ints(counts), out=out, scale=scale,
                               **as_args(window))
    assert got is out
    kv = as_type(held, dtype).to(DEV)
    for i in range(seqs):
        cap = cache.capacity
        live = [t for t in range(n) if (counts is None or t < counts[i]) and 0 <= starts[i] + t < cap]
        rest = [t for t in range(n) if t not in live]
        assert torch.equal(out[:, i, rest], before[:, i, rest]), what
        if not live:
            continue
        end = starts[i] + live[-1] + 1
        p = starts[i] + torch.tensor(live, device=DEV)
        seen = ref.visible(p, torch.arange(end, device=DEV), *window)
        for r in range(w):
            for h in range(hl):
                row = ref.Row(q[r, i, live, h], kv[0, r, i, :end, h // group], kv[1, r, i, :end, h // group], seen,
                              D ** -0.5 if scale is None else scale)
                want = row.out()
                act.assert_close(out[r, i, live, h], want, ref.forward_bound(row, dtype, want), f"{what} {r} {i} {h}")


# w, heads, key heads, D, sequences, capacity, n
CACHES = [(1, 1, 1, 8, 1, 1, 1), (2, 4, 4, 72, 3, 200, 1), (2, 8, 2, 128, 5, 515, 1), (1, 14, 2, 64, 2, 700, 2),
          (3, 6, 3, 32, 2, 400, 20), (1, 2, 2, 80, 2, 900, 150), (2, 14, 2, 96, 1, 300, 33), (1, 8, 1, 40, 33, 260, 5)]


@pytest.mark.parametrize("t,fmt", [("bf16", E4M3), ("fp16", E5M2), ("bf16", E5M2), ("fp16", E4M3)],
                         ids=["bf16-e4m3", "fp16-e5m2", "bf16-e5m2", "fp16-e4m3"])
@pytest.mark.parametrize("case", CACHES, ids=lambda v: "x".join(map(str, v)))
def test_cache_attention(case, t, fmt):
    w, H, kv, D, seqs, cap, n = case
    dtype = TYPES[t]
    plan = ua.Plan(w, 1, 1, H, D, dtype, device=DEV)
    cache, held = make_cache(w, seqs, cap, kv // w, D, fmt, 3)
    q = values((w, seqs, n, H // w, D), dtype, 50, 1.5)
    g = torch.Generator().manual_seed(4)
    for i, window in enumerate(WINDOWS):
        starts = torch.randint(0, max(1, cap - n + 1), (seqs,), generator=g).tolist()
        counts = None if i % 2 else torch.randint(0, n + 1, (seqs,), generator=g).tolist()
        if i % 3 == 0:
            starts[0] = cap - n
        note(f"cache {case} {t} {window} {starts[:4]} {None if counts is None else counts[:4]}")
        check_cache(plan, cache, held, q, starts, counts, window, f"{case} {window}")


def test_cache_attention_at_the_edges():
    """Tokens before the first position and past the last, counts beyond n, empty sequences."""
    plan = ua.Plan(1, 1, 1, 4, 64, torch.bfloat16, device=DEV)
    cache, held = make_cache(1, 6, 50, 2, 64, E4M3, 5)
    q = values((1, 6, 9, 4, 64), torch.bfloat16, 51)
    starts = [-3, 45, 50, 2 ** 31 - 1, -2 ** 31, 10]
    for counts in (None, [9, 9, 9, 9, 9, 0], [100, 3, 1, 2 ** 31 - 1, -1, -2 ** 31], [2, 9, 9, 9, 9, 9]):
        for window in ((None, 0, 0, 1), (4, 0, 2, 1), (1, 1, 3, 8)):
            note(f"edges {counts} {window}")
            check_cache(plan, cache, held, q, starts, counts, window, f"{counts}")
    fresh = plan.cache_attention(cache, q, ints(starts))
    assert bool((fresh[:, 2:5] == 0).all()) and bool((fresh[:, 5] != 0).any())


def test_cache_attention_long_in_parts():
    """One sequence of many positions: its keys go to several workgroups."""
    for dtype, H, kv, D, n, cap, window in ((torch.bfloat16, 4, 2, 128, 1, 20000, (None, 0, 0, 1)),
                                            (torch.float16, 2, 2, 64, 3, 30000, (9000, 0, 700, 1)),
                                            (torch.bfloat16, 3, 1, 96, 100, 9000, (None, 0, 0, 100))):
        plan = ua.Plan(1, 1, 1, H, D, dtype, device=DEV)
        cache, held = make_cache(1, 1, cap, kv, D, E4M3, 6)
        q = values((1, 1, n, H, D), dtype, 52, 1.5)
        for start in (cap - n, cap // 3, 0):
            note(f"long {H} {kv} {D} {n} {cap} {window} {start}")
            check_cache(plan, cache, held, q, [start], None, window, f"{cap} {start}")


def test_cache_attention_ignores_what_no_query_sees():
    """NaN behind a sequence's last position, and before its window, stays out."""
    plan = ua.Plan(1, 1, 1, 2, 64, torch.bfloat16, device=DEV)
    cache, held = make_cache(1, 2, 300, 2, 64, E4M3, 7)
    q = values((1, 2, 3, 2, 64), torch.bfloat16, 53)
    args = dict(left=30, right=0, sinks=2)
    want = plan.cache_attention(cache, q, ints([100, 290]), **args)
    codes = cache.codes.view(torch.uint8)
    scales = cache.scales.view(torch.uint8)
    codes[:, :, 0, 103:] = 0x7f
    codes[:, :, 0, 2:70] = 0xff
    scales[:, :, 1, 293:] = 255
    scales[:, :, 1, 2:260] = 255
    assert torch.equal(plan.cache_attention(cache, q, ints([100, 290]), **args), want)
    codes[1, :, 0, 102, 1, 9] = 0x7f                              # the last of three: its own row alone sees it
    got = plan.cache_attention(cache, q, ints([100, 290]), **args)
    nan = torch.isnan(got)
    assert bool(nan[0, 0, 2, 1, 9]) and int(nan.sum()) == 1
    assert torch.equal(got[~nan], want[~nan])


def test_they_run_together():
    """A step of a block over a growing cache: keys and queries rotated and exchanged,
    written, and attended over; the same step by prompts at once."""
    w, B, S, H, D = 2, 1, 24, 4, 64
    plan = ua.Plan(w, B, S, H, D, torch.bfloat16, device=DEV)
    rotary = ua.Rotary(D, (16, 24, 24), device=DEV)
    x = [values(plan.in_shape(0), torch.bfloat16, 60 + i) for i in range(3)]
    t = torch.arange(S * w, dtype=torch.int32, device=DEV)
    pos = torch.stack([t // 12, t // 4 % 3, t % 4])
    q, k = (plan.rope_exchange(y, rotary, pos, 0) for y in x[:2])
    v = plan.exchange(x[2], 0)
    window = dict(left=1, right=0, sinks=6, chunk=12)
    cache = ua.Cache(w, H, D, sequences=1, capacity=64, device=DEV)
    zero = ints([0])
    plan.cache_write(cache, plan.rope(x[1], rotary, pos), x[2], zero)
    got = plan.cache_attention(cache, q.view(w, 1, S * w, H // w, D), zero, **window)
    kk, vv = plan.cache_read(cache, S * w)
    want = plan.window_attention(q, kk.view(k.shape), vv.view(v.shape), **window).out
    assert torch.equal(got.view(want.shape), want)
    # frame by frame, each step's queries over the cache so far: the same rows
    held = [y.view(k.shape) for y in (kk, vv)]
    for f in range(4):
        rows = slice(12 * f, 12 * f + 12)
        part = plan.cache_attention(cache, q[:, :, rows].contiguous(), ints([12 * f]), **window)
        for (r, b, h, n), row in ref.rows_of(q, *held, tuple(window.values()), D ** -0.5):
            exact = row.out()
            bound = ref.forward_bound(row, q.dtype, exact)
            act.assert_close(part[r, b, :, h], exact[rows], bound[rows], f"frame {f}")
