"""GPU: numbers at which attention could go wrong: visible infinities, weights far below
the largest, and fp16's small gradients, each against the definition in 64 bits."""
from __future__ import annotations

import pytest
import torch

import ulysses_all_re_amd as ua
from tests import attn_reference as ref
from tests.test_gpu_attention import (DEV, E4M3, E5M2, TYPES, as_args, gpu, inputs, ints, make_cache, note,  # noqa: F401
                                      values)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t", ["bf16", "fp16"])
@pytest.mark.parametrize("n", [1, 3, 8, 20, 70])
def test_visible_infinities_of_a_cache(t, n):
    """A value's infinity, in a tile that every query sees whole and in one at a window's
    edge, reaches the rows that see it with its sign; both signs, or NaN, give NaN; the
    other rows and values keep their bits."""
    note(f"cache infinities {t} {n}")
    dtype = TYPES[t]
    plan = ua.Plan(1, 1, 1, 4, 128, dtype, device=DEV)
    q = values((1, 2, n, 4, 128), dtype, 9)
    starts = ints([400, 300])
    for window in ((None, 0, 0, 1), (200, 0, 3, 1), (None, None, 0, 1)):
        cache, _ = make_cache(1, 2, 520, 2, 128, E5M2, 8)
        codes = cache.codes.view(torch.uint8)
        want = plan.cache_attention(cache, q, starts, **as_args(window))
        # (part, rank, sequence, position, head, value); 0x7c and 0xfc are the format's infinities
        for j, h, d, code in ((290, 0, 5, 0x7c), (290, 0, 6, 0xfc), (295, 0, 70, 0x7c), (330, 0, 70, 0xfc), (250, 1, 127, 0x7f),
                              (204, 1, 0, 0x7c)):
            codes[1, :, :, j, h, d] = code
        got = plan.cache_attention(cache, q, starts, **as_args(window))
        for s, first in enumerate((400, 300)):
            p = first + torch.arange(n, device=DEV)
            sees = lambda j: ((p >= j) if window[1] == 0 else (p >= 0) & (j < first + n)) & (  # noqa: E731
                True if window[0] is None else p - j <= window[0])
            inf = float("inf")
            for j, h, d, x in ((290, 0, 5, inf), (290, 0, 6, -inf), (295, 0, 70, inf), (330, 0, 70, -inf), (250, 1, 127, float("nan")),
                               (204, 1, 0, inf)):
                want[0, s, :, 2 * h:2 * h + 2, d] += torch.where(sees(j), x, 0.0).to(dtype)[:, None]
        assert torch.equal(torch.isnan(got), torch.isnan(want)), window
        whole = torch.isinf(want)
        assert torch.equal(got[whole], want[whole]), window
        # what holds no infinity keeps its bits (an infinite value's own column has others' sums too)
        for d in (5, 6, 70):
            want[..., d], got[..., d] = 0, 0
        want[..., 127], got[..., 127], want[..., 0], got[..., 0] = 0, 0, 0, 0
        assert torch.equal(got, want), window


def small_weights_error(gap):
    """Of weights `gap` powers of two below the largest, relative: their rounding.  The
    largest is held at 2^13 at least, fp16 has 11 digits down to 2^-14 and half a step of
    2^-25 below; then the result's own rounding, and 2^-14 for the sums and exponentials."""
    return max(2.0 ** -11, 2.0 ** (gap - 13 - 25)) + 2.0 ** -11 + 2.0 ** -14


@pytest.mark.parametrize("t", ["bf16", "fp16"])
@pytest.mark.parametrize("gap", [6.0, 12.0, 17.4, 19.0])
def test_one_key_takes_most_of_the_weight(gap, t):
    """A token (a sink) `gap` nats above thousands of others, its value zero and theirs 16:
    what the others give together is right, by every kernel, wherever the token stands."""
    dtype = TYPES[t]
    N, D = 6000, 64
    x = torch.tensor(gap / 8, dtype=dtype)                        # a score of 8 x and others of 0
    x = float(x.double())
    weight = torch.exp(torch.tensor(-8 * x, dtype=torch.float64))
    error = 2.0 ** -7 if t == "bf16" else small_weights_error(8 * x * 1.4427)

    def check(got, others, what):
        want = 16 * others * weight / (1 + others * weight)           # no subnormal of the type
        off = float((got.double().cpu() - want).abs().max() / want)
        note(f"{what} {t} {gap}: {off:.2e} of {error:.2e}")
        assert off <= error, what

    plan = ua.Plan(1, 1, N, 1, D, dtype, device=DEV)
    one = ua.Plan(1, 1, 1, 1, D, dtype, device=DEV)
    for place in (0, N // 2, N - 1):
        q, v = (torch.full(plan.out_shape(0), a, dtype=dtype, device=DEV) for a in (1.0, 16.0))
        k = torch.zeros_like(q)
        k[0, 0, place] = x
        v[0, 0, place] = 0
        check(plan.window_attention(q, k, v).out, N - 1, f"prompt {place}")
        # the same scores over a cache
        cache = ua.Cache(1, 1, D, 1, N, E4M3, DEV)
        cache.scales.view(torch.uint8).fill_(127)
        codes = cache.codes.view(torch.uint8).zero_()
        codes[1] = 0x58                                           # 16
        codes[1, 0, 0, place] = 0
        codes[0, 0, 0, place] = 0x38                              # 1
        for n in (1, 20, 70):
            qn = torch.full((1, 1, n, 1, D), x, dtype=dtype, device=DEV)
            check(one.cache_attention(cache, qn, ints([N - n]), right=None), N - 1, f"cache {place} {n}")


def exact_gradients(dout, q, k, v, out, lse, window, scale):
    """dq, dk, dv of one head in float64, blocks of rows at a time."""
    q, k, v, dout, out, lse = (x.double() for x in (q, k, v, dout, out, lse))
    n = q.shape[0]
    left, right, sinks, chunk = window
    assert chunk == 1 and sinks == 0
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    j = torch.arange(n, device=q.device)
    for r in range(0, n, 2048):
        rows = slice(r, min(n, r + 2048))
        p = j[rows]
        seen = torch.ones(len(p), n, dtype=torch.bool, device=q.device)
        if left is not None:
            seen &= j >= p[:, None] - left
        if right is not None:
            seen &= j <= p[:, None] + right
        prob = torch.where(seen, torch.exp(scale * (q[rows] @ k.T) - lse[rows, None]), 0.0)
        ds = prob * (dout[rows] @ v.T - (dout[rows] * out[rows]).sum(-1, keepdim=True))
        dq[rows] = scale * (ds @ k)
        dk += scale * (ds.T @ q[rows])
        dv += prob.T @ dout[rows]
    return dq, dk, dv


# tokens, D, window, size of dout, of v, of q and k
GRADIENTS = [(6124, 64, (512, 512, 0, 1), 0.02, 1.0, 1.0), (6124, 64, (None, None, 0, 1), 1e-3, 1.0, 1.0),
             (24576, 64, (None, None, 0, 1), 0.02, 1.0, 1.0), (24576, 64, (None, None, 0, 1), 1e-3, 1.0, 1.0),
             (24576, 128, (None, 0, 0, 1), 0.02, 1.0, 1.0), (3000, 32, (None, 0, 0, 1), 1e-5, 1.0, 1.5),
             (1000, 128, (None, 0, 0, 1), 30.0, 1.0, 1.5), (700, 64, (300, 0, 0, 1), 4.0, 700.0, 0.5), (40, 72, (None, 0, 0, 1), 1.0, 1.0, 1.0)]


@pytest.mark.parametrize("t", ["bf16", "fp16"])
@pytest.mark.parametrize("case", GRADIENTS, ids=lambda v: "-".join(map(str, v[:2] + v[2][:2] + v[3:])))
def test_gradients_beside_their_own_rounding(case, t):
    """Root mean squares of what gradients are off by, beside that of rounding the exact
    ones.  dq takes dS as two values of the type: what is left is its own rounding (1.2 for
    scores, sums and chance).  dk takes dS and dv takes P rounded once more: errors as
    large as the result's own and independent of it, 1.42 together (1.7)."""
    n, D, window, size, vsize, qsize = case
    dtype = TYPES[t]
    plan = ua.Plan(1, 1, n, 1, D, dtype, device=DEV)
    q, k = (values(plan.out_shape(0), dtype, 70 + i, qsize) for i in range(2))
    v, dout = values(plan.out_shape(0), dtype, 72, vsize), values(plan.out_shape(0), dtype, 73, size)
    r = plan.window_attention(q, k, v, lse=True, **as_args(window))
    got = plan.window_attention_backward(dout, q, k, v, r.out, r.lse, **as_args(window))
    want = exact_gradients(*(x[0, 0, :, 0] for x in (dout, q, k, v, r.out)), r.lse[0, 0, 0], window, D ** -0.5)
    told = []
    for g, x, times, what in zip(got, want, (1.2, 1.7, 1.7), ("dq", "dk", "dv")):
        g = g[0, 0, :, 0]
        assert bool(torch.isfinite(g).all()), what
        off, own = (float((y.double() - x).norm() / x.norm()) for y in (g, x.to(dtype)))
        told.append(f"{what} {off:.3g} of {own:.3g}")
        assert off <= times * own, (told, times)
    note(f"gradients {case} {t}: {told}")


@pytest.mark.parametrize("D", [40, 128])
def test_large_dS_in_fp16(D):
    """Values so large that a dS passes fp16 at the power of two that its row's gradient
    would take: dq is right all the same, past fp16's own range too; dk and dv up to it."""
    n, window = 300, (None, 0, 0, 1)
    plan = ua.Plan(1, 1, n, 2, D, torch.float16, device=DEV)
    q, k = (values(plan.out_shape(0), torch.float16, 80 + i, 0.5) for i in range(2))
    base, dout = values(plan.out_shape(0), torch.float16, 82), values(plan.out_shape(0), torch.float16, 83, 4.0)
    j = torch.arange(n, device=DEV)

    def most(v):
        r = plan.window_attention(q, k, v, **as_args(window)).out.double()
        sizes = []
        for h in range(2):
            x = [t[0, 0, :, h].double() for t in (q, k, v, dout)]
            prob = torch.softmax(torch.where(j <= j[:, None], D ** -0.5 * (x[0] @ x[1].T), float("-inf")), -1)
            sizes.append(float((prob * (x[3] @ x[2].T - (x[3] * r[0, 0, :, h]).sum(-1, keepdim=True))).abs().max()))
        return max(sizes)

    for wanted, outputs in ((40000.0, 3), (200000.0, 1)):
        v = (base.float() * (wanted / most(base))).half()
        assert bool(torch.isfinite(v).all()) and 0.8 * wanted < most(v) < 1.2 * wanted
        # rows' |dout| is below 2^6, so they go in times 2^3 at least
        assert most(v) * 2.0 ** 3 > 65504 and float(dout.double().norm(dim=-1).max()) < 64
        r = plan.window_attention(q, k, v, lse=True, **as_args(window))
        got = plan.window_attention_backward(dout, q, k, v, r.out, r.lse, **as_args(window))
        for h in range(2):
            want = exact_gradients(*(x[0, 0, :, h] for x in (dout, q, k, v, r.out)), r.lse[0, 0, h], window, D ** -0.5)
            for g, x, times, what in list(zip(got, want, (1.2, 1.7, 1.7), ("dq", "dk", "dv")))[:outputs]:
                fits = x.abs() < 65504
                off, own = (float((y.double() - x)[fits].norm() / x[fits].norm()) for y in (g[0, 0, :, h], x.half()))
                note(f"large dS {D} {wanted} {what}: {off:.3g} of {own:.3g}")
                assert off <= times * own, what
    # an infinite gradient: its row has none, the others their bits
    dout[0, 0, 100, 1, 3] = float("inf")
    bad = plan.window_attention_backward(dout, q, k, v, r.out, r.lse, **as_args(window)).dq
    assert not bool(torch.isfinite(bad[0, 0, 100, 1]).any())
    bad[0, 0, 100, 1] = got.dq[0, 0, 100, 1]
    assert torch.equal(bad, got.dq)


@pytest.mark.parametrize("t", ["bf16", "fp16"])
@pytest.mark.parametrize("power", [5, 15, 16, 17, 22, 25, 26, 27, 28, 31, 33, 40, 100])
def test_scores_of_any_size(power, t):
    """Scores of +-2^power, about, and half of that, no whole steps in powers of two: the largest take all of the weight,
    shared alike, by every kernel, from the first key to the last."""
    dtype = TYPES[t]
    N, D, scale = 200, 64, 1.37 * 2.0 ** power
    plan, one = ua.Plan(1, 1, N, 1, D, dtype, device=DEV), ua.Plan(1, 1, 1, 1, D, dtype, device=DEV)
    scale32 = float(torch.tensor(scale))
    codes = {0.5: 0x30, 1.0: 0x38, -1.0: 0xb8, 0.0: 0}
    v = (torch.arange(N * D, device=DEV).view(N, D) % 15 - 7).to(dtype) / 8
    cache = ua.Cache(1, 1, D, 1, N, E4M3, DEV)
    cache.scales.view(torch.uint8).fill_(127)
    held = cache.codes.view(torch.uint8)
    held[1, 0, 0, :, 0] = (v.float()).to(E4M3).view(torch.uint8)
    # k's first value of most keys, and where the largest stand
    for rest, top, places in ((0.5, 1.0, [0]), (0.5, 1.0, [130]), (-1.0, 0.5, [199]), (0.0, 1.0, [3, 140]), (-1.0, 0.0, [64, 65, 66, 67]),
                              (-1.0, -1.0, [0])):
        k = torch.zeros(1, 1, N, 1, D, dtype=dtype, device=DEV)
        k[..., 0] = rest
        held[0].zero_()
        held[0, ..., 0] = codes[rest]
        for p in places:
            k[0, 0, p, 0, 0] = top
            held[0, 0, 0, p, 0, 0] = codes[top]
        q = torch.zeros_like(k)
        q[..., 0] = 0.73
        few = list(range(N)) if rest == top else places
        by = scale32 * float(q[0, 0, 0, 0, 0])                      # of a key's first value
        others = torch.exp(torch.tensor((rest - top) * by, dtype=torch.float64)).item() if rest != top else 0.0
        left = [j for j in range(N) if j not in few]
        x = v.double()
        want = (x[few].sum(0) + others * x[left].sum(0)) / (len(few) + others * len(left))
        # a weight and the result are rounded to the type; 2^-20 for the sums of equal weights
        error = 2.0 ** (-11 if t == "fp16" else -8) * 2 * 1.02
        size = (x[few].abs().sum(0) + others * x[left].abs().sum(0)) / (len(few) + others * len(left))
        r = plan.window_attention(q, k, v.view(1, 1, N, 1, D), scale=scale, lse=True)
        assert bool(((r.out.double()[0, 0, :, 0] - want).abs() <= size * error + 2.0 ** -24).all()), (rest, top)
        lse = top * by + torch.log(torch.tensor(len(few) + others * len(left), dtype=torch.float64)).item()
        # three roundings of 32 bits of a number of its size
        assert bool(((r.lse.double() - lse).abs() <= abs(lse) * 2.0 ** -22 + 2.0 ** -20).all()), (rest, top)
        for n in (1, 16, 20, 70):
            got = one.cache_attention(cache, q[:, :, :n].contiguous(), ints([N - n]), right=None, scale=scale)
            assert bool(((got.double()[0, 0, :, 0] - want).abs() <= size * error + 2.0 ** -24).all()), (rest, top, n)


@pytest.mark.parametrize("t,fmt,code,byte", [("fp16", E4M3, 0x7e, 136), ("fp16", E5M2, 0x7b, 129), ("bf16", E4M3, 0x7e, 248),
                                             ("bf16", E5M2, 0x7b, 241)], ids=["fp16-e4m3", "fp16-e5m2", "bf16-e4m3", "bf16-e5m2"])
def test_codes_past_the_type_are_its_largest(t, fmt, code, byte):
    """The format's largest code at a scale that takes it past the type: a query that sees
    that position alone gets the type's largest value, by every kernel of the cache; as a
    key it is the same value too."""
    dtype = TYPES[t]
    plan = ua.Plan(1, 1, 1, 2, 64, dtype, device=DEV)
    cache, _ = make_cache(1, 2, 300, 2, 64, fmt, 8)
    codes, scales = cache.codes.view(torch.uint8), cache.scales.view(torch.uint8)
    codes[:, 0, 0, 70, 1, 7], codes[:, 0, 0, 70, 1, 40] = code, code | 0x80
    scales[:, 0, 0, 70, 1] = byte
    kk, vv = plan.cache_read(cache, 300)
    most = torch.finfo(dtype).max
    assert float(vv[0, 0, 70, 1, 7]) == most and float(vv[0, 0, 70, 1, 40]) == -most
    for n in (1, 3, 16, 20, 32, 33, 70):
        # (bf16: the largest value times |q7 - q40|, which is up to 8, has to be a score of 32 bits)
        q = values((1, 2, n, 2, 64), dtype, 9, 1.0 if t == "fp16" else 2.0 ** -4)
        start = 70 - n // 2
        got, want = plan.cache_attention(cache, q, ints([start, 5]), left=0)[0, 0], vv[0, 0, start:start + n]
        # the row of the largest key has a score in the ten thousands (in fp16; any size in
        # bf16), whose exponent is off by 2^-10: a weight between two values of the type in
        # the product, not in the sum, so half a step of a weight and half of the result
        near = want.double().abs() * 2 * (2.0 ** -11 if t == "fp16" else 2.0 ** -8) * 1.02
        assert bool(((got.double() - want.double()).abs() <= near).all()), n
        rest = [i for i in range(n) if start + i != 70]
        assert torch.equal(got[rest], want[rest]), n
        # a score of a quarter of the key's largest value: it takes all of the weight, or none
        q.zero_()
        q[0, 0, :, 1, 7] = 0.25
        got = plan.cache_attention(cache, q, ints([100, 5]), scale=1.0)
        assert torch.equal(got[0, 0, :, 1], vv[0, 0, 70, 1].expand(n, -1)), n
        got = plan.cache_attention(cache, -q, ints([100, 5]), scale=1.0)
        assert float(got[0, 0, :, 1].abs().max()) < 100.0, n


@pytest.mark.parametrize("t", ["bf16", "fp16"])
def test_means_of_the_largest_values(t):
    """Values that are all the type's largest, or infinite: so are their means, whatever
    the weights, and for an infinity the kind is kept."""
    dtype = TYPES[t]
    N, D = 500, 64
    plan = ua.Plan(1, 1, N, 2, D, dtype, device=DEV)
    q, k = (values(plan.out_shape(0), dtype, 90 + i) for i in range(2))
    # weights' sums in 32 bits stay finite: bf16's largest value times no more than one key's weight
    window = (0, 0, 0, 1) if t == "bf16" else (None, 0, 0, 1)
    for x in (torch.finfo(dtype).max, -torch.finfo(dtype).max, float("inf"), float("-inf")):
        v = torch.full(plan.out_shape(0), x, dtype=dtype, device=DEV)
        assert torch.equal(plan.window_attention(q, k, v, **as_args(window)).out, v), x


# (w, B, S, H, D), key heads, window, counts
PARTS = [((1, 1, 3000, 1, 64), 1, (None, 0, 0, 1), None), ((1, 2, 2500, 2, 128), 1, (None, None, 0, 1), [1700, 2500]),
         ((2, 1, 2000, 4, 32), 4, (64, 0, 5, 1), None), ((1, 1, 5000, 8, 32), 8, (1, 1, 200, 50), [4321]),
         ((2, 2, 700, 12, 96), 4, (300, 20, 150, 1), [1, 1399])]


@pytest.mark.parametrize("t", ["bf16", "fp16"])
@pytest.mark.parametrize("shape,kv,window,counts", PARTS, ids=lambda v: str(v).replace(" ", ""))
def test_gradients_of_rows_of_every_size(shape, kv, window, counts, t):
    """Rows' gradients from 1e-4 to 10 in one call, walked in parts, with shared key heads,
    sinks and padding: each row's dq beside its own rounding, dk and dv within the
    definition's bounds, and the same bits again."""
    dtype = TYPES[t]
    w, B, S, H, D = shape
    plan = ua.Plan(*shape, dtype, device=DEV)
    q, k, v = inputs(shape, kv, dtype, 6, 1.0)
    rows = 10.0 ** (torch.arange(S * w, device=DEV) * 7 % 6 - 4.0)
    dout = (values(q.shape, torch.float32, 44) * rows.view(1, 1, -1, 1, 1)).to(dtype)
    n = None if counts is None else ints(counts)
    r = plan.window_attention(q, k, v, counts=n, lse=True, **as_args(window))
    got = plan.window_attention_backward(dout, q, k, v, r.out, r.lse, counts=n, **as_args(window))
    ref.check_backward(got, dout, q, k, v, r.out, r.lse, window, D ** -0.5, counts, f"{shape}")
    again = plan.window_attention_backward(dout, q, k, v, r.out, r.lse, counts=n, **as_args(window))
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    for (rank, b, h, m), row in ref.rows_of(q, k, v, window, D ** -0.5, counts):
        if m < 100:
            continue
        (dq, _, _), _ = ref.backward(row, r.out[rank, b, :m, h], dout[rank, b, :m, h], r.lse[rank, b, h, :m], dtype)
        for size in range(6):
            of = rows[:m] == rows[size]
            off, own = (float((y.double() - dq)[of].norm()) for y in (got.dq[rank, b, :m, h], dq.to(dtype)))
            assert off <= 1.2 * own, (rank, b, h, float(rows[size]), off, own)
