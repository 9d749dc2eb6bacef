"""GPU: numbers at which attention could go wrong: visible infinities, weights far below
the largest, and fp16's small gradients, each against the definition in 64 bits."""
from __future__ import annotations

import pytest
import torch

import ulysses_all_re_amd as ua
from tests.test_gpu_attention import DEV, E4M3, E5M2, TYPES, as_args, gpu, ints, make_cache, note, values  # noqa: F401

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
