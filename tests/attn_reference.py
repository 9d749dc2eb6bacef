"""Rotary positions and windowed attention in 64 bits, from their definitions
(tests only), and how far a kernel may be from them.

Tensors are rank-stacked as the library's: P ``[w, B, S, H, D]``, A ``[w, B,
S*w, heads, D]``.
"""
from __future__ import annotations

from fractions import Fraction

import torch

from tests.act_reference import HALF, assert_close, tiny, to_a, to_p

# ---------------------------------------------------------------- rotary


def _pi(bits: int = 256) -> Fraction:
    """pi by Machin's formula."""
    one = 1 << (bits + 32)

    def atan_inverse(x):
        term = one // x
        total, k, sign = term, 1, -1
        while term:
            term //= x * x
            k += 2
            total += sign * (term // k)
            sign = -sign
        return total

    return Fraction(4 * (4 * atan_inverse(5) - atan_inverse(239)), one)


TURN = 2 * _pi()


def angles(positions, frequencies, axes):
    """float64 angles within a turn [..., pairs] of int positions [naxes, ...], exact before their last rounding."""
    flat = positions.reshape(positions.shape[0], -1).tolist()
    rows = []
    for i, f in enumerate(frequencies):
        per = Fraction(f) / TURN                                # turns per position
        row = [float(((p * per) % 1) * TURN) for p in flat[axes[i]]]
        rows.append(torch.tensor(row, dtype=torch.float64))
    return torch.stack(rows, -1).view(positions.shape[1:] + (len(frequencies),))


def rope(x, positions, frequencies, axes, halves, w, from_a, to_a_side, inverse=False):
    """(result, |x| + |partner| of each value) in float64."""
    p = (x if not from_a else to_p(x, w)).double()
    _, B, S, H, D = p.shape
    ang = angles(positions, frequencies, axes)                  # [SG, pairs] or [B, SG, pairs]
    ang = ang.expand(B, S * w, -1).reshape(B, w, S, -1).transpose(0, 1).unsqueeze(3)
    c, s = torch.cos(ang), torch.sin(ang)
    if inverse:
        s = -s
    n = len(frequencies)
    u = slice(0, n) if halves else slice(0, 2 * n, 2)
    z = slice(n, 2 * n) if halves else slice(1, 2 * n, 2)
    y, size = p.clone(), p.abs()
    y[..., u] = p[..., u] * c - p[..., z] * s
    y[..., z] = p[..., z] * c + p[..., u] * s
    size[..., u] = size[..., z] = p[..., u].abs() + p[..., z].abs()
    return (to_a(y, w), to_a(size, w)) if to_a_side else (y, size)


def check_rope(got, want, size, dtype, what):
    """The angle is off by 2^-32 of a turn and three roundings of at most pi / 4
    (2^-22 in all), its series by 2^-26 and a rounding of each of two terms, the
    products and their sum by three roundings: under 2^-21 of both values; then
    half a step of the type."""
    assert got.dtype == dtype, what
    assert_close(got, want, want.abs() * HALF[dtype] + size * 2.0 ** -21 + tiny(dtype), what)


# ------------------------------------------------------------- attention


def visible(p, j, left, right, sinks, chunk):
    """[queries, keys] of integer vectors, straight from the definition."""
    cp, cj = (p // chunk)[:, None], (j // chunk)[None, :]
    seen = torch.ones(cp.shape[0], cj.shape[1], dtype=torch.bool, device=p.device)
    if left is not None:
        seen &= cj >= cp - left
    if right is not None:
        seen &= cj <= cp + right
    sink = (j < sinks)[None, :].expand_as(seen)
    if right == 0:
        sink = sink & (cj <= cp)
    return seen | sink


class Row:
    """One head of one sequence: n queries [n, D] over keys [m, D], with a mask."""

    def __init__(self, q, k, v, seen, scale):
        self.q, self.k, self.v, self.seen, self.scale = q.double(), k.double(), v.double(), seen, scale
        self.v = torch.where(seen.any(0)[:, None], self.v, 0.0)          # keys that nobody sees
        self.k = torch.where(seen.any(0)[:, None], self.k, 0.0)
        self.s = torch.where(seen, scale * (self.q @ self.k.T), float("-inf"))
        top = self.s.amax(-1, keepdim=True)
        top = torch.where(top == float("-inf"), 0.0, top)
        e = torch.exp(self.s - top)
        total = e.sum(-1, keepdim=True)
        self.lse = (torch.log(total) + top)[:, 0]
        self.p = e / torch.where(total > 0, total, 1.0)
        # sum of |q_d k_d| times the scale: what a score's rounding errors go by
        self.size = scale * (self.q.abs() @ self.k.abs().T)
        self.size = torch.where(seen, self.size, 0.0)

    def out(self):
        return self.p @ self.v


def _flush(dtype):
    """What a weight or dS may lose apart from its relative error: half a step of
    fp16's subnormals, 2^-25; of bf16, whose exponents are those of 32 bits, a
    value under 2^-126, for exp2 gives no subnormals of 32 bits (a weight whose
    score lies 88 under the largest is zero) and a product of one underflows."""
    return 2.0 ** -25 if dtype == torch.float16 else 2.0 ** -126


def _score_error(r, D):
    """Relative error of a row's weights before their rounding: a score's sum of
    D products is off by (D + 8) 2^-23 of the sum of their sizes, exp2's argument
    by two roundings of at most three times that sum, its result by 2^-22."""
    return r.size.amax(-1) * ((D + 8) * 2.0 ** -23 + 2.0 ** -20) + 2.0 ** -22


def forward_bound(r, dtype, out):
    """Of a row's result: its weights are off by their scores' error and rounded to
    the type (half a step, or of its subnormals), sums over n keys by n roundings
    of 2^-23, the sum of the weights likewise, and the result is rounded once."""
    n = r.s.shape[-1]
    sizes = r.p @ r.v.abs()
    rel = HALF[dtype] + 2 * _score_error(r, r.q.shape[-1])[:, None] + (2 * n + 64) * 2.0 ** -23
    low = _flush(dtype) * (r.seen.double() @ r.v.abs())
    return sizes * rel * (1 + 2 * rel) + out.abs() * HALF[dtype] * (1 + 4 * rel) + low + tiny(dtype)


def lse_bound(r):
    n = r.s.shape[-1]
    lse = torch.where(torch.isfinite(r.lse), r.lse, 0.0)
    return _score_error(r, r.q.shape[-1]) + (n + 8) * 2.0 ** -24 + lse.abs() * 2.0 ** -21 + 2.0 ** -21


def backward(r, o, g, lse, dtype):
    """(dq, dk, dv) of a Row from a result o, its gradient g and lse, in float64, and their bounds.

    P is off as forward and rounded to the type for dv; dS = P (dP - delta) by
    that and by the errors of both sums of D products, and rounded for dq, dk."""
    o, g, lse = o.double(), g.double(), lse.double()
    D, n, m = r.q.shape[-1], r.q.shape[0], r.k.shape[0]
    prob = torch.where(r.seen, torch.exp(r.s - torch.where(torch.isfinite(lse), lse, 0.0)[:, None]), 0.0)
    prob = torch.where(torch.isfinite(lse)[:, None], prob, 0.0)
    dp, delta = g @ r.v.T, (g * o).sum(-1, keepdim=True)
    ds = prob * (dp - delta)
    dq, dk, dv = r.scale * (ds @ r.k), r.scale * (ds.T @ r.q), prob.T @ g
    err = _score_error(r, D)[:, None] + (lse.abs()[:, None] * 2.0 ** -22).nan_to_num(posinf=0.0)
    u, low = HALF[dtype], _flush(dtype)
    sizes = (D + 8) * 2.0 ** -23 * (g.abs() @ r.v.abs().T + (g.abs() * o.abs()).sum(-1, keepdim=True))
    e_ds = prob * ((dp - delta).abs() * (u + 2 * err + 2.0 ** -20) + sizes) * 1.1 + torch.where(r.seen, low * (1 + (dp - delta).abs()), 0.0)
    e_p = prob * (u + 2 * err) * 1.1 + torch.where(r.seen, low, 0.0)
    bq = r.scale * (e_ds @ r.k.abs() + (m + 8) * 2.0 ** -23 * (ds.abs() @ r.k.abs()))
    bk = r.scale * (e_ds.T @ r.q.abs() + (n + 8) * 2.0 ** -23 * (ds.abs().T @ r.q.abs()))
    bv = e_p.T @ g.abs() + (n + 8) * 2.0 ** -23 * (prob.T @ g.abs())
    return (dq, dk, dv), (bq, bk, bv)


def rows_of(q, k, v, window, scale, counts=None):
    """For every (rank, plane, head): its place and Row over the tokens that exist."""
    w, B, SG, hl, D = q.shape
    group = hl // k.shape[3]
    for b in range(B):
        n = SG if counts is None else max(0, min(SG, counts[b]))
        if n == 0:
            continue
        t = torch.arange(n, device=q.device)
        seen = visible(t, t, *window)
        for r in range(w):
            for h in range(hl):
                yield (r, b, h, n), Row(q[r, b, :n, h], k[r, b, :n, h // group], v[r, b, :n, h // group], seen, scale)


def check_forward(out, lse, q, k, v, window, scale, counts, what):
    """A call's results against the definition; padding must be zeros and -inf."""
    for (r, b, h, n), row in rows_of(q, k, v, window, scale, counts):
        want = row.out()
        at = f"{what} rank {r} plane {b} head {h}"
        assert_close(out[r, b, :n, h], want, forward_bound(row, q.dtype, want), at)
        if lse is not None:
            assert_close(lse[r, b, h, :n], row.lse, lse_bound(row), at + " lse")
    if counts is not None:
        for b, c in enumerate(counts):
            n = max(0, min(q.shape[2], c))
            assert bool((out[:, b, n:] == 0).all()), what + " padding"
            assert lse is None or bool((lse[:, b, :, n:] == float("-inf")).all()), what + " lse of padding"


def check_backward(grads, dout, q, k, v, out, lse, window, scale, counts, what):
    dtype = q.dtype
    w, B, SG, hl, D = q.shape
    group = hl // k.shape[3]
    want = [torch.zeros(t.shape, dtype=torch.float64, device=q.device) for t in (q, k, v)]
    bound = [torch.zeros_like(t) for t in want]
    for (r, b, h, n), row in rows_of(q, k, v, window, scale, counts):
        got, bounds = backward(row, out[r, b, :n, h], dout[r, b, :n, h], lse[r, b, h, :n], dtype)
        for i, hh in enumerate((h, h // group, h // group)):
            want[i][r, b, :n, hh] += got[i]
            bound[i][r, b, :n, hh] += bounds[i]
    for g, x, e, name in zip(grads, want, bound, ("dq", "dk", "dv")):
        assert g.dtype == dtype, what
        assert_close(g, x, e + x.abs() * HALF[dtype] * 1.01 + tiny(dtype), f"{what} {name}")
        if counts is not None:
            for b in range(B):
                assert bool((g[:, b, max(0, min(SG, counts[b])):] == 0).all()), f"{what} {name} padding"
