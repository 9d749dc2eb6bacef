"""The activation operators in 64 bits, from their definitions (tests only).

Tensors are CPU tensors; layouts are the exchange's (P ``[w, B, S, H, D]``,
A ``[w, B, S*w, H/w, D]``).  Codes and scales are returned as the bytes that
the library stores.
"""
from __future__ import annotations

import torch

BLOCK = 32
FORMATS = {torch.float8_e4m3fn: (448.0, 8), torch.float8_e5m2: (57344.0, 15)}
# half a step relative to a value, by type
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24,
        torch.float8_e4m3fn: 2.0 ** -4, torch.float8_e5m2: 2.0 ** -3}


def to_a(x, w):
    j, B, S, H, d = x.shape
    out = x.new_empty(w, B, S * w, H // w, d)
    for r in range(w):
        for k in range(w):
            out[r, :, k * S:(k + 1) * S] = x[k, :, :, r * (H // w):(r + 1) * (H // w)]
    return out


def to_p(x, w):
    r, B, SG, hl, d = x.shape
    S = SG // w
    out = x.new_empty(w, B, S, hl * w, d)
    for k in range(w):
        for q in range(w):
            out[k, :, :, q * hl:(q + 1) * hl] = x[q, :, k * S:(k + 1) * S]
    return out


def quantise(v, fmt):
    """(code bytes, scale bytes) of values [..., D] (exact in float64)."""
    most, top = FORMATS[fmt]
    v = v.double()
    D = v.shape[-1]
    codes = torch.empty(v.shape, dtype=torch.uint8)
    scales = torch.empty(v.shape[:-1] + (-(-D // BLOCK),), dtype=torch.uint8)
    for b in range(scales.shape[-1]):
        x = v[..., b * BLOCK:(b + 1) * BLOCK]
        a = x.abs()
        m = torch.where(torch.isfinite(a), a, torch.zeros_like(a)).amax(-1, keepdim=True)
        frac, ex = torch.frexp(m)                               # m = frac * 2**ex, frac in [0.5, 1)
        k = ex.double() - 1 - top + (frac > 0.875)
        k = torch.where(m == 0, torch.full_like(k, -127.0), k.clamp_min(-127.0))
        assert bool((m <= most * torch.exp2(k)).all())
        assert bool(((m > most * torch.exp2(k - 1)) | (k == -127)).all())
        # x * 2**-k in 64 bits is exact; in 32 bits too unless it is far below the smallest code
        q = (x * torch.exp2(-k)).float()
        c = q.to(fmt).view(torch.uint8)
        # NaN has several bit patterns: one for all, with the sign
        nan = torch.isnan(c.view(fmt).float())
        codes[..., b * BLOCK:(b + 1) * BLOCK] = torch.where(nan, torch.full_like(c, 0x7f), c)
        scales[..., b] = (k + 127).squeeze(-1).to(torch.uint8)
    return codes, scales


def canonical(codes, fmt):
    """Code bytes with every NaN as 0x7f."""
    c = codes.view(torch.uint8)
    return torch.where(torch.isnan(c.view(fmt).float()), torch.full_like(c, 0x7f), c)


def dequantise(codes, scales, fmt):
    """float64 values of code and scale bytes."""
    D = codes.shape[-1]
    s = torch.exp2(scales.view(torch.uint8).double() - 127)
    return codes.view(torch.uint8).view(fmt).double() * s.repeat_interleave(BLOCK, -1)[..., :D]


def norm(x, weight, mode, w, residual=None, per_head=False, eps=1e-6):
    """(out, h, rstd) in float64; with a residual h is the sum in 32 bits rounded to x's type."""
    h = x if mode == 0 else to_p(x, w)
    if residual is not None:
        h = (h.float() + residual.float()).to(x.dtype)
    h = h.double()
    dims = (-1,) if per_head else (-2, -1)
    rstd = 1.0 / torch.sqrt(h.square().mean(dims, keepdim=True) + eps)
    y = h * rstd
    if weight is not None:
        y = y * (weight.double() if per_head else weight.double().view(h.shape[-2:]))
    rstd = rstd.reshape(h.shape[:4] if per_head else h.shape[:3])
    return (to_a(y, w) if mode == 0 else y), h, rstd


def norm_backward(dy, weight, mode, w, h, rstd, dsum=None, per_head=False):
    """(dx, dh, dweight) in float64; h in P layout, float64."""
    dy = (dy if mode == 1 else to_p(dy, w)).double()
    dims = (-1,) if per_head else (-2, -1)
    r = rstd.double()[..., None] if per_head else rstd.double()[..., None, None]
    n = h * r
    g = dy
    if weight is not None:
        g = dy * (weight.double() if per_head else weight.double().view(h.shape[-2:]))
    dh = r * (g - n * (g * n).mean(dims, keepdim=True))
    if dsum is not None:
        dh = dh + dsum.double()
    dw = (dy * n).sum((0, 1, 2, 3) if per_head else (0, 1, 2)).flatten()
    return (dh if mode == 0 else to_a(dh, w)), dh, dw


def cache_write(codes, scales, x, fmt, w, starts, counts, part):
    """Writes x (P layout) into the bytes of codes/scales in place."""
    n = len(starts)
    q, s = quantise(x, fmt)
    q, s = to_a(q, w), to_a(s, w)
    q = q.reshape(w, n, -1, *q.shape[-2:])
    s = s.reshape(w, n, -1, *s.shape[-2:])
    for i in range(n):
        for t in range(min(q.shape[2], counts[i])):
            pos = starts[i] + t
            if 0 <= pos < codes.shape[3]:
                codes[part, :, i, pos] = q[:, i, t]
                scales[part, :, i, pos] = s[:, i, t]


def cache_read(out, codes, scales, fmt, starts, counts, part):
    """Reads into out [w, n, tokens, hl, D] in place (out's type, largest finite value kept)."""
    most = torch.finfo(out.dtype).max
    for i in range(out.shape[1]):
        for t in range(min(out.shape[2], counts[i])):
            pos = starts[i] + t
            if 0 <= pos < codes.shape[3]:
                v = dequantise(codes[part, :, i, pos], scales[part, :, i, pos], fmt)
                fin = torch.isfinite(v)
                out[:, i, t] = torch.where(fin, v.clamp(-most, most), v).to(out.dtype)


# ---------------------------------------------------------------- tolerances
#
# A norm's sum of squares adds V * items <= 64 squares per lane, then joins
# <= 64 lanes and <= 16 waves: under 96 roundings of 2^-24 on positive terms,
# half of which reach rstd, and a few for its root, quotient and products: the
# result is off by less than 64 * 2^-24 = 2^-18, and by half a step of its type.
SUM = 2.0 ** -18


def tiny(dtype):
    """Half a step of the type's subnormals."""
    f = torch.finfo(dtype)
    return f.tiny * f.eps / 2


def assert_close(got, want, bound, what):
    got = got.double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    fine = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), what
    assert torch.equal(got[~fine & ~torch.isnan(want)], want[~fine & ~torch.isnan(want)]), what
    off = (got - want).abs()
    bad = fine & (off > bound)
    if bool(bad.any()):
        k = int(torch.where(bad, off / bound.clamp_min(1e-300), torch.zeros_like(off)).argmax())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} values off; worst {float(got.flatten()[k])!r} "
                             f"against {float(want.flatten()[k])!r}, bound {float(bound.flatten()[k]):.3g}")


def check_values(got, want, dtype, what, rel=SUM):
    """A result rounded once to its type from a value off by `rel`."""
    assert got.dtype == dtype, what
    assert_close(got, want, want.abs() * (HALF[dtype] * (1 + rel) + rel) + tiny(dtype), what)


def check_codes(codes, scales, want, fmt, what, rel=SUM):
    """8 bits of values off by `rel`: the scale is the right one for a largest
    magnitude that far off, the codes' values within half a step (of the
    format's smallest values too) of it."""
    most, _ = FORMATS[fmt]
    D = want.shape[-1]
    s = torch.exp2(scales.view(torch.uint8).double() - 127)
    nb = -(-D // BLOCK)
    assert scales.shape[-1] == nb, what
    for b in range(nb):
        m = want[..., b * BLOCK:(b + 1) * BLOCK].abs().amax(-1)
        sb = s[..., b]
        assert bool((m * (1 - rel) <= most * sb).all()), (what, "overflows")
        assert bool(((m * (1 + rel) > most * sb / 2) | (scales.view(torch.uint8)[..., b] == 0)).all()), (what, "scale")
    sv = s.repeat_interleave(BLOCK, -1)[..., :D]
    step = sv * float(torch.finfo(fmt).tiny) * HALF[fmt]        # half a step of the subnormals
    got = dequantise(codes, scales, fmt)
    assert_close(got, want, want.abs() * (HALF[fmt] * (1 + rel) + rel) + step, what)


def check_same_codes(codes, scales, values, fmt, what):
    """8 bits of values that are given exactly: the same bytes."""
    q, s = quantise(values, fmt)
    assert torch.equal(scales.view(torch.uint8), s), (what, "scales")
    assert torch.equal(canonical(codes, fmt), canonical(q, fmt)), (what, "codes")


def check_backward(dx, dh, dw, want, parts, dtype, mode, w, what):
    """Gradients against norm_backward's: cancellation in g - n * mean is
    bounded by its terms (`parts` = rstd * (|g| + |n| * mean|g n|) + |dsum|,
    P layout, and sum |dy n| of dweight)."""
    rdx, rdh, rdw = want
    terms, wterms = parts
    bound = rdh.abs() * HALF[dtype] + terms * SUM + tiny(dtype)
    assert dx.dtype == dtype, what
    assert_close(dx, rdx, bound if mode == 0 else to_a(bound, w), what + " dx")
    if dh is not None:
        assert_close(dh, rdh, bound, what + " dresidual")
    if dw is not None:
        # under 2^8 additions in a row for the tests' rows
        assert_close(dw, rdw, wterms * 2.0 ** -16 + 1e-30, what + " dweight")


def backward_terms(dy, weight, mode, w, h, rstd, dsum=None, per_head=False):
    dy = (dy if mode == 1 else to_p(dy, w)).double()
    r = rstd.double()[..., None] if per_head else rstd.double()[..., None, None]
    n = h * r
    g = dy
    if weight is not None:
        g = dy * (weight.double() if per_head else weight.double().view(h.shape[-2:]))
    terms = r * (g.abs() + n.abs() * (g * n).abs().mean((-1,) if per_head else (-2, -1), keepdim=True))
    if dsum is not None:
        terms = terms + dsum.double().abs()
    return terms, (dy * n).abs().sum((0, 1, 2, 3) if per_head else (0, 1, 2)).flatten()
