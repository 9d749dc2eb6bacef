"""GPU: norms joined with the exchange (forward, backward, 8-bit output and
checkpoint) and the 8-bit cache, against their definitions in 64 bits."""
from __future__ import annotations

import sys

import pytest
import torch

import ulysses_all_re_amd as ua
from tests import act_reference as ref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


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


def values(shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype)


def dev(t):
    return None if t is None else t.to(DEV)


def cpu(t):
    if t is None:
        return None
    return t.view(torch.uint8).cpu() if "float8" in str(t.dtype) else t.cpu()


SHAPES = [(1, 1, 1, 1, 8), (2, 1, 5, 8, 128), (5, 1, 9, 5, 32), (1, 1, 7, 10, 128), (2, 1, 8, 4, 16), (3, 2, 5, 6, 40), (2, 1, 3, 4, 7), (5, 1, 4, 10, 2), (1, 2, 3, 5, 33),
          (4, 2, 7, 8, 80), (2, 1, 3, 6, 128), (2, 1, 2, 12, 128), (2, 1, 2, 32, 128), (8, 1, 3, 40, 128),
          (1, 1, 2, 96, 128), (1, 1, 2, 256, 128), (2, 1, 1, 60, 7), (4, 1, 700, 8, 64), (3, 2, 211, 12, 80),
          (1, 1, 1, 1, 8191), (2, 1, 3, 2, 640), (1, 2, 2, 3, 1000)]


def check_norm(plan, mode, per_head, with_res, weight_type, out_fmt, save, seed=0, scale=3.0):
    """One forward call and the backward call that goes with it."""
    w, B, S, H, D = plan.w, plan.B, plan.S_local, plan.H, plan.D
    dtype = plan.dtype
    what = f"{(w, B, S, H, D)} {dtype} mode {mode} head {per_head} residual {with_res} weight {weight_type} " \
           f"out {out_fmt} save {save}"
    note(what)
    n = D if per_head else H * D
    x = values(plan.in_shape(mode), dtype, 10 + seed, scale)
    res = values(plan.in_shape(0), dtype, 20 + seed) if with_res else None
    weight = None if weight_type is None else values((n,), weight_type, 30 + seed)
    r = plan.norm_exchange(dev(x), dev(weight), mode, residual=dev(res), per_head=per_head, out_dtype=out_fmt,
                           checkpoint=save, rstd=True)
    torch.cuda.synchronize()
    y, h, rstd = ref.norm(x, weight, mode, w, res, per_head)
    rs = cpu(r.rstd)
    ref.check_values(rs, rstd, torch.float32, what)
    if with_res:
        assert torch.equal(cpu(r.sum).double(), h), what
    else:
        assert r.sum is None
    if out_fmt:
        assert r.out.dtype == out_fmt and r.scales.dtype == torch.float8_e8m0fnu
        ref.check_codes(cpu(r.out), cpu(r.scales), y, out_fmt, what)
    else:
        ref.check_values(cpu(r.out), y, dtype, what)
    if save:
        assert r.saved.dtype == save
        ref.check_same_codes(cpu(r.saved), cpu(r.saved_scales), h, save, what)
    dy = values(plan.out_shape(mode), dtype, 40 + seed)
    dsum = values(plan.in_shape(0), dtype, 50 + seed) if with_res else None
    if save:
        hq, saved = ref.dequantise(cpu(r.saved), cpu(r.saved_scales), save), r.saved
    else:
        hq, saved = h, (r.sum if with_res else dev(x))
    b = plan.norm_exchange_backward(dev(dy), dev(weight), mode, saved, r.rstd, saved_scales=r.saved_scales,
                                    dsum=dev(dsum), residual=with_res, per_head=per_head)
    torch.cuda.synchronize()
    want = ref.norm_backward(dy, weight, mode, w, hq, rs, dsum, per_head)
    parts = ref.backward_terms(dy, weight, mode, w, hq, rs, dsum, per_head)
    if with_res and mode == 0:
        assert b.dresidual is b.dx
    ref.check_backward(cpu(b.dx), cpu(b.dresidual) if with_res and mode == 1 else None, cpu(b.dweight), want, parts,
                       dtype, mode, w, what)
    assert (b.dweight is None) == (weight is None)
    return r, b


@pytest.mark.parametrize("t", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_norm_and_backward(shape, t):
    dtype = TYPES[t]
    plan = ua.Plan(*shape, dtype, device=DEV)
    check_norm(plan, 0, False, False, dtype, None, E4M3)
    check_norm(plan, 1, False, True, torch.float32, E4M3, E5M2, 1)
    check_norm(plan, 0, True, True, dtype, E5M2, None, 2)
    check_norm(plan, 1, True, False, None, None, None, 3)
    check_norm(plan, 1, False, False, dtype, None, None, 4)
    check_norm(plan, 0, True, False, torch.float32, None, E5M2, 5)
    plan.close()


def test_long_norms():
    """Norms of more lanes' worth of values than a workgroup of 256 holds, up to the longest."""
    for shape, t in [((2, 1, 3, 128, 128), "bf16"), ((1, 1, 3, 512, 128), "fp16"), ((1, 1, 2, 1, 65536), "bf16"),
                     ((2, 1, 2, 128, 256), "fp32"), ((1, 1, 1, 64, 127), "fp32")]:
        plan = ua.Plan(*shape, TYPES[t], device=DEV)
        check_norm(plan, 0, False, False, TYPES[t], None, E4M3)
        check_norm(plan, 1, False, True, TYPES[t], None, None, 1)
        check_norm(plan, 0, True, True, torch.float32, E5M2, E4M3, 2)
        plan.close()


CACHES = [(1, 1, 1, 1, 8, 1, 4), (2, 2, 4, 4, 16, 2, 11), (4, 1, 3, 8, 80, 12, 5), (2, 3, 2, 4, 7, 3, 6),
          (3, 1, 4, 6, 40, 4, 9), (2, 1, 8, 4, 33, 1, 30), (8, 1, 4, 8, 128, 32, 40), (2, 2, 100, 4, 128, 2, 231),
          (2, 2, 50, 4, 72, 50, 7)]


@pytest.mark.parametrize("t", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("c", CACHES, ids=lambda s: "x".join(map(str, s)))
def test_cache(c, t):
    """Starts before, inside and past the cache, counts of zero, one and more
    than there are; rows that nothing names stay as they were."""
    w, B, S, H, D, seqs, cap = c
    dtype = TYPES[t]
    nb = -(-D // 32)
    g = torch.Generator().manual_seed(7)
    each = B * S * w // seqs
    plan = ua.Plan(w, B, S, H, D, dtype, device=DEV)
    for k, fmt in enumerate((E4M3, E5M2)):
        note(f"cache {c} {t} {fmt}")
        codes = torch.randint(0, 120, (2, w, seqs, cap, H // w, D), generator=g, dtype=torch.uint8)
        scales = torch.randint(120, 130, (2, w, seqs, cap, H // w, nb), generator=g, dtype=torch.uint8)
        cache = ua.Cache.of(codes.to(DEV).view(fmt), scales.to(DEV).view(torch.float8_e8m0fnu))
        starts = torch.randint(-3, cap + 2, (seqs,), generator=g, dtype=torch.int32)
        counts = torch.randint(-1, each + 3, (seqs,), generator=g, dtype=torch.int32) if k else None
        kk, vv = values(plan.in_shape(0), dtype, 60 + k), values(plan.in_shape(0), dtype, 70 + k, 100.0)
        plan.cache_write(cache, dev(kk), dev(vv), dev(starts), dev(counts))
        torch.cuda.synchronize()
        cnt = counts.tolist() if k else [each] * seqs
        for part, x in ((0, kk), (1, vv)):
            ref.cache_write(codes, scales, x, fmt, w, starts.tolist(), cnt, part)
        assert bool((cpu(cache.codes) == codes).all()) and bool((cpu(cache.scales) == scales).all())
        n = min(cap, 5)
        want = [torch.full((w, seqs, n, H // w, D), 3.0, dtype=dtype) for _ in range(2)]
        outs = plan.cache_read(cache, n, dev(starts), dev(counts), out=tuple(dev(o) for o in want))
        torch.cuda.synchronize()
        for part in (0, 1):
            ref.cache_read(want[part], codes, scales, fmt, starts.tolist(), counts.tolist() if k else [n] * seqs, part)
            assert bool((cpu(outs[part]) == want[part]).all())
    plan.close()


def special(dtype, D=96):
    x = torch.zeros(1, 1, 1, 2, D)
    f = torch.finfo(dtype)
    x[..., 0, :5] = torch.tensor([float("nan"), float("inf"), float("-inf"), 1.0, f.min])
    x[..., 0, 32:36] = torch.tensor([f.tiny * f.eps, -f.tiny, f.tiny * 3, 0.0])
    x[..., 0, 64:68] = torch.tensor([f.max, f.min, f.max * 0.9, 1e-3])
    x[..., 1, :3] = torch.tensor([448.0, 449.0, 0.25])       # borders of the scales
    x[..., 1, 32:35] = torch.tensor([57344.0, 57000.0, -1.0])
    x[..., 1, 64:70] = torch.tensor([1.75, 1.0625, 1.1875, -1.0625, 0.03125, 2.0 ** -11])    # ties
    return x.to(dtype)


@pytest.mark.parametrize("t", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("fmt", [E4M3, E5M2], ids=["e4m3", "e5m2"])
def test_special_values_in_8_bits(t, fmt):
    """NaN, infinities, zeros, subnormals, the largest values, borders and ties:
    the same bytes as the definition, and what they read back as."""
    dtype = TYPES[t]
    x = special(dtype)
    plan = ua.Plan(1, 1, 1, 2, 96, dtype, device=DEV)
    cache = ua.Cache(1, 2, 96, 1, 2, fmt, DEV)
    starts = torch.tensor([1], dtype=torch.int32)
    plan.cache_write(cache, dev(x), None, dev(starts))
    torch.cuda.synchronize()
    ref.check_same_codes(cpu(cache.codes)[0, :, :, 1:], cpu(cache.scales)[0, :, :, 1:], x.view(1, 1, 1, 2, 96), fmt, t)
    assert int(cpu(cache.codes)[1].sum()) == 0 and int(cpu(cache.codes)[0, :, :, 0].sum()) == 0
    k, v = plan.cache_read(cache, 2)
    want = torch.zeros(1, 1, 2, 2, 96, dtype=dtype)
    ref.cache_read(want, cpu(cache.codes), cpu(cache.scales), fmt, [0], [2], 0)
    got = cpu(k)
    assert torch.equal(got.nan_to_num(123.0, 1.0, -1.0), want.nan_to_num(123.0, 1.0, -1.0))
    assert torch.equal(torch.isinf(got), torch.isinf(want))
    plan.close()


@pytest.mark.parametrize("per_head", [False, True], ids=["token", "head"])
@pytest.mark.parametrize("t,size,eps", [("fp16", 2.0 ** -18, 2.0 ** -38), ("bf16", 2.0 ** -64, 2.0 ** -126),
                                        ("fp32", 2.0 ** -64, 2.0 ** -126)], ids=["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("D", [64, 33])
def test_norms_of_the_smallest_values(t, size, eps, per_head, D):
    """Values that are fp16's subnormals, or whose squares are fp32's, beside
    an eps of their size.  A square's subnormal step is 2^-149, at most 2^-24
    of mean + eps with its rounding, which the tolerance's 2^-18 holds."""
    dtype = TYPES[t]
    plan = ua.Plan(2, 1, 3, 4, D, dtype, device=DEV)
    n = D if per_head else 4 * D
    x, weight = values(plan.in_shape(0), dtype, 1, size), values((n,), dtype, 2)
    y, h, rstd = ref.norm(x, weight, 0, 2, None, per_head, eps)
    r = plan.norm_exchange(dev(x), dev(weight), 0, per_head=per_head, eps=eps, rstd=True)
    torch.cuda.synchronize()
    ref.check_values(cpu(r.rstd), rstd, torch.float32, t)
    ref.check_values(cpu(r.out), y, dtype, t)
    dy = values(plan.out_shape(0), dtype, 3, 2.0 ** -12)
    b = plan.norm_exchange_backward(dev(dy), dev(weight), 0, dev(x), r.rstd, per_head=per_head)
    torch.cuda.synchronize()
    rs = cpu(r.rstd)
    ref.check_backward(cpu(b.dx), None, cpu(b.dweight), ref.norm_backward(dy, weight, 0, 2, h, rs, None, per_head),
                       ref.backward_terms(dy, weight, 0, 2, h, rs, None, per_head), dtype, 0, 2, t)
    plan.close()


@pytest.mark.parametrize("save", [None, E4M3, E5M2], ids=["values", "e4m3", "e5m2"])
@pytest.mark.parametrize("up", [50, -50])
@pytest.mark.parametrize("t", ["bf16", "fp32"])
@pytest.mark.parametrize("mode,per_head", [(0, False), (1, True)], ids=["token", "head"])
def test_backward_of_values_far_from_one(mode, per_head, t, up, save):
    """Values of 2^50 with gradients of 2^90, and of 2^-50 with 2^-90: every
    result lies well within 32 bits, the products h * dy do not."""
    dtype = TYPES[t]
    plan = ua.Plan(2, 1, 5, 4, 64, dtype, device=DEV)
    eps = 2.0 ** -106
    n = 64 if per_head else 4 * 64
    x, weight = values(plan.in_shape(mode), dtype, 1, 2.0 ** up), values((n,), dtype, 2)
    dy = values(plan.out_shape(mode), dtype, 3, 2.0 ** (90 if up > 0 else -90))
    _, h, _ = ref.norm(x, weight, mode, 2, None, per_head, eps)
    r = plan.norm_exchange(dev(x), dev(weight), mode, per_head=per_head, eps=eps, rstd=True, checkpoint=save)
    b = plan.norm_exchange_backward(dev(dy), dev(weight), mode, r.saved if save else dev(x), r.rstd,
                                    saved_scales=r.saved_scales if save else None, per_head=per_head)
    torch.cuda.synchronize()
    rs = cpu(r.rstd)
    if save:
        h = ref.dequantise(cpu(r.saved), cpu(r.saved_scales), save)
    want = ref.norm_backward(dy, weight, mode, 2, h, rs, None, per_head)
    assert all(bool(torch.isfinite(v).all()) for v in want)
    ref.check_backward(cpu(b.dx), None, cpu(b.dweight), want, ref.backward_terms(dy, weight, mode, 2, h, rs, None, per_head),
                       dtype, mode, 2, t)
    plan.close()
