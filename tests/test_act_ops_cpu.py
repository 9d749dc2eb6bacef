"""The norm operator's and the activation calls' host side: shapes of fake
tensors, refusals, the cache object.  No GPU needed."""
from __future__ import annotations

import os
import re
import subprocess

import pytest
import torch

import ulysses_all_re_amd as ua
from tests.test_binding_cpu import _host_plan
from ulysses_all_re_amd import activations, ops

E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2
HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "ua2a_act.h")


def test_header_binding_and_library_agree():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    declared = sorted(set(re.findall(r"^\s*int\s+(ua2a_\w+)\s*\(", text, flags=re.M)))
    assert declared == sorted(activations.EXPORTED)
    syms = subprocess.check_output(["nm", "-D", "--defined-only", ua.LIBRARY], text=True)
    exported = {line.split()[-1] for line in syms.splitlines() if " T " in line}
    assert set(declared) <= exported


def test_header_is_plain_c():
    code = '#include "ua2a_act.h"\nint main(void) { ua2a_norm_t n; ua2a_cache_t c; (void)n; (void)c; return UA2A_BLOCK - 32; }\n'
    cmd = ["gcc", "-std=c99", "-Wall", "-Wextra", "-pedantic", "-Werror", "-fsyntax-only", "-x", "c", "-I",
           os.path.dirname(HEADER), "-"]
    subprocess.run(cmd, input=code, text=True, check=True, timeout=60)


@pytest.mark.parametrize("per_head", [False, True])
@pytest.mark.parametrize("w,B,S,H,D", [(2, 1, 8, 4, 16), (8, 1, 9450, 40, 128), (3, 2, 4681, 12, 80)])
def test_fake_shapes(w, B, S, H, D, per_head):
    p, a = (w, B, S, H, D), (w, B, S * w, H // w, D)
    n = D if per_head else H * D
    x = torch.empty(p, device="meta", dtype=torch.bfloat16)
    weight = torch.empty(n, device="meta", dtype=torch.float32)
    y = ops.norm_all_to_all_4D(x, weight, 2, 1, w, per_head=per_head)
    assert y.shape == a and y.dtype == x.dtype
    z, total = ops.norm_all_to_all_4D(y, None, 1, 2, w, residual=x, per_head=per_head)
    assert z.shape == p and total.shape == p and total.dtype == x.dtype
    (codes, scales), total = ops.norm_all_to_all_4D(y, weight, 1, 2, w, residual=x, per_head=per_head, out_dtype=E4M3)
    assert codes.shape == p and codes.dtype == E4M3 and total.shape == p
    assert scales.shape == p[:-1] + (-(-D // 32),) and scales.dtype == torch.float8_e8m0fnu
    r = ops.norm_exchange(x, weight, None, w, 0, per_head, 1e-6, 0, 2)
    assert r[3].shape == p and r[3].dtype == E5M2 and r[5].shape == (p[:4] if per_head else p[:3])
    dx, dres, dw = ops.norm_exchange_backward(z, weight, x, None, r[5], z, w, 1, per_head, True, True)
    assert dx.shape == a and dres.shape == p and dw.shape == (n,) and dw.dtype == torch.float32


def test_gradients_have_shapes_on_fake_tensors():
    x = torch.empty((2, 1, 8, 4, 16), device="meta", requires_grad=True)
    res = torch.empty((2, 1, 8, 4, 16), device="meta", requires_grad=True)
    weight = torch.empty(16, device="meta", requires_grad=True)
    y, total = ops.norm_all_to_all_4D(x, weight, 2, 1, 2, residual=res, per_head=True, checkpoint=E4M3)
    (y.sum() + total.sum()).backward()
    assert x.grad.shape == x.shape and res.grad.shape == res.shape and weight.grad.shape == weight.shape


def test_operator_refusals():
    x = torch.empty((2, 1, 8, 4, 16), device="meta")
    with pytest.raises(ValueError, match="unsupported"):
        ops.norm_all_to_all_4D(x, None, 3, 1, 2)
    with pytest.raises(ValueError):
        ops.norm_all_to_all_4D(torch.empty((3, 1, 8, 4, 16), device="meta"), None, 2, 1, 2)
    with pytest.raises(ValueError, match="weight has shape"):
        ops.norm_all_to_all_4D(x, torch.empty(16, device="meta"), 2, 1, 2)
    with pytest.raises(ValueError, match="weight has shape"):
        ops.norm_all_to_all_4D(x, torch.empty(64, device="meta"), 2, 1, 2, per_head=True)
    with pytest.raises(ValueError, match="residual has shape"):
        ops.norm_all_to_all_4D(x, None, 2, 1, 2, residual=torch.empty((2, 1, 16, 2, 16), device="meta"))
    with pytest.raises(TypeError, match="residual has dtype"):
        ops.norm_all_to_all_4D(x, None, 2, 1, 2, residual=x.half())
    with pytest.raises(TypeError, match="checkpoint"):
        ops.norm_all_to_all_4D(x, None, 2, 1, 2, checkpoint=torch.int8)
    with pytest.raises(TypeError, match="out_dtype"):
        ops.norm_all_to_all_4D(x, None, 2, 1, 2, out_dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="no gradient"):
        ops.norm_all_to_all_4D(x.clone().requires_grad_(), None, 2, 1, 2, out_dtype=E4M3)
    with pytest.raises(RuntimeError, match="GPU only"):
        ops.norm_all_to_all_4D(torch.zeros((2, 1, 8, 4, 16)), None, 2, 1, 2)


def _plan():
    return _host_plan(w=2, B=1, S=4, H=4, D=16)


def test_plan_refusals():
    plan = _plan()
    p, a = plan.in_shape(0), plan.in_shape(1)
    x = torch.zeros(p, dtype=torch.bfloat16)
    rstd = torch.zeros(p[:3])
    bad = [
        (ValueError, dict(mode=2), {}),
        (TypeError, dict(x=x.float()), {}),
        (ValueError, dict(x=torch.zeros(a, dtype=torch.bfloat16)), {}),
        (ValueError, dict(x=x.transpose(2, 3).contiguous().transpose(2, 3)), {}),
        (ValueError, dict(weight=torch.zeros(16, dtype=torch.bfloat16)), {}),
        (TypeError, dict(weight=torch.zeros(64, dtype=torch.float16)), {}),
        (TypeError, dict(weight=torch.zeros(64, dtype=torch.int32)), {}),
        (ValueError, dict(weight=torch.zeros(128, dtype=torch.bfloat16)[::2]), {}),
        (ValueError, {}, dict(residual=torch.zeros(a, dtype=torch.bfloat16))),
        (TypeError, {}, dict(out_dtype=torch.bfloat16)),
        (TypeError, {}, dict(checkpoint=torch.float8_e4m3fnuz)),
        (ValueError, {}, dict(out=ua.NormExchange(None))),
        (TypeError, {}, dict(out=ua.NormExchange(torch.zeros(a)))),
        (ValueError, {}, dict(out=ua.NormExchange(torch.zeros(a, dtype=torch.bfloat16)), rstd=True)),
    ]
    for kind, first, kw in bad:
        args = dict(x=x, weight=None, mode=0)
        args.update(first)
        with pytest.raises(kind):
            plan.norm_exchange(args["x"], args["weight"], args["mode"], **kw)
    dy = torch.zeros(a, dtype=torch.bfloat16)
    for kind, args, kw in [
            (ValueError, (dy, None, 2, x, rstd), {}),
            (ValueError, (x, None, 0, x, rstd), {}),
            (ValueError, (dy, None, 0, dy, rstd), {}),
            (TypeError, (dy, None, 0, x, rstd.double()), {}),
            (ValueError, (dy, None, 0, x, rstd), dict(per_head=True)),
            (ValueError, (dy, None, 0, x, rstd), dict(dsum=x)),                  # a sum without a residual
            (TypeError, (dy, None, 0, x, rstd), dict(saved_scales=torch.zeros(p[:4] + (1,), dtype=torch.uint8))),
            (ValueError, (dy, None, 0, x.to(E4M3), rstd), dict(saved_scales=torch.zeros(p[:4] + (2,), dtype=torch.uint8))),
            (TypeError, (dy, None, 0, x.to(E4M3), rstd), {}),
    ]:
        with pytest.raises(kind):
            plan.norm_exchange_backward(*args, **kw)
    plan.close()
    with pytest.raises(ua.UA2AError):
        plan.norm_exchange(x, None, 0, out=ua.NormExchange(torch.zeros(a, dtype=torch.bfloat16)),
                           stream=_Stream())


class _Stream:
    """Stands for a stream where nothing is launched."""
    cuda_stream = 0


def test_plans_of_other_types_have_no_norms():
    plan = _host_plan(w=2, B=1, S=4, H=4, D=16, dtype=torch.int32)
    with pytest.raises(TypeError, match="bfloat16"):
        plan.norm_exchange(torch.zeros(plan.in_shape(0), dtype=torch.int32), None, 0)
    plan.close()


def test_cache_object_and_refusals():
    cache = ua.Cache(2, 4, 40, 3, 7, device="cpu")
    assert cache.codes.shape == (2, 2, 3, 7, 2, 40) and cache.scales.shape == (2, 2, 3, 7, 2, 2)
    assert cache.codes.dtype == E4M3 and cache.scales.dtype == torch.float8_e8m0fnu
    with pytest.raises(AttributeError):                 # its library struct holds their addresses
        cache.codes = cache.codes.clone()
    for args in [(2, 3, 16, 1, 1), (0, 4, 16, 1, 1), (2, 4, 16, 0, 1), (2, 4, 16, 1, 0), (2, 4, 0, 1, 1)]:
        with pytest.raises(ValueError):
            ua.Cache(*args, device="cpu")
    with pytest.raises(TypeError):
        ua.Cache(2, 4, 16, 1, 1, torch.bfloat16, "cpu")
    codes, scales = cache.codes, cache.scales
    with pytest.raises(TypeError):
        ua.Cache.of(codes.view(torch.uint8), scales)
    with pytest.raises(TypeError):
        ua.Cache.of(codes, scales.view(torch.float8_e4m3fn))
    with pytest.raises(ValueError):
        ua.Cache.of(codes[0], scales[0])
    with pytest.raises(ValueError):
        ua.Cache.of(codes, scales[..., :1])
    with pytest.raises(ValueError):
        ua.Cache.of(codes[:, :, :, ::2], scales[:, :, :, ::2])
    plan = _plan()
    k = torch.zeros(plan.in_shape(0), dtype=torch.bfloat16)
    good = ua.Cache(2, 4, 16, 8, 5, device="cpu")
    starts = torch.zeros(8, dtype=torch.int32)
    for kind, args in [
            (ValueError, (cache, k, k, starts)),                                 # other heads
            (ValueError, (good, None, None, starts)),
            (ValueError, (good, k, k, None)),
            (TypeError, (good, k, k, starts.long())),
            (ValueError, (good, k, k, starts[:4])),
            (TypeError, (good, k.float(), k, starts)),
            (ValueError, (good, k, k[:1], starts)),
            (TypeError, (good, k, k, starts, starts.long())),
    ]:
        with pytest.raises(kind):
            plan.cache_write(*args)
    out = torch.zeros(2, 8, 3, 2, 16, dtype=torch.bfloat16)
    for kind, args, kw in [
            (ValueError, (good, 0), {}), (ValueError, (good, 3), dict(out=(None, None))),
            (ValueError, (good, 4), dict(out=(out, None))), (TypeError, (good, 3), dict(out=(out.float(), None))),
            (ValueError, (good, 3), dict(out=(out,))), (TypeError, (good, 3, starts.float()), {})]:
        with pytest.raises(kind):
            plan.cache_read(*args, **kw)
    plan.close()
