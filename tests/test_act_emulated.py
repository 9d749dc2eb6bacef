"""The activation operators' host code and index math on the CPU: every launch
is carried out lane by lane on host memory (tests/emu/act_backend.cpp), each
access checked against its buffer, and the results compared with the
definition in 64 bits.  Then the refusals: what the calls must turn down."""
from __future__ import annotations

import ctypes

import pytest
import torch

import ulysses_all_re_amd as ua
from tests import act_reference as ref
from tests.emu import act_build
from ulysses_all_re_amd.activations import ua2a_cache_t, ua2a_norm_grad_t, ua2a_norm_t

E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2
TYPES = {"bf16": (torch.bfloat16, 0), "fp16": (torch.float16, 1), "fp32": (torch.float32, 2)}
FORMAT = {None: 0, E4M3: 1, E5M2: 2}


@pytest.fixture(scope="module")
def lib():
    so = ctypes.CDLL(act_build.build())
    i32, i64, vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p
    so.ua2a_plan.argtypes = [ctypes.POINTER(vp), i32, i64, i64, i64, i64, i32, i32, vp, i64, i32]
    so.ua2a_destroy.argtypes = [vp]
    so.ua2a_act_emu_last.argtypes = [i32]
    return ua.declare_activation_signatures(so)


class Plan:
    def __init__(self, lib, w, B, S, H, D, dtype, device=0):
        self.lib, self.shape, self.dtype = lib, (w, B, S, H, D), dtype
        self.h = ctypes.c_void_p()
        e = torch.empty((), dtype=dtype).element_size()
        assert lib.ua2a_plan(ctypes.byref(self.h), w, B, S, H, D, e, 0, None, 0, device) == 0

    def __enter__(self):
        self.lib.ua2a_act_emu_reset()
        return self

    def __exit__(self, *a):
        self.lib.ua2a_destroy(self.h)

    @property
    def p(self):
        return self.shape

    @property
    def a(self):
        w, B, S, H, D = self.shape
        return (w, B, S * w, H // w, D)


def ptr(t):
    return None if t is None else t.data_ptr()


def values(shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype)


def run_norm(lib, plan, x, weight, mode, residual=None, per_head=False, out_fmt=None, save=None, rstd=True, eps=1e-6):
    w, B, S, H, D = plan.shape
    nb = -(-D // 32)
    oshape = plan.a if mode == 0 else plan.p
    out = torch.full(oshape, 99, dtype=torch.uint8) if out_fmt else torch.full(oshape, 7.0, dtype=plan.dtype)
    osc = torch.full(oshape[:-1] + (nb,), 99, dtype=torch.uint8) if out_fmt else None
    total = torch.zeros(plan.p, dtype=plan.dtype) if residual is not None else None
    saved = torch.full(plan.p, 99, dtype=torch.uint8) if save else None
    ssc = torch.full(plan.p[:-1] + (nb,), 99, dtype=torch.uint8) if save else None
    rs = torch.zeros((w, B, S, H) if per_head else (w, B, S)) if rstd else None
    wt = 0 if weight is None else [c for d, c in TYPES.values() if d == weight.dtype][0]
    args = ua2a_norm_t(ptr(x), ptr(residual), ptr(weight), ptr(out), ptr(osc), ptr(total), ptr(saved), ptr(ssc), ptr(rs),
                       eps, [c for d, c in TYPES.values() if d == plan.dtype][0], wt, int(per_head), FORMAT[out_fmt],
                       FORMAT[save])
    rc = lib.ua2a_norm_exchange(plan.h, mode, ctypes.byref(args), None)
    assert rc == 0, rc
    assert lib.ua2a_act_emu_error() == 0
    return out, osc, total, saved, ssc, rs


# (w, B, S, H, D): one lane to several workgroups' worth of slots, heads that
# are no multiple of a block or of 16 bytes, one token, long norms
SHAPES = [(1, 1, 1, 1, 8), (2, 1, 5, 8, 128), (5, 1, 9, 5, 32), (1, 1, 7, 10, 128), (2, 1, 8, 4, 16), (3, 2, 5, 6, 40), (2, 1, 3, 4, 7), (5, 1, 4, 10, 2), (1, 2, 3, 5, 33),
          (4, 2, 7, 8, 80), (2, 1, 3, 6, 128), (2, 1, 2, 12, 128), (2, 1, 2, 32, 128), (8, 1, 3, 40, 128),
          (1, 1, 2, 96, 128), (1, 1, 2, 256, 128), (2, 1, 1, 60, 7), (2, 1, 3, 2, 640), (1, 2, 2, 3, 1000)]


@pytest.mark.parametrize("t", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_norm_and_backward(lib, shape, t):
    dtype, _ = TYPES[t]
    w, B, S, H, D = shape
    for case, (mode, per_head, with_res, out_fmt, save) in enumerate([
            (0, False, False, None, E4M3), (1, False, True, E4M3, E5M2), (0, True, True, E5M2, None),
            (1, True, False, None, None)]):
        with Plan(lib, *shape, dtype) as plan:
            n = D if per_head else H * D
            x = values(plan.p if mode == 0 else plan.a, dtype, 10 + case, 3.0)
            res = values(plan.p, dtype, 20 + case) if with_res else None
            weight = [None, values((n,), dtype, 30), values((n,), torch.float32, 31), values((n,), dtype, 32)][case]
            out, osc, total, saved, ssc, rs = run_norm(lib, plan, x, weight, mode, res, per_head, out_fmt, save)
            y, h, rstd = ref.norm(x, weight, mode, w, res, per_head)
            what = f"{shape} {t} case {case}"
            ref.check_values(rs, rstd, torch.float32, what)
            if with_res:
                assert torch.equal(total.double(), h), what
            if out_fmt:
                ref.check_codes(out, osc, y, out_fmt, what)
            else:
                ref.check_values(out, y, dtype, what)
            if save:
                ref.check_same_codes(saved, ssc, h, save, what)
            # and back
            dy = values(plan.a if mode == 0 else plan.p, dtype, 40 + case)
            dsum = values(plan.p, dtype, 50 + case) if with_res else None
            if save:
                hq = ref.dequantise(saved, ssc, save)
                sv, sg = saved, 0
            else:
                hq, sv, sg = h, (total if with_res else x), int(mode == 1 and not with_res)
            dx = torch.zeros_like(x)
            dres = torch.zeros(plan.p, dtype=dtype) if with_res and mode == 1 else None
            dw = torch.zeros(n) if weight is not None else None
            need = ctypes.c_int64()
            assert lib.ua2a_norm_workspace(plan.h, int(per_head), ctypes.byref(need)) == 0
            space = torch.zeros(need.value // 4) if weight is not None else None
            code = TYPES[t][1]
            wt = 0 if weight is None else [c for d, c in TYPES.values() if d == weight.dtype][0]
            args = ua2a_norm_grad_t(ptr(dy), ptr(dsum), ptr(sv), ptr(ssc), ptr(weight), ptr(rs), ptr(dx), ptr(dres),
                                    ptr(dw), ptr(space), need.value, code, wt, int(per_head), FORMAT[save], sg)
            assert lib.ua2a_norm_exchange_backward(plan.h, mode, ctypes.byref(args), None) == 0
            assert lib.ua2a_act_emu_error() == 0
            want = ref.norm_backward(dy, weight, mode, w, hq, rs, dsum, per_head)
            parts = ref.backward_terms(dy, weight, mode, w, hq, rs, dsum, per_head)
            ref.check_backward(dx, dres, dw, want, parts, dtype, mode, w, what)


def test_misaligned_tensors_take_single_values(lib):
    """A tensor that starts off a 16-byte boundary is moved value by value."""
    shape, dtype = (2, 1, 4, 4, 16), torch.bfloat16
    with Plan(lib, *shape, dtype) as plan:
        x = values((2 * 4 * 4 * 16 + 1,), dtype, 1)[1:].view(plan.p)
        assert x.data_ptr() % 16 != 0
        out, *_ = run_norm(lib, plan, x, None, 0)
        assert lib.ua2a_act_emu_last(0) == 1
        y, _, _ = ref.norm(x, None, 0, 2)
        ref.check_values(out, y, dtype, "offset")


def test_special_values_in_8_bits(lib):
    """NaN, infinities, zeros, subnormal and largest values, by block."""
    dtype = torch.float32
    w, B, S, H, D = 1, 1, 1, 1, 96
    x = torch.zeros(1, 1, 1, 1, 96)
    x[..., :5] = torch.tensor([float("nan"), float("inf"), float("-inf"), 1.0, -3e38])
    x[..., 32:36] = torch.tensor([2.0 ** -140, -2.0 ** -149, 2.0 ** -127, 0.0])
    for fmt in (E4M3, E5M2):
        codes, scales = torch.zeros(2, 1, 1, 2, 1, 96, dtype=torch.uint8), torch.zeros(2, 1, 1, 2, 1, 3, dtype=torch.uint8)
        with Plan(lib, w, B, S, H, D, dtype) as plan:
            starts = torch.tensor([1], dtype=torch.int32)
            cache = ua2a_cache_t(ptr(codes), ptr(scales), 1, 2, FORMAT[fmt])
            assert lib.ua2a_cache_write(plan.h, ctypes.byref(cache), 2, ptr(x), None, ptr(starts), None, None) == 0
            ref.check_same_codes(codes[0, :, :, 1:], scales[0, :, :, 1:], x.view(1, 1, 1, 1, 96), fmt, "special")
            assert int(codes[1].sum()) == 0 and int(codes[0, :, :, 0].sum()) == 0
            out = torch.full((1, 1, 1, 1, 96), 5.0)
            assert lib.ua2a_cache_read(plan.h, ctypes.byref(cache), 2, 1, ptr(starts), None, ptr(out), None, None) == 0
            want = torch.full_like(out, 5.0)
            ref.cache_read(want, codes, scales, fmt, [1], [1], 0)
            assert torch.equal(out.nan_to_num(123.0), want.nan_to_num(123.0))


CACHES = [(1, 1, 1, 1, 8, 1, 4), (2, 2, 4, 4, 16, 2, 11), (4, 1, 3, 8, 80, 12, 5), (2, 3, 2, 4, 7, 3, 6),
          (3, 1, 4, 6, 40, 4, 9), (2, 1, 8, 4, 33, 1, 30)]


@pytest.mark.parametrize("t", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("c", CACHES, ids=lambda s: "x".join(map(str, s)))
def test_cache(lib, c, t):
    """Starts before, inside and past the cache, counts of zero, one and more
    than there are; rows that nothing names stay as they were."""
    w, B, S, H, D, seqs, cap = c
    dtype, code = TYPES[t]
    nb = -(-D // 32)
    g = torch.Generator().manual_seed(7)
    each = B * S * w // seqs
    with Plan(lib, w, B, S, H, D, dtype) as plan:
        for k, fmt in enumerate((E4M3, E5M2)):
            codes = torch.randint(0, 120, (2, w, seqs, cap, H // w, D), generator=g, dtype=torch.uint8)
            scales = torch.randint(120, 130, (2, w, seqs, cap, H // w, nb), generator=g, dtype=torch.uint8)
            wc, ws = codes.clone(), scales.clone()
            starts = torch.randint(-3, cap + 2, (seqs,), generator=g, dtype=torch.int32)
            counts = torch.randint(-1, each + 3, (seqs,), generator=g, dtype=torch.int32) if k else None
            kk, vv = values(plan.p, dtype, 60 + k), values(plan.p, dtype, 70 + k, 100.0)
            cache = ua2a_cache_t(ptr(codes), ptr(scales), seqs, cap, FORMAT[fmt])
            assert lib.ua2a_cache_write(plan.h, ctypes.byref(cache), code, ptr(kk), ptr(vv), ptr(starts), ptr(counts), None) == 0
            cnt = counts.tolist() if k else [each] * seqs
            for part, x in ((0, kk), (1, vv)):
                ref.cache_write(wc, ws, x, fmt, w, starts.tolist(), cnt, part)
            assert torch.equal(codes, wc) and torch.equal(scales, ws)
            n = min(cap, 5)
            outs = [torch.full((w, seqs, n, H // w, D), 3.0, dtype=dtype) for _ in range(2)]
            want = [o.clone() for o in outs]
            rc = lib.ua2a_cache_read(plan.h, ctypes.byref(cache), code, n, ptr(starts), ptr(counts), ptr(outs[0]),
                                     ptr(outs[1]), None)
            assert rc == 0
            for part in (0, 1):
                ref.cache_read(want[part], codes, scales, fmt, starts.tolist(), counts.tolist() if k else [n] * seqs, part)
                assert torch.equal(outs[part], want[part])
            assert lib.ua2a_act_emu_error() == 0


def test_half_precision_of_the_emulation(lib):
    """The stand-in's own half conversions, through a cache read: every code
    and scale comes back as torch rounds it."""
    codes = torch.arange(256, dtype=torch.uint8).repeat(2, 1).view(2, 1, 1, 8, 1, 32).contiguous()
    for scale in (90, 101, 112, 120, 127, 134, 140):
        scales = torch.full((2, 1, 1, 8, 1, 1), scale, dtype=torch.uint8)
        out = torch.zeros(1, 1, 8, 1, 32, dtype=torch.float16)
        with Plan(lib, 1, 1, 1, 1, 32, torch.float16) as plan:
            cache = ua2a_cache_t(ptr(codes), ptr(scales), 1, 8, 1)
            assert lib.ua2a_cache_read(plan.h, ctypes.byref(cache), 1, 8, None, None, ptr(out), None, None) == 0
        want = torch.zeros_like(out)
        ref.cache_read(want, codes, scales, E4M3, [0], [8], 0)
        assert torch.equal(out.nan_to_num(7.0), want.nan_to_num(7.0)), scale


# ------------------------------------------------------------------ refusals

def _norm_args(**kw):
    base = 1 << 40
    a = dict(x=base, out=base + (1 << 30), eps=1e-6)
    a.update(kw)
    return ua2a_norm_t(**a)


@pytest.mark.parametrize("kw,mode,code", [
    (dict(x=None), 0, ua.UA2A_ERR_INVALID_ARG),
    (dict(out=None), 0, ua.UA2A_ERR_INVALID_ARG),
    (dict(), 2, ua.UA2A_ERR_INVALID_ARG),
    (dict(per_head=2), 0, ua.UA2A_ERR_INVALID_ARG),
    (dict(type=2), 0, ua.UA2A_ERR_INVALID_ARG),                            # fp32 on a 2-byte plan
    (dict(type=7), 0, ua.UA2A_ERR_INVALID_ARG),
    (dict(eps=0.0), 0, ua.UA2A_ERR_INVALID_ARG),
    (dict(eps=-1.0), 0, ua.UA2A_ERR_INVALID_ARG),
    (dict(eps=float("nan")), 0, ua.UA2A_ERR_INVALID_ARG),
    (dict(eps=float("inf")), 0, ua.UA2A_ERR_INVALID_ARG),
    (dict(residual=1 << 41), 0, ua.UA2A_ERR_INVALID_ARG),                  # no sum
    (dict(sum=1 << 41), 0, ua.UA2A_ERR_INVALID_ARG),                       # no residual
    (dict(out_format=3, out_scales=1 << 41), 0, ua.UA2A_ERR_INVALID_ARG),
    (dict(out_format=1), 0, ua.UA2A_ERR_INVALID_ARG),                      # no scales
    (dict(out_scales=1 << 41), 0, ua.UA2A_ERR_INVALID_ARG),                # scales without a format
    (dict(saved_format=1, saved=1 << 41), 0, ua.UA2A_ERR_INVALID_ARG),
    (dict(saved=1 << 41, saved_scales=1 << 42), 0, ua.UA2A_ERR_INVALID_ARG),
    (dict(weight=1 << 41, weight_type=1), 0, ua.UA2A_ERR_INVALID_ARG),     # fp16 weight, bf16 plan
    (dict(x=(1 << 40) + 1), 0, ua.UA2A_ERR_ALIGN),
    (dict(rstd=(1 << 41) + 2), 0, ua.UA2A_ERR_ALIGN),
    (dict(weight=(1 << 41) + 2, weight_type=2), 0, ua.UA2A_ERR_ALIGN),
    (dict(out=1 << 40), 0, ua.UA2A_ERR_ALIAS),
    (dict(out=(1 << 40) + 64), 1, ua.UA2A_ERR_ALIAS),
    (dict(rstd=1 << 40), 0, ua.UA2A_ERR_ALIAS),
    (dict(residual=1 << 40, sum=1 << 40), 0, ua.UA2A_ERR_ALIAS),           # in place
    (dict(saved_format=1, saved=1 << 41, saved_scales=(1 << 41) + 16), 0, ua.UA2A_ERR_ALIAS),
    (dict(weight=1 << 41, rstd=(1 << 41) + 4), 0, ua.UA2A_ERR_ALIAS),
])
def test_norm_refusals(lib, kw, mode, code):
    with Plan(lib, 2, 1, 8, 4, 16, torch.bfloat16) as plan:
        args = _norm_args(**kw)
        assert lib.ua2a_norm_exchange(plan.h, mode, ctypes.byref(args), None) == code
        assert lib.ua2a_act_emu_launches() == 0


def test_norm_refuses_what_it_cannot_hold(lib):
    for shape, per_head, code in [((1, 1, 1, 1, 65536), 0, 0), ((1, 1, 1, 1, 65544), 0, ua.UA2A_ERR_SHAPE),
                                  ((1, 1, 1, 2, 65536), 0, ua.UA2A_ERR_SHAPE), ((1, 1, 1, 1, 8193), 0, ua.UA2A_ERR_SHAPE),
                                  ((1, 1, 1, 1, 8191), 0, 0), ((1, 2 ** 12, 2 ** 15, 16, 8), 1, ua.UA2A_ERR_SHAPE)]:
        with Plan(lib, *shape, torch.bfloat16) as plan:
            n = shape[0] * shape[1] * shape[2] * shape[3] * shape[4]
            if code == 0:
                x = values(plan.p, torch.bfloat16, 1)
                out, *_ = run_norm(lib, plan, x, None, 0)
                ref.check_values(out, ref.norm(x, None, 0, 1)[0], torch.bfloat16, str(shape))
            else:
                args = _norm_args(per_head=per_head, out=(1 << 40) + 2 * n)
                assert lib.ua2a_norm_exchange(plan.h, 0, ctypes.byref(args), None) == code
                need = ctypes.c_int64()
                if per_head:
                    assert lib.ua2a_norm_workspace(plan.h, per_head, ctypes.byref(need)) == code


def _grad_args(**kw):
    base = 1 << 40
    a = dict(dy=base, saved=base + (1 << 20), rstd=base + (1 << 21), dx=base + (1 << 22))
    a.update(kw)
    return ua2a_norm_grad_t(**a)


@pytest.mark.parametrize("kw,mode,code", [
    (dict(dy=None), 0, ua.UA2A_ERR_INVALID_ARG),
    (dict(saved=None), 0, ua.UA2A_ERR_INVALID_ARG),
    (dict(rstd=None), 0, ua.UA2A_ERR_INVALID_ARG),
    (dict(dx=None), 0, ua.UA2A_ERR_INVALID_ARG),
    (dict(), 3, ua.UA2A_ERR_INVALID_ARG),
    (dict(type=2), 0, ua.UA2A_ERR_INVALID_ARG),
    (dict(saved_format=1), 0, ua.UA2A_ERR_INVALID_ARG),
    (dict(saved_scales=1 << 42), 0, ua.UA2A_ERR_INVALID_ARG),
    (dict(saved_gathered=1), 0, ua.UA2A_ERR_INVALID_ARG),                  # mode 0 holds P
    (dict(dresidual=1 << 42), 0, ua.UA2A_ERR_INVALID_ARG),                 # mode 0: dx is it
    (dict(dweight=1 << 42), 0, ua.UA2A_ERR_INVALID_ARG),                   # no workspace
    (dict(dweight=1 << 42, workspace=1 << 43, workspace_bytes=-1), 0, ua.UA2A_ERR_INVALID_ARG),
    (dict(dweight=1 << 42, workspace=1 << 43, workspace_bytes=64), 0, ua.UA2A_ERR_CAPACITY),
    (dict(dweight=1 << 42, workspace=(1 << 43) + 4, workspace_bytes=1 << 20), 0, ua.UA2A_ERR_ALIGN),
    (dict(dx=(1 << 40) + 1), 0, ua.UA2A_ERR_ALIGN),
    (dict(dx=1 << 40), 0, ua.UA2A_ERR_ALIAS),
    (dict(dresidual=(1 << 40) + (1 << 22) + 2), 1, ua.UA2A_ERR_ALIAS),
    (dict(dsum=(1 << 40) + (1 << 22)), 1, ua.UA2A_ERR_ALIAS),
])
def test_backward_refusals(lib, kw, mode, code):
    with Plan(lib, 2, 1, 8, 4, 16, torch.bfloat16) as plan:
        args = _grad_args(**kw)
        assert lib.ua2a_norm_exchange_backward(plan.h, mode, ctypes.byref(args), None) == code
        assert lib.ua2a_act_emu_launches() == 0


def _cache(**kw):
    a = dict(codes=1 << 40, scales=1 << 41, sequences=2, capacity=8, format=1)
    a.update(kw)
    return ua2a_cache_t(**a)


@pytest.mark.parametrize("ckw,kw,code", [
    (dict(codes=None), {}, ua.UA2A_ERR_INVALID_ARG),
    (dict(scales=None), {}, ua.UA2A_ERR_INVALID_ARG),
    (dict(format=0), {}, ua.UA2A_ERR_INVALID_ARG),
    (dict(format=3), {}, ua.UA2A_ERR_INVALID_ARG),
    (dict(sequences=0), {}, ua.UA2A_ERR_SHAPE),
    (dict(capacity=0), {}, ua.UA2A_ERR_SHAPE),
    (dict(capacity=2 ** 31), {}, ua.UA2A_ERR_SHAPE),
    (dict(sequences=2 ** 20, capacity=2 ** 20), {}, ua.UA2A_ERR_SHAPE),
    (dict(sequences=3), {}, ua.UA2A_ERR_SHAPE),                            # 16 tokens, 3 sequences
    ({}, dict(starts=None), ua.UA2A_ERR_INVALID_ARG),
    ({}, dict(k=None, v=None), ua.UA2A_ERR_INVALID_ARG),
    ({}, dict(type=2), ua.UA2A_ERR_INVALID_ARG),
    ({}, dict(k=(1 << 42) + 1), ua.UA2A_ERR_ALIGN),
    ({}, dict(starts=(1 << 43) + 2), ua.UA2A_ERR_ALIGN),
    (dict(scales=1 << 40), {}, ua.UA2A_ERR_ALIAS),
    (dict(codes=1 << 42), {}, ua.UA2A_ERR_ALIAS),
])
def test_cache_write_refusals(lib, ckw, kw, code):
    a = dict(type=0, k=1 << 42, v=(1 << 42) + (1 << 30), starts=1 << 43)
    a.update(kw)
    with Plan(lib, 2, 1, 8, 4, 16, torch.bfloat16) as plan:
        c = _cache(**ckw)
        assert lib.ua2a_cache_write(plan.h, ctypes.byref(c), a["type"], a["k"], a["v"], a["starts"], None, None) == code
        assert lib.ua2a_act_emu_launches() == 0


@pytest.mark.parametrize("ckw,kw,code", [
    (dict(codes=None), {}, ua.UA2A_ERR_INVALID_ARG),
    (dict(format=5), {}, ua.UA2A_ERR_INVALID_ARG),
    ({}, dict(k=None, v=None), ua.UA2A_ERR_INVALID_ARG),
    ({}, dict(n=0), ua.UA2A_ERR_SHAPE),
    ({}, dict(n=2 ** 31), ua.UA2A_ERR_SHAPE),
    ({}, dict(n=2 ** 28), ua.UA2A_ERR_SHAPE),                              # 2^31 pieces or more
    ({}, dict(v=(1 << 42) + 64), ua.UA2A_ERR_ALIAS),
    ({}, dict(k=1 << 40), ua.UA2A_ERR_ALIAS),
    ({}, dict(k=(1 << 42) + 1), ua.UA2A_ERR_ALIGN),
])
def test_cache_read_refusals(lib, ckw, kw, code):
    a = dict(n=4, k=1 << 42, v=(1 << 42) + (1 << 38))
    a.update(kw)
    with Plan(lib, 2, 1, 8, 4, 16, torch.bfloat16) as plan:
        c = _cache(**ckw)
        assert lib.ua2a_cache_read(plan.h, ctypes.byref(c), 0, a["n"], None, None, a["k"], a["v"], None) == code
        assert lib.ua2a_act_emu_launches() == 0


def test_wrong_device_is_refused(lib):
    with Plan(lib, 2, 1, 8, 4, 16, torch.bfloat16, device=1) as plan:
        args = _norm_args()
        assert lib.ua2a_norm_exchange(plan.h, 0, ctypes.byref(args), None) == ua.UA2A_ERR_DEVICE
        c = _cache()
        assert lib.ua2a_cache_write(plan.h, ctypes.byref(c), 0, 1 << 42, None, 1 << 43, None, None) == ua.UA2A_ERR_DEVICE
        assert lib.ua2a_act_emu_launches() == 0
