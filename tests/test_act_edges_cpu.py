"""Activation calls at the edges of what they take: the host side, without a GPU."""
from __future__ import annotations

import ctypes

import pytest
import torch

import ulysses_all_re_amd as ua
from tests import act_reference as ref
from tests.emu import act_build
from tests.test_act_emulated import TYPES, ptr, values
from tests.test_binding_cpu import _host_plan
from tests.test_gpu_act_walks import WALKS
from ulysses_all_re_amd.activations import ua2a_cache_t, ua2a_norm_grad_t, ua2a_norm_t


class Calls:
    """Stands in for the library: what each call would have passed."""

    def __init__(self, plan):
        self.seen = []
        plan._issue = lambda name, stream, *args: self.seen.append((name, args))

    def addresses(self):
        cache = self.seen[-1][1][0]._obj
        return cache.codes, cache.scales


def test_a_cache_follows_its_tensors():
    """The library gets the addresses that a cache's tensors have at the call: a
    tensor given other memory is used there, one without memory is refused."""
    plan = _host_plan(w=2, B=1, S=4, H=4, D=16)
    calls = Calls(plan)
    cache = ua.Cache(2, 4, 16, 8, 5, device="cpu")
    k = torch.zeros(plan.in_shape(0), dtype=torch.bfloat16)
    starts = torch.zeros(8, dtype=torch.int32)
    plan.cache_write(cache, k, k, starts)
    assert calls.addresses() == (cache.codes.data_ptr(), cache.scales.data_ptr())
    keep = cache.codes
    cache.codes.set_(torch.zeros_like(cache.codes.view(torch.uint8)).view(cache.codes.dtype))
    for call in (lambda: plan.cache_write(cache, k, k, starts), lambda: plan.cache_read(cache, 2, out=(torch.zeros(
            2, 8, 2, 2, 16, dtype=torch.bfloat16), None))):
        call()
        assert calls.addresses() == (cache.codes.data_ptr(), cache.scales.data_ptr())
    assert cache.codes is keep
    done = len(calls.seen)
    cache.scales.untyped_storage().resize_(0)
    with pytest.raises(ValueError, match="memory"):
        plan.cache_write(cache, k, k, starts)
    with pytest.raises(ValueError, match="memory"):
        plan.cache_read(cache, 2)
    cache.scales.untyped_storage().resize_(cache.scales.numel())
    plan.cache_write(cache, k, k, starts)
    assert calls.addresses() == (cache.codes.data_ptr(), cache.scales.data_ptr())
    cache.codes.set_(torch.zeros(2, 2, 8, 5, 2, 8, dtype=torch.uint8).view(cache.codes.dtype))
    cache.scales.set_(torch.zeros(2, 2, 8, 5, 2, 1, dtype=torch.uint8).view(cache.scales.dtype))
    with pytest.raises(ValueError, match="the plan"):                            # heads of 8 now
        plan.cache_write(cache, k, k, starts)
    assert len(calls.seen) == done + 1
    plan.close()


@pytest.fixture(scope="module")
def lib():
    so = ctypes.CDLL(act_build.build())
    i32, i64, vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p
    so.ua2a_plan.argtypes = [ctypes.POINTER(vp), i32, i64, i64, i64, i64, i32, i32, vp, i64, i32]
    so.ua2a_destroy.argtypes = [vp]
    return ua.declare_activation_signatures(so)


@pytest.fixture
def dry(lib):
    """Launches are recorded and not carried out: any size, any address."""
    lib.ua2a_act_emu_reset()
    lib.ua2a_act_emu_dry(1)
    yield lib
    lib.ua2a_act_emu_dry(0)


def make_plan(lib, w, B, S, H, D, e=2):
    h = ctypes.c_void_p()
    assert lib.ua2a_plan(ctypes.byref(h), w, B, S, H, D, e, 0, None, 0, 0) == 0
    return h


def grid(lib):
    """Workgroups along x and y of the last launch, and lanes of one."""
    x, y, lanes = (lib.ua2a_act_emu_last(k) for k in (3, 5, 2))
    assert x * lanes <= 2 ** 31 and y <= 65535
    return x, y, lanes


@pytest.mark.parametrize("H,D,pieces,chunks", [
    (40, 128, 640, 3),             # 640 vectors of 16 bytes on three workgroups of 256 lanes
    (16, 128, 256, 1),
    (257, 32, 1028, 5),
    (9, 1, 288, 2),                # single values, a block of 32 for each head
])
def test_cache_writes_up_to_the_stated_size(dry, H, D, pieces, chunks):
    """2^31 - 1 pieces at most, however many lanes the tokens' padding adds."""
    most = (2 ** 31 - 1) // pieces
    for tokens in (most, most + 1, 2 ** 23 // chunks - 600, 2 ** 23 // chunks + 600):
        code = 0 if tokens <= most else ua.UA2A_ERR_SHAPE
        plan = make_plan(dry, 1, tokens, 1, H, D)
        cache = ua2a_cache_t(1 << 44, 1 << 46, 1, 1, 1)
        assert dry.ua2a_cache_write(plan, ctypes.byref(cache), 0, 1 << 40, None, 1 << 47, None, None) == code, tokens
        if code == 0:
            x, y, _ = grid(dry)
            assert x * y >= tokens * chunks and (y > 1) == (tokens * chunks > 2 ** 23)
        dry.ua2a_destroy(plan)


@pytest.mark.parametrize("w,H,D,n,vectors,lanes", [
    (1, 1, 8, 1, 1, 64),           # one vector of 16 bytes a sequence, on a wave
    (2, 2, 8, 65, 65, 128),
    (1, 1, 8, 257, 257, 256),
    (1, 3, 1, 1, 3, 64),           # single values
])
def test_cache_reads_up_to_the_stated_size(dry, w, H, D, n, vectors, lanes):
    """2^31 - 1 pieces at most, however short the sequences."""
    most = (2 ** 31 - 1) // (vectors * w)
    turn = 2 ** 23 // (-(-vectors // lanes) * w)                # sequences that fill x
    for seqs in (most, most + 1, turn, turn + 1):
        code = 0 if seqs <= most else ua.UA2A_ERR_SHAPE
        plan = make_plan(dry, w, 1, 1, H, D)
        cache = ua2a_cache_t(1 << 44, 1 << 46, seqs, 1, 1)
        assert dry.ua2a_cache_read(plan, ctypes.byref(cache), 0, n, None, None, 1 << 40, None, None) == code, seqs
        if code == 0:
            x, y, block = grid(dry)
            assert block == lanes and x * y >= seqs * w * -(-vectors // lanes) and (y > 1) == (seqs > turn)
        dry.ua2a_destroy(plan)


@pytest.mark.parametrize("fp32", [False, True], ids=["type", "fp32"])
def test_a_weight_at_any_address_leaves_the_path(lib, fp32):
    """A weight off a 16-byte boundary (a view into a flat parameter buffer)
    costs a call neither its vectors nor its longest norm."""
    for shape, per_head in (((2, 1, 4, 4, 16), 0), ((2, 1, 4, 4, 16), 1), ((1, 1, 2, 4, 4096), 0)):
        w, B, S, H, D = shape
        plan = make_plan(lib, *shape)
        lib.ua2a_act_emu_reset()
        n = D if per_head else H * D
        x = values(shape, torch.bfloat16, 1)
        weight = values((n + 1,), torch.float32 if fp32 else torch.bfloat16, 2)[1:]
        assert weight.data_ptr() % 16 != 0
        out, rstd = torch.zeros((w, B, S * w, H // w, D), dtype=torch.bfloat16), torch.zeros(w * B * S * H)
        args = ua2a_norm_t(x=ptr(x), weight=ptr(weight), out=ptr(out), rstd=ptr(rstd), eps=1e-6, per_head=per_head,
                           weight_type=2 if fp32 else 0)
        assert lib.ua2a_norm_exchange(plan, 0, ctypes.byref(args), None) == 0
        assert lib.ua2a_act_emu_last(0) == 8 and lib.ua2a_act_emu_error() == 0
        y, h, _ = ref.norm(x, weight, 0, w, None, bool(per_head))
        ref.check_values(out, y, torch.bfloat16, str(shape))
        rstd = rstd[:w * B * S * (H if per_head else 1)].view((w, B, S) + ((H,) if per_head else ()))
        dy, dx, dw = values(tuple(out.shape), torch.bfloat16, 3), torch.zeros_like(x), torch.zeros(n)
        need = ctypes.c_int64()
        assert lib.ua2a_norm_workspace(plan, per_head, ctypes.byref(need)) == 0
        space = torch.zeros(need.value // 4)
        args = ua2a_norm_grad_t(dy=ptr(dy), saved=ptr(x), weight=ptr(weight), rstd=ptr(rstd), dx=ptr(dx), dweight=ptr(dw),
                                workspace=ptr(space), workspace_bytes=need.value, per_head=per_head,
                                weight_type=2 if fp32 else 0)
        assert lib.ua2a_norm_exchange_backward(plan, 0, ctypes.byref(args), None) == 0
        assert lib.ua2a_act_emu_error() == 0
        want = ref.norm_backward(dy, weight, 0, w, h, rstd, None, bool(per_head))
        parts = ref.backward_terms(dy, weight, 0, w, h, rstd, None, bool(per_head))
        ref.check_backward(dx, None, dw, want, parts, torch.bfloat16, 0, w, str(shape))
        lib.ua2a_destroy(plan)


# (shape, per head, type): every way that segments lie on lanes, among them the
# ones that only long norms or single values take
LANES = [((3, 2, 5, 6, 40), True, "bf16"), ((2, 1, 7, 10, 96), True, "fp16"), ((5, 1, 3, 15, 32), True, "fp32"),
         ((2, 1, 3, 2, 2048), True, "bf16"), ((1, 1, 5, 3, 24), False, "fp32"), ((4, 1, 3, 8, 80), False, "bf16"),
         ((2, 1, 3, 10, 520), False, "fp16"), ((1, 1, 3, 86, 128), False, "bf16"), ((2, 1, 2, 32, 520), False, "bf16"),
         ((2, 1, 2, 64, 512), False, "fp16"), ((1, 1, 2, 2, 32768), False, "bf16"), ((2, 1, 2, 28, 250), False, "fp32"),
         ((2, 1, 2, 66, 33), False, "bf16"), ((3, 1, 2, 3, 1001), False, "fp32"), ((1, 1, 2, 1, 8191), True, "fp16")]


@pytest.mark.parametrize("mode", [0, 1])
@pytest.mark.parametrize("shape,per_head,t", LANES, ids=lambda v: "x".join(map(str, v)) if isinstance(v, tuple) else str(v))
def test_every_lane_has_its_place(lib, shape, per_head, t, mode):
    """A forward and a backward call of each kind, each lane's places checked."""
    w, B, S, H, D = shape
    dtype, code = TYPES[t]
    e = torch.empty((), dtype=dtype).element_size()
    plan = make_plan(lib, *shape, e=e)
    lib.ua2a_act_emu_reset()
    p, a = shape, (w, B, S * w, H // w, D)
    n = D if per_head else H * D
    nb = -(-D // 32)
    x, weight = values(p if mode == 0 else a, dtype, 1), values((n,), dtype, 2)
    oshape = a if mode == 0 else p
    out, osc = torch.zeros(oshape, dtype=torch.uint8), torch.zeros(oshape[:-1] + (nb,), dtype=torch.uint8)
    saved, ssc = torch.zeros(p, dtype=torch.uint8), torch.zeros(p[:-1] + (nb,), dtype=torch.uint8)
    rstd = torch.zeros(p[:4] if per_head else p[:3])
    args = ua2a_norm_t(ptr(x), None, ptr(weight), ptr(out), ptr(osc), None, ptr(saved), ptr(ssc), ptr(rstd), 1e-6, code,
                       code, int(per_head), 1, 1)
    assert lib.ua2a_norm_exchange(plan, mode, ctypes.byref(args), None) == 0
    assert lib.ua2a_act_emu_error() == 0
    y, h, r = ref.norm(x, weight, mode, w, None, per_head)
    ref.check_values(rstd, r, torch.float32, "rstd")
    ref.check_codes(out, osc, y, torch.float8_e4m3fn, "out")
    dy, dx, dw = values(oshape, dtype, 3), torch.zeros_like(x), torch.zeros(n)
    need = ctypes.c_int64()
    assert lib.ua2a_norm_workspace(plan, int(per_head), ctypes.byref(need)) == 0
    space = torch.zeros(need.value // 4)
    args = ua2a_norm_grad_t(ptr(dy), None, ptr(saved), ptr(ssc), ptr(weight), ptr(rstd), ptr(dx), None, ptr(dw), ptr(space),
                            need.value, code, code, int(per_head), 1, 0)
    assert lib.ua2a_norm_exchange_backward(plan, mode, ctypes.byref(args), None) == 0
    assert lib.ua2a_act_emu_error() == 0
    hq = ref.dequantise(saved, ssc, torch.float8_e4m3fn)
    want = ref.norm_backward(dy, weight, mode, w, hq, rstd, None, per_head)
    parts = ref.backward_terms(dy, weight, mode, w, hq, rstd, None, per_head)
    ref.check_backward(dx, None, dw, want, parts, dtype, mode, w, "lanes")
    lib.ua2a_destroy(plan)


def test_walks_are_walks(dry):
    """Each shape of the walk tests has more than two segments for a workgroup's
    every place, and together they take every way that segments lie on lanes."""
    kinds = set()
    for shape, per_head, t in WALKS:
        dtype, code = TYPES[t]
        plan = make_plan(dry, *shape, e=torch.empty((), dtype=dtype).element_size())
        args = ua2a_norm_grad_t(dy=1 << 40, saved=1 << 42, rstd=1 << 44, dx=1 << 45, type=code, per_head=int(per_head))
        assert dry.ua2a_norm_exchange_backward(plan, 0, ctypes.byref(args), None) == 0
        V, items, _, x, _, _, groups, span = (dry.ua2a_act_emu_last(k) for k in range(8))
        assert groups > 2 * x, shape
        kinds.add((span, items, V == 1))
        dry.ua2a_destroy(plan)
    part, wide, waves, bundle, bundles = range(5)
    assert kinds >= {(part, 1, False), (wide, 1, True), (wide, 4, True), (waves, 2, False), (waves, 3, False),
                     (waves, 4, False), (waves, 5, False), (wide, 2, False), (bundle, 2, False), (bundle, 1, False),
                     (bundles, 1, False)}, kinds
