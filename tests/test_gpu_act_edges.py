"""GPU: activation calls at the edges of what they take -- rows of NaN beside
others, scale bytes that are NaN, weights at any address, many sequences."""
from __future__ import annotations

import sys
import threading

import pytest
import torch

import ulysses_all_re_amd as ua
from tests import act_reference as ref
from tests.test_gpu_activations import E4M3, E5M2, TYPES, cpu, dev, values
from ulysses_all_re_amd import ops

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


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


# heads of 40: eight lanes of which three are padding; of 24 in fp32: eight, two of
# them padding; of 33: single values; heads that share a bundle, or a wave
@pytest.mark.parametrize("save", [None, E4M3, E5M2], ids=["values", "e4m3", "e5m2"])
@pytest.mark.parametrize("mode", [0, 1])
@pytest.mark.parametrize("t,H,D", [("bf16", 16, 40), ("fp16", 10, 40), ("fp32", 16, 24), ("fp32", 6, 40),
                                   ("bf16", 8, 33), ("bf16", 3, 72)])
def test_a_head_of_nan_leaves_the_others_alone(t, H, D, mode, save):
    """Norms per head with NaN in the first head of a token: that head's
    gradients are NaN, every other head's are those of the definition."""
    dtype, w = TYPES[t], 1
    note(f"nan head {t} {H}x{D} mode {mode} {save}")
    plan = ua.Plan(w, 1, 5, H, D, dtype, device=DEV)
    x, weight = values(plan.in_shape(mode), dtype, 1), values((D,), dtype, 2)
    x[0, 0, 2, 0, 1] = float("nan")                             # w = 1: P and A are the same
    dy = values(plan.out_shape(mode), dtype, 3)
    r = plan.norm_exchange(dev(x), dev(weight), mode, per_head=True, checkpoint=save, rstd=True)
    b = plan.norm_exchange_backward(dev(dy), dev(weight), mode, r.saved if save else dev(x), r.rstd,
                                    saved_scales=r.saved_scales, per_head=True)
    torch.cuda.synchronize()
    y, h, _ = ref.norm(x, weight, mode, w, None, True)
    ref.check_values(cpu(r.out), y, dtype, "out")
    rs = cpu(r.rstd)
    assert int(torch.isnan(rs).sum()) == 1
    if save:
        h = ref.dequantise(cpu(r.saved), cpu(r.saved_scales), save)
    want = ref.norm_backward(dy, weight, mode, w, h, rs, None, True)
    parts = ref.backward_terms(dy, weight, mode, w, h, rs, None, True)
    assert int(torch.isnan(want[0]).sum()) == D
    ref.check_backward(cpu(b.dx), None, None, want, parts, dtype, mode, w, "nan head")
    assert bool(torch.isnan(cpu(b.dweight)).all())
    plan.close()


@pytest.mark.parametrize("save", [None, E4M3], ids=["values", "e4m3"])
@pytest.mark.parametrize("per_head", [False, True], ids=["token", "head"])
@pytest.mark.parametrize("t,H,D", [("bf16", 8, 40), ("fp32", 6, 24), ("fp16", 3, 33), ("bf16", 24, 40)])
def test_an_infinite_weight_meets_values_only(t, H, D, per_head, save):
    """The first weight is infinite: gradients are the definition's infinities,
    which lanes of padding (they hold that weight too) do not turn into NaN."""
    dtype, w = TYPES[t], 1
    note(f"infinite weight {t} {H}x{D} head {per_head} {save}")
    plan = ua.Plan(w, 1, 5, H, D, dtype, device=DEV)
    x, weight = values(plan.in_shape(0), dtype, 1), values((D if per_head else H * D,), dtype, 2)
    weight[0] = float("inf")
    dy = values(plan.out_shape(0), dtype, 3)
    r = plan.norm_exchange(dev(x), dev(weight), 0, per_head=per_head, checkpoint=save, rstd=True)
    b = plan.norm_exchange_backward(dev(dy), dev(weight), 0, r.saved if save else dev(x), r.rstd,
                                    saved_scales=r.saved_scales, per_head=per_head)
    torch.cuda.synchronize()
    _, h, _ = ref.norm(x, weight, 0, w, None, per_head)
    if save:
        h = ref.dequantise(cpu(r.saved), cpu(r.saved_scales), save)
    rs = cpu(r.rstd)
    want = ref.norm_backward(dy, weight, 0, w, h, rs, None, per_head)
    parts = ref.backward_terms(dy, weight, 0, w, h, rs, None, per_head)
    assert bool(torch.isinf(want[0]).any())
    ref.check_backward(cpu(b.dx), None, cpu(b.dweight), want, parts, dtype, 0, w, "infinite weight")
    plan.close()


@pytest.mark.parametrize("fmt", [E4M3, E5M2], ids=["e4m3", "e5m2"])
@pytest.mark.parametrize("t", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("D", [96, 40, 33])
def test_a_scale_of_nan_reads_back_as_nan(t, fmt, D):
    """The scale byte 255 is NaN: its block reads back as NaN, codes of zero and
    infinities among it, and every other block as before."""
    dtype = TYPES[t]
    note(f"nan scale read {t} {fmt} {D}")
    nb = -(-D // 32)
    plan = ua.Plan(2, 1, 1, 4, D, dtype, device=DEV)
    g = torch.Generator().manual_seed(5)
    codes = torch.randint(0, 256, (2, 2, 3, 7, 2, D), generator=g, dtype=torch.uint8)
    codes[..., 0] = 0
    scales = torch.randint(100, 130, (2, 2, 3, 7, 2, nb), generator=g, dtype=torch.uint8)
    hit = torch.rand(scales.shape, generator=g) < 0.2
    scales[hit] = 255
    cache = ua.Cache.of(dev(codes).view(fmt), dev(scales).view(torch.float8_e8m0fnu))
    got = plan.cache_read(cache, 7)
    torch.cuda.synchronize()
    want = [torch.zeros(2, 3, 7, 2, D, dtype=dtype) for _ in range(2)]
    plain = torch.where(hit, torch.full_like(scales, 127), scales)
    for part in (0, 1):
        ref.cache_read(want[part], codes, plain, fmt, [0] * 3, [7] * 3, part)
        want[part][hit[part].repeat_interleave(32, -1)[..., :D]] = float("nan")
        k = cpu(got[part])
        assert torch.equal(torch.isnan(k), torch.isnan(want[part]))
        assert torch.equal(k.nan_to_num(1.0, 2.0, 3.0), want[part].nan_to_num(1.0, 2.0, 3.0))
    plan.close()


@pytest.mark.parametrize("per_head", [False, True], ids=["token", "head"])
@pytest.mark.parametrize("t,H,D", [("bf16", 8, 64), ("fp16", 6, 40), ("fp32", 4, 72), ("bf16", 3, 33), ("bf16", 40, 128)])
def test_a_scale_of_nan_in_a_checkpoint(t, H, D, per_head):
    """A checkpoint with the scale byte 255: its norm's gradients are NaN, all others as before."""
    dtype, w = TYPES[t], 1
    note(f"nan scale backward {t} {H}x{D} head {per_head}")
    plan = ua.Plan(w, 1, 5, H, D, dtype, device=DEV)
    x, weight = values(plan.in_shape(0), dtype, 1), values((D if per_head else H * D,), dtype, 2)
    dy = values(plan.out_shape(0), dtype, 3)
    r = plan.norm_exchange(dev(x), dev(weight), 0, per_head=per_head, checkpoint=E4M3)
    codes, scales = cpu(r.saved), cpu(r.saved_scales)
    h = ref.dequantise(codes, scales, E4M3)
    scales[0, 0, 2, 0, 0] = 255
    h[0, 0, 2, 0, :32] = float("nan")
    b = plan.norm_exchange_backward(dev(dy), dev(weight), 0, r.saved, r.rstd, per_head=per_head,
                                    saved_scales=dev(scales).view(torch.float8_e8m0fnu))
    torch.cuda.synchronize()
    rs = cpu(r.rstd)
    want = ref.norm_backward(dy, weight, 0, w, h, rs, None, per_head)
    parts = ref.backward_terms(dy, weight, 0, w, h, rs, None, per_head)
    assert int(torch.isnan(want[0]).sum()) == (D if per_head else H * D)
    ref.check_backward(cpu(b.dx), None, cpu(b.dweight), want, parts, dtype, 0, w, "nan scale")
    plan.close()


def test_a_write_of_more_workgroups_than_fit_along_x():
    """4.3 million tokens of nine heads of one value: two workgroups a token."""
    w, H, D, S = 1, 9, 1, 4_300_000
    note("cache write, 8.6 million workgroups")
    plan = ua.Plan(w, 1, S, H, D, torch.bfloat16, device=DEV)
    k = values(plan.in_shape(0), torch.bfloat16, 1)
    cache = ua.Cache(w, H, D, 1, S + 3, E4M3, DEV)
    starts = torch.tensor([2], dtype=torch.int32)
    plan.cache_write(cache, dev(k), None, dev(starts))
    torch.cuda.synchronize()
    q, s = ref.quantise(k, E4M3)
    codes, scales = cpu(cache.codes), cpu(cache.scales)
    assert torch.equal(codes[0, 0, 0, 2:S + 2], q[0, 0]) and torch.equal(scales[0, 0, 0, 2:S + 2], s[0, 0])
    for t in (codes, scales):
        assert not bool(t[1].any()) and not bool(t[0, 0, 0, :2].any()) and not bool(t[0, 0, 0, S + 2:].any())
    plan.close()


def test_a_read_of_more_workgroups_than_fit_along_x():
    """The first position of 33.6 million sequences, a vector each."""
    seqs = 2 ** 25 + 5
    note("cache read, 33.6 million workgroups")
    plan = ua.Plan(1, 1, 1, 1, 8, torch.bfloat16, device=DEV)
    codes = torch.arange(2 * seqs * 8, device=DEV).remainder_(251).remainder_(120).to(torch.uint8)
    codes = codes.view(2, 1, seqs, 1, 1, 8).view(E4M3)
    scales = torch.full((2, 1, seqs, 1, 1, 1), 128, dtype=torch.uint8, device=DEV)
    out = torch.zeros(1, seqs, 1, 1, 8, dtype=torch.bfloat16, device=DEV)
    plan.cache_read(ua.Cache.of(codes, scales), 1, out=(None, out))
    torch.cuda.synchronize()
    assert torch.equal(out, (codes[1].float() * 2).bfloat16())
    plan.close()


@pytest.mark.parametrize("t,wt", [("bf16", "bf16"), ("fp16", "fp32"), ("fp32", "fp32")])
@pytest.mark.parametrize("shape", [(2, 1, 5, 8, 128), (2, 1, 9, 4, 16), (1, 1, 5, 128, 128), (3, 1, 5, 6, 40)],
                         ids=lambda s: "x".join(map(str, s)))
def test_weights_at_any_address_give_the_same_bits(shape, t, wt):
    """Weights one value past a 16-byte boundary, forward and backward, against aligned ones."""
    note(f"weight address {shape} {t} {wt}")
    plan = ua.Plan(*shape, TYPES[t], device=DEV)
    w, B, S, H, D = shape
    x = values(plan.in_shape(0), TYPES[t], 1).to(DEV)
    dy = values(plan.out_shape(0), TYPES[t], 2).to(DEV)
    for per_head in (False, True):
        n = D if per_head else H * D
        weight = values((n,), TYPES[wt], 3).to(DEV)
        flat = torch.zeros(n + 1, dtype=TYPES[wt], device=DEV)
        flat[1:] = weight
        assert weight.data_ptr() % 16 == 0 and flat[1:].data_ptr() % 16 != 0
        got = []
        for v in (weight, flat[1:]):
            r = plan.norm_exchange(x, v, 0, per_head=per_head, checkpoint=E4M3)
            b = plan.norm_exchange_backward(dy, v, 0, r.saved, r.rstd, saved_scales=r.saved_scales, per_head=per_head)
            got.append((r.out, b.dx, b.dweight))
        torch.cuda.synchronize()
        for p, q in zip(*got):
            assert torch.equal(p, q)
    plan.close()


@pytest.mark.parametrize("mode", [0, 1])
@pytest.mark.parametrize("checkpoint", [None, E5M2], ids=["values", "e5m2"])
def test_an_unused_norm_adds_nothing_to_the_sums_gradient(mode, checkpoint):
    """Where only the sum is used its gradient is x's and the residual's, beside
    NaN, infinities and rows of zeros too, and the weight's is zero."""
    w, B, S, H, D = 2, 1, 6, 4, 40
    p, a = (w, B, S, H, D), (w, B, S * w, H // w, D)
    x, res, g = values(p if mode == 0 else a, torch.bfloat16, 1), values(p, torch.bfloat16, 2), values(p, torch.bfloat16, 3)
    res[0, 0, 1, 2, 3], res[1, 0, 0, 0, 0] = float("nan"), float("inf")
    x[0, 0, 3], x[1, 0, 2] = float("inf"), 0
    xd, rd = x.to(DEV).requires_grad_(True), res.to(DEV).requires_grad_(True)
    wd = values((H * D,), torch.float32, 4).to(DEV).requires_grad_(True)
    _, total = ops.norm_all_to_all_4D(xd, wd, *((2, 1) if mode == 0 else (1, 2)), w, residual=rd, checkpoint=checkpoint)
    total.backward(g.to(DEV))
    assert torch.equal(xd.grad.cpu(), g if mode == 0 else ref.to_a(g, w)) and torch.equal(rd.grad.cpu(), g)
    assert xd.grad.data_ptr() != rd.grad.data_ptr()
    assert wd.grad.shape == wd.shape and not bool(wd.grad.any())
    rd.grad = None
    _, total = ops.norm_all_to_all_4D(x.to(DEV), None, *((2, 1) if mode == 0 else (1, 2)), w, residual=rd)
    total.backward(g.to(DEV))
    assert torch.equal(rd.grad.cpu(), g)


def test_a_norm_of_more_workgroups_than_fit_along_x():
    """11.3 million tokens of five heads of one value, a workgroup of 192 lanes
    each, forward and backward.  The weight's gradient: a workgroup of 512 adds
    11,300,000 / 512 products in a row, with the rows' joins under 2^14.5."""
    w, H, D, S = 1, 5, 1, 11_300_000
    note("norm, 11.3 million workgroups")
    plan = ua.Plan(w, 1, S, H, D, torch.bfloat16, device=DEV)
    x, weight = values(plan.in_shape(0), torch.bfloat16, 1), values((H * D,), torch.float32, 2)
    dy = values(plan.out_shape(0), torch.bfloat16, 3)
    r = plan.norm_exchange(dev(x), dev(weight), 0, rstd=True)
    b = plan.norm_exchange_backward(dev(dy), dev(weight), 0, dev(x), r.rstd)
    torch.cuda.synchronize()
    y, h, rstd = ref.norm(x, weight, 0, w)
    rs = cpu(r.rstd)
    ref.check_values(rs, rstd, torch.float32, "rstd")
    ref.check_values(cpu(r.out), y, torch.bfloat16, "out")
    want, parts = ref.norm_backward(dy, weight, 0, w, h, rs), ref.backward_terms(dy, weight, 0, w, h, rs)
    ref.check_backward(cpu(b.dx), None, None, want, parts, torch.bfloat16, 0, w, "dx")
    ref.assert_close(cpu(b.dweight), want[2], parts[1] * 2.0 ** (14.5 - 24), "dweight")
    plan.close()


@pytest.mark.parametrize("t", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("eps", [1e-45, 1e38], ids=["least", "large"])
def test_the_least_and_large_eps_on_rows_of_zeros(t, eps):
    """Tokens of zeros have rstd = 1 / sqrt(eps), eps being any positive float."""
    plan = ua.Plan(2, 1, 3, 4, 16, TYPES[t], device=DEV)
    x = values(plan.in_shape(0), TYPES[t], 1)
    x[0, 0, 1], x[1, 0, 2] = 0, 0
    eps32 = float(torch.tensor(eps, dtype=torch.float32))
    y, h, rstd = ref.norm(x, None, 0, 2, None, False, eps32)
    r = plan.norm_exchange(dev(x), None, 0, eps=eps, rstd=True)
    dy = values(plan.out_shape(0), TYPES[t], 2, 2.0 ** -24)
    b = plan.norm_exchange_backward(dev(dy), None, 0, dev(x), r.rstd)
    torch.cuda.synchronize()
    rs = cpu(r.rstd)
    ref.check_values(rs, rstd, torch.float32, "rstd")
    ref.check_values(cpu(r.out), y, TYPES[t], "out")
    want = ref.norm_backward(dy, None, 0, 2, h, rs)
    most = torch.finfo(TYPES[t]).max
    fits = bool((want[0].abs() < most).all())                   # fp16 holds no gradient of 2^50
    assert fits or t == "fp16"
    if fits:
        ref.check_backward(cpu(b.dx), None, None, want, ref.backward_terms(dy, None, 0, 2, h, rs), TYPES[t], 0, 2, "dx")
    plan.close()


def test_forward_and_backward_captured_together():
    """The operator's forward and backward pass in one graph, replayed on new
    inputs with eager work in between: the eager bits every time."""
    w, B, S, H, D = 2, 1, 300, 8, 64
    note("operator captured")
    p, a = (w, B, S, H, D), (w, B, S * w, H // w, D)
    x = values(p, torch.bfloat16, 1).to(DEV).requires_grad_(True)
    res = values(p, torch.bfloat16, 2).to(DEV).requires_grad_(True)
    weight = values((H * D,), torch.float32, 3).to(DEV).requires_grad_(True)
    gy, gs = values(a, torch.bfloat16, 4).to(DEV), values(p, torch.bfloat16, 5).to(DEV)

    def step():
        y, total = ops.norm_all_to_all_4D(x, weight, 2, 1, w, residual=res, checkpoint=E4M3)
        return (y, total) + torch.autograd.grad([y, total], [x, res, weight], [gy, gs])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [t.detach() for t in step()]
    for seed in (10, 20, 30):
        with torch.no_grad():
            for t, s in ((x, 0), (res, 1), (weight, 2), (gy, 3), (gs, 4)):
                t.copy_(values(tuple(t.shape), t.dtype, seed + s))
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in got]
        want = [t.detach() for t in step()]
        torch.cuda.synchronize()
        for k, e in zip(kept, want):
            assert torch.equal(k, e), seed


def test_one_plan_in_several_threads():
    """Calls of one plan from four threads on streams of their own: each thread's bits are its own."""
    plan = ua.Plan(4, 1, 400, 8, 64, torch.bfloat16, device=DEV)
    weight = values((512,), torch.float32, 1).to(DEV)
    sets = []
    for i in range(4):
        x, dy = values(plan.in_shape(0), torch.bfloat16, 10 + i).to(DEV), values(plan.out_shape(0), torch.bfloat16, 20 + i).to(DEV)
        starts = torch.tensor([3 * i], dtype=torch.int32, device=DEV)
        sets.append((x, dy, starts, ua.Cache(4, 8, 64, 1, 1700, E4M3, DEV)))

    def calls(x, dy, starts, cache, stream):
        f = plan.norm_exchange(x, weight, 0, checkpoint=E5M2, stream=stream)
        b = plan.norm_exchange_backward(dy, weight, 0, f.saved, f.rstd, saved_scales=f.saved_scales, stream=stream)
        plan.cache_write(cache, x, x, starts, stream=stream)
        k, v = plan.cache_read(cache, 1600, starts, stream=stream)
        return f.out, f.saved, f.rstd, b.dx, b.dweight, k, v

    want = [calls(*s, torch.cuda.current_stream()) for s in sets]
    torch.cuda.synchronize()
    got = [None] * 4

    def run(i):
        stream = torch.cuda.Stream()
        for _ in range(5):
            got[i] = calls(*sets[i], stream)
        stream.synchronize()

    threads = [threading.Thread(target=run, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for g, e in zip(got, want):
        for p, q in zip(g, e):
            assert torch.equal(cpu(p), cpu(q))
    plan.close()
