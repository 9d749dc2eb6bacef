"""GPU: the norm operator (autograd, torch.compile), and the activation calls as
they are used: together, on other streams, captured and replayed, at sizes past
32-bit offsets, with rows of special values."""
from __future__ import annotations

import sys
import threading

import pytest
import torch

import ulysses_all_re_amd as ua
from tests import act_reference as ref
from tests.test_gpu_activations import E4M3, E5M2, cpu, dev, values
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


@pytest.mark.parametrize("mode", [0, 1])
@pytest.mark.parametrize("per_head", [False, True])
@pytest.mark.parametrize("checkpoint", [None, E4M3], ids=["values", "e4m3"])
def test_gradients_match_the_definition(mode, per_head, checkpoint):
    """x's, the weight's and the residual's gradients through autograd, with both outputs used."""
    w, B, S, H, D = 3, 2, 11, 6, 40
    note(f"ops gradients mode {mode} head {per_head} {checkpoint}")
    p, a = (w, B, S, H, D), (w, B, S * w, H // w, D)
    n = D if per_head else H * D
    for dtype, wt in ((torch.float32, torch.float32), (torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32)):
        x = values(p if mode == 0 else a, dtype, 1)
        res, weight = values(p, dtype, 2), values((n,), wt, 3)
        xd, rd, wd = (t.to(DEV).requires_grad_(True) for t in (x, res, weight))
        dims = (2, 1) if mode == 0 else (1, 2)
        y, total = ops.norm_all_to_all_4D(xd, wd, *dims, w, residual=rd, per_head=per_head, checkpoint=checkpoint)
        gy, gs = values(tuple(y.shape), dtype, 4), values(p, dtype, 5)
        torch.autograd.backward([y, total], [gy.to(DEV), gs.to(DEV)])
        _, h, rstd = ref.norm(x, weight, mode, w, res, per_head)
        hq = ref.dequantise(*ref.quantise(h, checkpoint), checkpoint) if checkpoint else h
        want = ref.norm_backward(gy, weight, mode, w, hq, rstd, gs, per_head)
        parts = ref.backward_terms(gy, weight, mode, w, hq, rstd, gs, per_head)
        ref.check_backward(xd.grad.cpu(), rd.grad.cpu(), None, want, parts, dtype, mode, w, "ops")
        bound = parts[1] * 2.0 ** -16 + want[2].abs() * ref.HALF[wt] + 1e-30
        ref.assert_close(wd.grad.cpu(), want[2], bound, "dweight")
        # without the residual, and only its sum used
        xd.grad = None
        y = ops.norm_all_to_all_4D(xd, None, *dims, w, per_head=per_head, checkpoint=checkpoint)
        y.backward(gy.to(DEV))
        _, h, rstd = ref.norm(x, None, mode, w, None, per_head)
        hq = ref.dequantise(*ref.quantise(h, checkpoint), checkpoint) if checkpoint else h
        want = ref.norm_backward(gy, None, mode, w, hq, rstd, None, per_head)
        parts = ref.backward_terms(gy, None, mode, w, hq, rstd, None, per_head)
        ref.check_backward(xd.grad.cpu(), None, None, want, parts, dtype, mode, w, "no residual")
        xd.grad = None
        _, total = ops.norm_all_to_all_4D(xd, wd, *dims, w, residual=rd, per_head=per_head, checkpoint=checkpoint)
        total.backward(gs.to(DEV))
        back = gs if mode == 0 else ref.to_a(gs, w)
        assert torch.equal(xd.grad.cpu(), back)


def test_gradient_matches_differences():
    """The gradient of <g, out> along random directions against central
    differences of the definition in 64 bits (their error, about the third
    derivative times h^2 / 6 with h = 1e-5, is far below the operator's)."""
    w, B, S, H, D = 2, 1, 3, 4, 8
    for mode in (0, 1):
        for per_head in (False, True):
            p, a = (w, B, S, H, D), (w, B, S * w, H // w, D)
            x, weight = values(p if mode == 0 else a, torch.float32, 1), values((D if per_head else H * D,), torch.float32, 2)
            xd, wd = x.to(DEV).requires_grad_(True), weight.to(DEV).requires_grad_(True)
            y = ops.norm_all_to_all_4D(xd, wd, *((2, 1) if mode == 0 else (1, 2)), w, per_head=per_head)
            g = values(tuple(y.shape), torch.float32, 3)
            y.backward(g.to(DEV))
            for seed in (4, 5, 6):
                u, v = values(tuple(x.shape), torch.float64, seed), values(tuple(weight.shape), torch.float64, seed + 9)
                h = 1e-5
                f = [(ref.norm(x.double() + s * h * u, weight.double() + s * h * v, mode, w, None, per_head)[0]
                      * g.double()).sum() for s in (1, -1)]
                want = float(f[0] - f[1]) / (2 * h)
                parts = [(xd.grad.cpu().double() * u), (wd.grad.cpu().double() * v)]
                got = sum(float(t.sum()) for t in parts)
                size = sum(float(t.abs().sum()) for t in parts)
                assert abs(got - want) <= 1e-5 * size, (mode, per_head, got, want)


def test_gradients_of_shared_and_broadcast_inputs():
    """One weight for queries and keys; a gradient that autograd hands over as
    an expanded scalar; a residual that is the input itself."""
    w, B, S, H, D = 2, 1, 5, 4, 16
    q, k = values((w, B, S, H, D), torch.float32, 1), values((w, B, S, H, D), torch.float32, 2)
    weight = values((D,), torch.float32, 3)
    qd, kd, wd = (t.to(DEV).requires_grad_(True) for t in (q, k, weight))
    y = ops.norm_all_to_all_4D(qd, wd, 2, 1, w, per_head=True) + ops.norm_all_to_all_4D(kd, wd, 2, 1, w, per_head=True)
    y.sum().backward()
    one = torch.ones(w, B, S * w, H // w, D)
    dw, terms = 0, 0
    for t in (q, k):
        _, h, rstd = ref.norm(t, weight, 0, w, None, True)
        dw = dw + ref.norm_backward(one, weight, 0, w, h, rstd, None, True)[2]
        terms = terms + ref.backward_terms(one, weight, 0, w, h, rstd, None, True)[1]
    ref.assert_close(wd.grad.cpu(), dw, terms * 2.0 ** -16, "shared weight")
    xd = q.to(DEV).requires_grad_(True)
    y, total = ops.norm_all_to_all_4D(xd, None, 2, 1, w, residual=xd)
    (y.sum() + total.sum()).backward()
    _, h, rstd = ref.norm(q, None, 0, w, q)
    one_p = torch.ones_like(q)
    want = ref.norm_backward(one, None, 0, w, h, rstd, one_p)[1] * 2
    bound = ref.backward_terms(one, None, 0, w, h, rstd, one_p)[0] * 2 * ref.SUM + want.abs() * 2.0 ** -22
    ref.assert_close(xd.grad.cpu(), want, bound, "x as its own residual")


def test_checkpoint_keeps_eight_bits():
    """With a checkpoint autograd keeps the codes, their scales, rstd and the weight -- not the values."""
    w, B, S, H, D = 2, 1, 64, 4, 64
    x = values((w, B, S, H, D), torch.bfloat16, 1).to(DEV).requires_grad_(True)
    weight = values((H * D,), torch.bfloat16, 2).to(DEV).requires_grad_(True)
    sizes = {}
    for checkpoint in (None, E4M3):
        kept = []
        with torch.autograd.graph.saved_tensors_hooks(lambda t: kept.append(t) or t, lambda t: t):
            y = ops.norm_all_to_all_4D(x, weight, 2, 1, w, checkpoint=checkpoint)
        sizes[checkpoint] = sum(t.numel() * t.element_size() for t in kept if t.dtype != weight.dtype or t.numel() != H * D)
        y.sum().backward()
    n = x.numel()
    assert sizes[None] == 2 * n + 4 * w * B * S
    assert sizes[E4M3] == n + n // 32 + 4 * w * B * S
    with torch.no_grad():
        y = ops.norm_all_to_all_4D(x, weight, 2, 1, w, checkpoint=E4M3)
    assert not y.requires_grad


def test_strided_and_compiled():
    """Strided inputs and gradients are laid out by the operator; a compiled call gives the same bits."""
    w, B, S, H, D = 2, 2, 7, 4, 32
    base = values((w, B, S, D, H), torch.bfloat16, 1).to(DEV)
    x = base.transpose(3, 4)
    weight = values((2 * H * D,), torch.bfloat16, 2).to(DEV)[::2]
    y = ops.norm_all_to_all_4D(x, weight, 2, 1, w)
    assert torch.equal(y, ops.norm_all_to_all_4D(x.contiguous(), weight.contiguous(), 2, 1, w))

    def f(x, weight):
        y = ops.norm_all_to_all_4D(x * 2, weight, 2, 1, w, checkpoint=E5M2)
        return (y * y).sum()

    grads = []
    for fn in (f, torch.compile(f, fullgraph=True, backend="aot_eager")):
        xd, wd = x.detach().contiguous().requires_grad_(True), weight.detach().contiguous().requires_grad_(True)
        fn(xd, wd).backward()
        grads.append((xd.grad, wd.grad))
    assert torch.equal(grads[0][0], grads[1][0]) and torch.equal(grads[0][1], grads[1][1])


def test_repeated_calls_give_the_same_bits():
    """dweight is summed in a fixed order."""
    plan = ua.Plan(4, 1, 900, 8, 64, torch.bfloat16, device=DEV)
    x, weight = values(plan.in_shape(0), torch.bfloat16, 1).to(DEV), values((512,), torch.float32, 2).to(DEV)
    dy = values(plan.out_shape(0), torch.bfloat16, 3).to(DEV)
    f = plan.norm_exchange(x, weight, 0, checkpoint=E4M3)
    first = plan.norm_exchange_backward(dy, weight, 0, f.saved, f.rstd, saved_scales=f.saved_scales)
    for _ in range(5):
        g = plan.norm_exchange(x, weight, 0, checkpoint=E4M3, out=f)
        b = plan.norm_exchange_backward(dy, weight, 0, g.saved, g.rstd, saved_scales=g.saved_scales)
        assert torch.equal(b.dweight, first.dweight) and torch.equal(b.dx, first.dx)
    plan.close()


def _block(plan, q, k, v, wq, cache, starts, counts):
    """What a sequence-parallel attention layer does around its attention: query
    norm and exchange, new keys and values into the cache, the cache read back."""
    y = plan.norm_exchange(q, wq, 0, per_head=True)
    plan.cache_write(cache, k, v, starts, counts)
    kk, vv = plan.cache_read(cache, cache.capacity)
    z = plan.norm_exchange(y.out, None, 1, residual=q, out_dtype=E4M3)
    return y.out, kk, vv, z.out, z.scales, z.sum


def test_a_layer_together_captured_and_replayed():
    """The calls of a layer in a row, eager and captured; replays see new inputs,
    with eager work between them, and equal the eager results bit for bit."""
    w, B, S, H, D = 4, 2, 6, 8, 64
    plan = ua.Plan(w, B, S, H, D, torch.float16, device=DEV)
    wq = values((D,), torch.float16, 1).to(DEV)
    q, k, v = (values(plan.in_shape(0), torch.float16, s).to(DEV) for s in (2, 3, 4))
    starts = torch.tensor([3, 7], dtype=torch.int32, device=DEV)
    counts = torch.tensor([S * w, 5], dtype=torch.int32, device=DEV)
    cache, eager_cache = ua.Cache(w, H, D, B, 40, E5M2, DEV), ua.Cache(w, H, D, B, 40, E5M2, DEV)
    note("layer, eager and captured")
    _block(plan, q, k, v, wq, cache, starts, counts)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = _block(plan, q, k, v, wq, cache, starts, counts)
    for seed in (10, 20, 30, 40):
        for t, s in ((q, 0), (k, 1), (v, 2)):
            t.copy_(values(plan.in_shape(0), torch.float16, seed + s))
        starts.copy_(torch.tensor([seed // 10, 12 - seed // 10], dtype=torch.int32))
        graph.replay()
        want = _block(plan, q, k, v, wq, eager_cache, starts, counts)
        torch.cuda.synchronize()
        if seed == 10:                                  # the caches started from different histories
            cache.codes.view(torch.uint8).copy_(eager_cache.codes.view(torch.uint8))
            cache.scales.view(torch.uint8).copy_(eager_cache.scales.view(torch.uint8))
            graph.replay()
            torch.cuda.synchronize()
        for g, e in zip(got, want):
            assert torch.equal(cpu(g), cpu(e)), seed
        assert torch.equal(cpu(cache.codes), cpu(eager_cache.codes))
    y, h, _ = ref.norm(q.cpu(), wq.cpu(), 0, w, None, True)
    ref.check_values(cpu(got[0]), y, torch.float16, "layer")
    plan.close()


def test_two_captured_backward_passes_share_no_workspace():
    """Two graphs with backward calls of different inputs, replayed in turn."""
    plan = ua.Plan(2, 1, 300, 4, 64, torch.bfloat16, device=DEV)
    weight = values((256,), torch.bfloat16, 1).to(DEV)
    sets = []
    for seed in (10, 20):
        x, dy = values(plan.in_shape(0), torch.bfloat16, seed).to(DEV), values(plan.out_shape(0), torch.bfloat16, seed + 1).to(DEV)
        f = plan.norm_exchange(x, weight, 0, checkpoint=E4M3)
        want = plan.norm_exchange_backward(dy, weight, 0, f.saved, f.rstd, saved_scales=f.saved_scales)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = plan.norm_exchange_backward(dy, weight, 0, f.saved, f.rstd, saved_scales=f.saved_scales)
        sets.append((graph, got, want, (x, dy, f)))         # a graph holds no references to its inputs
    for _ in range(3):
        for graph, got, _, _ in sets:
            got.dx.zero_()
            got.dweight.zero_()
            graph.replay()
        torch.cuda.synchronize()
        for _, got, want, _ in sets:
            assert torch.equal(got.dx, want.dx) and torch.equal(got.dweight, want.dweight)
    plan.close()


def test_other_streams_and_threads():
    """Calls on side streams (results and workspaces belong to them), and one
    plan each in several threads at once."""
    plan = ua.Plan(2, 1, 500, 4, 64, torch.bfloat16, device=DEV)
    x, weight = values(plan.in_shape(0), torch.bfloat16, 1).to(DEV), values((256,), torch.bfloat16, 2).to(DEV)
    dy = values(plan.out_shape(0), torch.bfloat16, 3).to(DEV)
    want = plan.norm_exchange(x, weight, 0, checkpoint=E4M3)
    wantb = plan.norm_exchange_backward(dy, weight, 0, want.saved, want.rstd, saved_scales=want.saved_scales)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(4):
        got = plan.norm_exchange(x, weight, 0, checkpoint=E4M3, stream=side)
        b = plan.norm_exchange_backward(dy, weight, 0, got.saved, got.rstd, saved_scales=got.saved_scales, stream=side)
        junk = [torch.full((1 << 18,), 7.0, device=DEV) for _ in range(8)]      # reuses no memory of the side stream's
        side.synchronize()
        assert torch.equal(got.out, want.out) and torch.equal(b.dx, wantb.dx) and torch.equal(b.dweight, wantb.dweight)
        del junk
    results = [None] * 4

    def run(i):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            y = ops.norm_all_to_all_4D(x, weight, 2, 1, 2)
        stream.synchronize()
        results[i] = y

    threads = [threading.Thread(target=run, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert all(torch.equal(r, want.out) for r in results)
    plan.close()


def test_rows_of_special_values():
    """Rows of zeros, of NaN and of infinities: as the definition has them, and no other row is touched."""
    for t in (torch.bfloat16, torch.float32):
        plan = ua.Plan(2, 1, 6, 4, 64, t, device=DEV)
        x = values(plan.in_shape(0), t, 1)
        x[0, 0, 1] = 0
        x[0, 0, 2, 1, 5] = float("nan")
        x[1, 0, 3, 2, 7] = float("inf")
        x[1, 0, 4] = torch.finfo(t).max / 4                     # squares overflow: rstd is zero
        weight = values((256,), t, 2)
        for per_head in (False, True):
            wt = weight[:64] if per_head else weight
            r = plan.norm_exchange(dev(x), dev(wt), 0, per_head=per_head, checkpoint=E5M2, rstd=True)
            torch.cuda.synchronize()
            ref.check_same_codes(cpu(r.saved), cpu(r.saved_scales), x, E5M2, "special")
            h = x.float()                                       # sums of squares overflow in 32 bits
            ms = (h * h).mean(-1, keepdim=True) if per_head else (h * h).mean((-2, -1), keepdim=True)
            y = h.double() * (1.0 / torch.sqrt(ms + 1e-6)).double()
            y = y * (wt.double() if per_head else wt.double().view(4, 64))
            ref.check_values(cpu(r.out), ref.to_a(y, 2), t, "special rows")
        plan.close()


def test_offsets_past_32_bits():
    """A cache of over 2^32 codes a part, and a tensor of over 2^32 values."""
    note("long cache")
    w, H, D, cap = 1, 8, 128, 4_400_000
    cache = ua.Cache(w, H, D, 1, cap, E4M3, DEV)
    plan = ua.Plan(w, 1, 64, H, D, torch.bfloat16, device=DEV)
    k, v = values(plan.in_shape(0), torch.bfloat16, 1), values(plan.in_shape(0), torch.bfloat16, 2)
    starts = torch.tensor([cap - 70], dtype=torch.int32, device=DEV)
    plan.cache_write(cache, dev(k), dev(v), starts)
    kk, vv = plan.cache_read(cache, 80, starts)
    torch.cuda.synchronize()
    for got, x in ((kk, k), (vv, v)):
        q, s = ref.quantise(x, E4M3)
        want = ref.dequantise(q, s, E4M3).bfloat16().view(1, 1, 64, H, D)
        assert torch.equal(got.cpu()[:, :, :64], want) and not bool(got[:, :, 64:].any())
    assert not bool(cache.codes.view(torch.uint8)[:, :, :, :cap - 70].any())
    assert not bool(cache.codes.view(torch.uint8)[:, :, :, cap - 6:].any())
    plan.close()
    del cache, kk, vv
    torch.cuda.empty_cache()
    note("large tensor")
    w, B, S, H, D = 2, 3, 100_000, 64, 128                      # 4.9e9 values
    plan = ua.Plan(w, B, S, H, D, torch.bfloat16, device=DEV)
    x = torch.empty(plan.in_shape(0), dtype=torch.bfloat16, device=DEV)
    x.fill_(0.5)
    tail = values((50, H, D), torch.bfloat16, 3)
    x[-1, -1, -50:] = tail.to(DEV)
    weight = values((H * D,), torch.bfloat16, 4).to(DEV)
    r = plan.norm_exchange(x, weight, 0, checkpoint=E4M3)
    torch.cuda.synchronize()
    y, h, rstd = ref.norm(tail.view(1, 1, 50, H, D), weight.cpu(), 0, 1)
    got = torch.cat([r.out[0, -1, -50:], r.out[1, -1, -50:]], 1).cpu()
    ref.check_values(got, y.view(50, H, D), torch.bfloat16, "tail")
    ref.check_same_codes(cpu(r.saved[-1, -1, -50:]), cpu(r.saved_scales[-1, -1, -50:]), tail, E4M3, "tail codes")
    dy = torch.zeros(plan.out_shape(0), dtype=torch.bfloat16, device=DEV)
    gy = values((50, H, D), torch.bfloat16, 5)
    dy[0, -1, -50:], dy[1, -1, -50:] = gy[:, :32].to(DEV), gy[:, 32:].to(DEV)
    b = plan.norm_exchange_backward(dy, weight, 0, r.saved, r.rstd, saved_scales=r.saved_scales)
    torch.cuda.synchronize()
    hq = ref.dequantise(*ref.quantise(tail, E4M3), E4M3).view(1, 1, 50, H, D)
    rs = r.rstd[-1, -1, -50:].cpu().view(1, 1, 50)
    gy = gy.view(1, 1, 50, H, D)
    want = ref.norm_backward(gy, weight.cpu(), 0, 1, hq, rs)
    parts = ref.backward_terms(gy, weight.cpu(), 0, 1, hq, rs)
    ref.check_backward(b.dx[-1:, -1:, -50:].cpu(), None, b.dweight.cpu(), want, parts, torch.bfloat16, 0, 1, "tail")
    assert not bool(b.dx[0].any())
    plan.close()


def test_one_token_for_each_sequence_step_by_step():
    """Tokens of 24 sequences written one at a time (some idle) hold what one prompt's write holds."""
    w, S, H, D = 4, 6, 8, 80
    plan = ua.Plan(w, 1, S, H, D, torch.bfloat16, device=DEV)
    cache = ua.Cache(w, H, D, S * w, 9, E4M3, DEV)
    codes, scales = torch.zeros(cache.codes.shape, dtype=torch.uint8), torch.zeros(cache.scales.shape, dtype=torch.uint8)
    length = torch.zeros(S * w, dtype=torch.int32)
    for step in range(12):                                      # past the capacity at the end
        k, v = values(plan.in_shape(0), torch.bfloat16, 2 * step), values(plan.in_shape(0), torch.bfloat16, 2 * step + 1)
        on = torch.tensor([(i + step) % 5 != 0 for i in range(S * w)], dtype=torch.int32)
        plan.cache_write(cache, dev(k), dev(v), dev(length), dev(on))
        for part, t in ((0, k), (1, v)):
            ref.cache_write(codes, scales, t, E4M3, w, length.tolist(), on.tolist(), part)
        length += on
    torch.cuda.synchronize()
    assert bool((cpu(cache.codes) == codes).all()) and bool((cpu(cache.scales) == scales).all())
    plan.close()


def test_library_refuses_overlap_on_the_device():
    """In-place and overlapping calls are errors, and the plan stays usable."""
    plan = ua.Plan(2, 1, 8, 4, 16, torch.bfloat16, device=DEV)
    x = values(plan.in_shape(0), torch.bfloat16, 1).to(DEV)
    with pytest.raises(ua.UA2AError) as e:
        plan.norm_exchange(x, None, 0, out=ua.NormExchange(x.view(plan.out_shape(0))))
    assert e.value.code == ua.UA2A_ERR_ALIAS
    with pytest.raises(ua.UA2AError) as e:
        plan.norm_exchange(x, None, 0, eps=0.0)
    assert e.value.code == ua.UA2A_ERR_INVALID_ARG
    out = torch.zeros(2, 1, 4, 2, 16, dtype=torch.bfloat16, device=DEV)
    cache = ua.Cache(2, 4, 16, 1, 4, E4M3, DEV)
    with pytest.raises(ua.UA2AError) as e:
        plan.cache_read(cache, 4, out=(out, out))
    assert e.value.code == ua.UA2A_ERR_ALIAS
    y = plan.norm_exchange(x, None, 0)
    torch.cuda.synchronize()
    ref.check_values(y.out.cpu(), ref.norm(x.cpu(), None, 0, 2)[0], torch.bfloat16, "after refusals")
    plan.close()
