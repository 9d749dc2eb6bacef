"""GPU: backward norms whose workgroups walk over several segments each.

A backward launch has at most 512 to 1024 workgroups; these calls have more than
twice the segments those hold at once, all with gradients, so each workgroup's
sums of the weight's gradient, its two sets of registers in turn and the loads
ahead of the work take part in every result.

The weight's gradient: a lane adds up to five segments' products (twice as many
in bundles), then at most 6 exchanges between lanes, 64 joins in LDS, 128 rows and
16 waves: under 2^8 additions in a row, as in the other tests."""
from __future__ import annotations

import sys

import pytest
import torch

import ulysses_all_re_amd as ua
from tests import act_reference as ref
from tests.test_gpu_activations import E4M3, E5M2, TYPES, cpu, dev, values

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ua.load_library()
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()


# shape (w, B, S, H, D), per head, type
WALKS = [
    ((2, 1, 4801, 8, 64), False, "bf16"),      # a norm on 64 lanes of a wave
    ((1, 3, 25_667, 2, 24), False, "fp16"),    # on 8, with padding
    ((4, 1, 19_251, 4, 8), True, "fp32"),      # heads of 8 values in bundles
    ((2, 1, 1301, 3 * 2, 33), False, "bf16"),  # single values on a workgroup: one slot per lane,
    ((1, 1, 1303, 40, 33), False, "fp16"),     # and four
    ((3, 1, 3203, 12, 72), False, "bf16"),     # three slots per lane of a wave
    ((1, 1, 4203, 10, 128), False, "fp32"),    # five
    ((2, 1, 1061, 32, 128), False, "fp16"),     # four of two
    ((1, 1, 1601, 48, 128), False, "bf16"),    # three of four
    ((2, 1, 651, 80, 128), False, "bf16"),     # five of four
    ((1, 1, 1301, 88, 128), False, "bf16"),    # a workgroup of more than 256 lanes
    ((1, 1, 1301, 24, 264), False, "fp32"),    # the same, with padding
    ((2, 1, 4807, 16, 64), True, "fp16"),      # bundles of two slots per lane
    ((2, 1, 3203, 24, 64), True, "bf16"),      # of one
    ((2, 2, 4807, 6, 40), True, "bf16"),       # bundles on part of a wave, with padding
    ((5, 1, 1931, 5, 96), True, "bf16"),
    ((1, 1, 4103, 2, 640), True, "bf16"),      # a head on two slots per lane of a wave
]


def walk(shape, per_head, t, mode, save, residual, weight_type):
    w, B, S, H, D = shape
    dtype = TYPES[t]
    print(f"[gpu-case] walk {shape} head {per_head} {t} mode {mode} {save} residual {residual}", flush=True)
    sys.stdout.flush()
    plan = ua.Plan(*shape, dtype, device=DEV)
    p = plan.in_shape(0)
    h, dy = values(p, dtype, 1), values(plan.out_shape(mode), dtype, 2)
    dsum = values(p, dtype, 3) if residual else None
    weight = values((D if per_head else H * D,), weight_type, 4)
    _, h64, rstd = ref.norm(h, None, 0, w, None, per_head)
    rstd = rstd.float()
    if save:
        codes, scales = ref.quantise(h, save)
        saved, ss = dev(codes).view(save), dev(scales).view(torch.float8_e8m0fnu)
        h64 = ref.dequantise(codes, scales, save)
    else:
        saved, ss = dev(h if mode == 0 or residual else ref.to_a(h, w)), None
    b = plan.norm_exchange_backward(dev(dy), dev(weight), mode, saved, dev(rstd), saved_scales=ss, dsum=dev(dsum),
                                    residual=residual, per_head=per_head)
    torch.cuda.synchronize()
    want = ref.norm_backward(dy, weight, mode, w, h64, rstd, dsum, per_head)
    parts = ref.backward_terms(dy, weight, mode, w, h64, rstd, dsum, per_head)
    ref.check_backward(cpu(b.dx), cpu(b.dresidual) if residual and mode == 1 else None, cpu(b.dweight), want, parts, dtype,
                       mode, w, "walk")
    plan.close()


@pytest.mark.parametrize("shape,per_head,t", WALKS, ids=lambda v: "x".join(map(str, v)) if isinstance(v, tuple) else str(v))
@pytest.mark.parametrize("mode,save,residual", [(0, E4M3, False), (1, None, True), (1, E5M2, False), (0, None, True)],
                         ids=["checkpoint", "residual", "gathered", "sum"])
def test_walks(shape, per_head, t, mode, save, residual):
    walk(shape, per_head, t, mode, save, residual, torch.float32 if mode else TYPES[t])


def test_a_walk_without_a_weight_or_from_gathered_values():
    walk((2, 1, 4801, 8, 64), False, "bf16", 1, None, False, torch.bfloat16)
    walk((2, 1, 651, 80, 128), False, "bf16", 1, None, False, torch.float32)
    plan = ua.Plan(2, 1, 651, 80, 128, torch.bfloat16, device=DEV)
    h, dy = values(plan.in_shape(0), torch.bfloat16, 1), values(plan.out_shape(0), torch.bfloat16, 2)
    _, h64, rstd = ref.norm(h, None, 0, 2)
    rstd = rstd.float()
    b = plan.norm_exchange_backward(dev(dy), None, 0, dev(h), dev(rstd))
    torch.cuda.synchronize()
    assert b.dweight is None
    ref.check_backward(cpu(b.dx), None, None, ref.norm_backward(dy, None, 0, 2, h64, rstd),
                       ref.backward_terms(dy, None, 0, 2, h64, rstd), torch.bfloat16, 0, 2, "no weight")
    plan.close()
