"""The attention operators' host side in Python: shapes of fake tensors, refusals,
rotary tables, the header.  No GPU needed."""
from __future__ import annotations

import os
import re
import subprocess
from fractions import Fraction

import pytest
import torch

import ulysses_all_re_amd as ua
from tests import attn_reference as ref
from tests.test_binding_cpu import _host_plan
from ulysses_all_re_amd import attention, ops

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "ua2a_attn.h")


def test_header_binding_and_library_agree():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    declared = sorted(set(re.findall(r"^\s*int\s+(ua2a_\w+)\s*\(", text, flags=re.M)))
    assert declared == sorted(attention.EXPORTED)
    syms = subprocess.check_output(["nm", "-D", "--defined-only", ua.LIBRARY], text=True)
    exported = {line.split()[-1] for line in syms.splitlines() if " T " in line}
    assert set(declared) <= exported


def test_header_is_plain_c_and_structures_agree(tmp_path):
    names = ("rope", "window", "attention", "attention_grad", "cache_attention")
    body = "".join(f'printf("%zu\\n", sizeof(ua2a_{n}_t));' for n in names)
    exe = tmp_path / "sizes"
    code = f'#include "ua2a_attn.h"\n#include <stdio.h>\nint main(void) {{ {body} return 0; }}\n'
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-pedantic", "-Werror", "-x", "c", "-I", os.path.dirname(HEADER),
                    "-", "-o", str(exe)], input=code, text=True, check=True, timeout=60)
    import ctypes
    sizes = [int(x) for x in subprocess.check_output([str(exe)], text=True).split()]
    assert sizes == [ctypes.sizeof(getattr(attention, f"ua2a_{n}_t")) for n in names]


def test_rotary_turns():
    """Each entry is the frequency over 2 pi, modulo one, to 64 bits."""
    for freqs in ([1.0, 10000.0 ** -0.5, 1e-9, 0.0], [-0.25, 100.0, 6.283185307179586, 1e6]):
        r = ua.Rotary.of(16, freqs, [0] * len(freqs), device="cpu")
        for f, t in zip(freqs, r.turns.tolist()):
            want = (Fraction(f) / ref.TURN) % 1
            assert abs(Fraction(t % (1 << 64), 1 << 64) - want) <= Fraction(1, 1 << 63), f
    r = ua.Rotary(32, (8, 4, 6), device="cpu")
    assert (r.pairs, r.naxes, r.axes.tolist()) == (9, 3, [0] * 4 + [1] * 2 + [2] * 3)
    assert r.turns.dtype == torch.int64 and r.axes.dtype == torch.int32 and not r.halves


@pytest.mark.parametrize("make,match", [
    (lambda: ua.Rotary(16, (18,), device="cpu"), "dims"), (lambda: ua.Rotary(16, (3,), device="cpu"), "dims"),
    (lambda: ua.Rotary(16, (), device="cpu"), "dims"), (lambda: ua.Rotary(16, (0, 0), device="cpu"), "dims"),
    (lambda: ua.Rotary(16, (-2, 8), device="cpu"), "dims"), (lambda: ua.Rotary(16, (8,), theta=0.0, device="cpu"), "theta"),
    (lambda: ua.Rotary(16, (8,), theta=float("nan"), device="cpu"), "theta"),
    (lambda: ua.Rotary.of(16, [], [], device="cpu"), "frequencies"), (lambda: ua.Rotary.of(4, [1.0] * 3, [0] * 3, device="cpu"), "at most"),
    (lambda: ua.Rotary.of(16, [1.0], [0, 1], device="cpu"), "axes"),
    (lambda: ua.Rotary.of(16, [float("inf")], [0], device="cpu"), "finite"),
    (lambda: ua.Rotary.of(16, [1.0], [-1], device="cpu"), "axes")])
def test_rotary_refusals(make, match):
    with pytest.raises(ValueError, match=match):
        make()


class Calls:
    """Stands in for the library: what each call would have passed."""

    def __init__(self, plan):
        self.seen = []
        plan._issue = lambda name, stream, *args: self.seen.append((name, args))


def test_rope_arguments():
    plan = _host_plan(w=2, B=3, S=4, H=4, D=16)
    calls = Calls(plan)
    r = ua.Rotary(16, (6, 6), device="cpu")
    x, y = torch.zeros(plan.in_shape(0), dtype=torch.bfloat16), torch.zeros(plan.out_shape(0), dtype=torch.bfloat16)
    flat, planes = torch.zeros(2, 8, dtype=torch.int32), torch.zeros(2, 3, 8, dtype=torch.int32)
    assert plan.rope_exchange(x, r, flat, 0).shape == plan.out_shape(0)
    assert plan.rope_exchange(y, r, planes, 1).shape == plan.in_shape(0)
    assert plan.rope(y, r, planes[:, :1].contiguous(), gathered=True, out=y) is y
    seen = [c[1][0]._obj for c in calls.seen]
    assert [(s.from_, s.to, s.per_plane) for s in seen] == [(0, 1, 0), (1, 0, 1), (1, 1, 0)]
    for bad, error in ((lambda: plan.rope_exchange(y, r, flat, 0), ValueError), (lambda: plan.rope_exchange(x, r, flat, 2), ValueError),
                       (lambda: plan.rope_exchange(x.float(), r, flat, 0), TypeError),
                       (lambda: plan.rope_exchange(x, r, flat.long(), 0), TypeError),
                       (lambda: plan.rope_exchange(x, r, flat[:1], 0), ValueError),
                       (lambda: plan.rope_exchange(x, r, flat[:, :7], 0), ValueError),
                       (lambda: plan.rope_exchange(x, r, planes.transpose(1, 2).contiguous().transpose(1, 2), 0), ValueError),
                       (lambda: plan.rope_exchange(x, ua.Rotary(32, (6, 6), device="cpu"), flat, 0), ValueError),
                       (lambda: plan.rope(x, r, flat, out=y), ValueError)):
        with pytest.raises(error):
            bad()
    assert len(calls.seen) == 3
    eight = _host_plan(w=2, B=3, S=4, H=4, D=16, dtype=torch.float64)
    with pytest.raises(TypeError):
        eight.rope(torch.zeros(eight.in_shape(0), dtype=torch.float64), r, flat)


def test_attention_arguments():
    plan = _host_plan(w=2, B=3, S=4, H=8, D=16)
    calls = Calls(plan)
    q = torch.zeros(plan.out_shape(0), dtype=torch.bfloat16)
    k = torch.zeros(2, 3, 8, 2, 16, dtype=torch.bfloat16)
    counts = torch.zeros(3, dtype=torch.int32)
    r = plan.window_attention(q, k, k, left=3, right=0, sinks=1, chunk=2, counts=counts, lse=True, scale=0.7)
    assert r.out.shape == q.shape and r.lse.shape == (2, 3, 4, 8)
    args = calls.seen[-1][1][0]._obj
    assert (args.window.left, args.window.right, args.window.sinks, args.window.chunk, args.kv_heads) == (3, 0, 1, 2, 4)
    assert plan.window_attention(q, k, k).lse is None
    assert calls.seen[-1][1][0]._obj.scale == 0.25 and calls.seen[-1][1][0]._obj.window.left == -1
    g = plan.window_attention_backward(q, q, k, k, r.out, r.lse, left=3)
    assert [t.shape for t in g] == [q.shape, k.shape, k.shape] and calls.seen[-1][1][0]._obj.workspace_bytes > 0
    done = len(calls.seen)
    for bad, error in ((lambda: plan.window_attention(q[:, :2], k, k), ValueError), (lambda: plan.window_attention(q, k[..., :8], k), ValueError),
                       (lambda: plan.window_attention(q, k, k[:, :, :4]), ValueError), (lambda: plan.window_attention(q, q[:, :, :, :3].contiguous(), k), ValueError),
                       (lambda: plan.window_attention(q, k.half(), k), TypeError), (lambda: plan.window_attention(q, k, k, left=-1), ValueError),
                       (lambda: plan.window_attention(q, k, k, sinks=-1), ValueError), (lambda: plan.window_attention(q, k, k, chunk=0), ValueError),
                       (lambda: plan.window_attention(q, k, k, left=1 << 31), ValueError), (lambda: plan.window_attention(q, k, k, scale=0.0), ValueError),
                       (lambda: plan.window_attention(q, k, k, scale=float("nan")), ValueError),
                       (lambda: plan.window_attention(q, k, k, counts=counts.long()), TypeError),
                       (lambda: plan.window_attention(q, k, k, counts=counts[:2]), ValueError),
                       (lambda: plan.window_attention(q, k, k, lse=True, out=ua.Attention(q)), ValueError),
                       (lambda: plan.window_attention_backward(q, q, k, k, q, r.lse[0]), ValueError),
                       (lambda: plan.window_attention_backward(q, q, k, k, q, r.lse, grads=(q, k, q)), ValueError)):
        with pytest.raises(error):
            bad()
    assert len(calls.seen) == done
    for dtype, D, error in ((torch.float32, 16, TypeError), (torch.bfloat16, 12, ValueError), (torch.bfloat16, 136, ValueError)):
        other = _host_plan(w=2, B=3, S=4, H=8, D=D, dtype=dtype)
        t = torch.zeros(other.out_shape(0), dtype=dtype)
        with pytest.raises(error, match="attention"):
            other.window_attention(t, t, t)


def test_cache_attention_arguments():
    plan = _host_plan(w=2, B=1, S=1, H=8, D=16)
    calls = Calls(plan)
    cache = ua.Cache(2, 4, 16, 3, 50, device="cpu")
    q, starts = torch.zeros(2, 3, 5, 4, 16, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)
    out = plan.cache_attention(cache, q, starts, starts, left=7, sinks=2)
    assert out.shape == q.shape
    args = calls.seen[-1][1][1]._obj
    assert (args.n, args.kv_heads, args.window.right, args.window.left) == (5, 4, 0, 7)
    for bad, error in ((lambda: plan.cache_attention(cache, q, None), ValueError), (lambda: plan.cache_attention(cache, q[:, :2], starts), ValueError),
                       (lambda: plan.cache_attention(cache, q[:, :, :0], starts), ValueError), (lambda: plan.cache_attention(cache, q.half(), starts), TypeError),
                       (lambda: plan.cache_attention(cache, q, starts.long()), TypeError), (lambda: plan.cache_attention(cache, q, starts[:2]), ValueError),
                       (lambda: plan.cache_attention(cache, q, starts, out=q[:, :, :4]), ValueError),
                       (lambda: plan.cache_attention(ua.Cache(2, 6, 16, 3, 50, device="cpu"), q, starts), ValueError),
                       (lambda: plan.cache_attention(ua.Cache(1, 4, 16, 3, 50, device="cpu"), q, starts), ValueError),
                       (lambda: plan.cache_attention(ua.Cache(2, 4, 8, 3, 50, device="cpu"), q, starts), ValueError)):
        with pytest.raises(error):
            bad()


def test_fake_shapes_and_gradients():
    w, B, S, H, D = 2, 3, 8, 4, 16
    r = ua.Rotary(D, (8, 8), device="cpu")
    pos = torch.empty((2, S * w), device="meta", dtype=torch.int32)
    meta = ua.Rotary.__new__(ua.Rotary)
    meta.__dict__.update(r.__dict__, turns=r.turns.to("meta"), axes=r.axes.to("meta"))
    x = torch.empty((w, B, S, H, D), device="meta", requires_grad=True)
    q = ops.rope_all_to_all_4D(x, meta, pos, 2, 1, w)
    assert q.shape == (w, B, S * w, H // w, D)
    assert ops.rope_all_to_all_4D(q, meta, pos, 1, 2, w, inverse=True).shape == x.shape
    k = torch.empty((w, B, S * w, 1, D), device="meta", requires_grad=True)
    o = ops.window_attention(q, k, k, w, left=4, right=0, sinks=1)
    assert o.shape == q.shape
    o.sum().backward()
    assert x.grad.shape == x.shape and k.grad.shape == k.shape
    with pytest.raises(ValueError, match="unsupported"):
        ops.rope_all_to_all_4D(x, meta, pos, 3, 1, w)
    with pytest.raises(RuntimeError, match="GPU only"):
        ops.rope_all_to_all_4D(torch.zeros(w, B, S, H, D), r, torch.zeros(2, S * w, dtype=torch.int32), 2, 1, w)
    with pytest.raises(RuntimeError, match="GPU only"):
        ops.window_attention(*[torch.zeros(w, B, S * w, 2, D)] * 3, w)


def test_rotary_tables_are_checked():
    """A rotary's tensors that were replaced, or an operator's of other sizes, never reach the library."""
    plan = _host_plan(w=2, B=3, S=4, H=4, D=16)
    calls = Calls(plan)
    x, flat = torch.zeros(plan.in_shape(0), dtype=torch.bfloat16), torch.zeros(2, 8, dtype=torch.int32)
    for change, error in ((dict(turns=torch.zeros(5, dtype=torch.int64)), ValueError), (dict(turns=torch.zeros(6, dtype=torch.int32)), TypeError),
                          (dict(turns=torch.zeros(12, dtype=torch.int64)[::2]), ValueError), (dict(axes=torch.zeros(5, dtype=torch.int32)), ValueError),
                          (dict(axes=torch.zeros(6, dtype=torch.int64)), TypeError), (dict(axes=torch.zeros(6, device="meta", dtype=torch.int32)), ValueError)):
        r = ua.Rotary(16, (6, 6), device="cpu")
        r.__dict__.update(change)
        with pytest.raises(error, match="rotary"):
            plan.rope_exchange(x, r, flat, 0)
        if "axes" in change:                                   # as the operator makes it from its tensors
            with pytest.raises(error, match="rotary"):
                plan.rope_exchange(x, ops._rotary(16, r.turns, r.axes, 2, False), flat, 0)
    assert not calls.seen
    with pytest.raises(ValueError, match="heads of 32"):
        ops.rope_all_to_all_4D(x, ua.Rotary(32, (6, 6), device="cpu"), flat, 2, 1, 2)


def test_a_scale_in_a_tensor_is_read_at_each_call():
    plan = _host_plan(w=2, B=3, S=4, H=8, D=16)
    calls = Calls(plan)
    q = torch.zeros(plan.out_shape(0), dtype=torch.bfloat16)
    scale, left = torch.tensor(0.5), torch.tensor(3)
    for value in (0.5, 0.25, 2.0):
        scale.fill_(value)
        left.fill_(int(value * 4))
        plan.window_attention(q, q, q, scale=scale, left=left)
        args = calls.seen[-1][1][0]._obj
        assert (args.scale, args.window.left) == (value, int(value * 4))
    for scale in (1e-40, 3e38, float("inf")):
        with pytest.raises(ValueError, match="scale"):
            plan.window_attention(q, q, q, scale=scale)
