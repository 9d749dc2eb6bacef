"""Activation calls at the edges of what they take: the host side, without a GPU."""
from __future__ import annotations

import pytest
import torch

import ulysses_all_re_amd as ua
from tests.test_binding_cpu import _host_plan


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
