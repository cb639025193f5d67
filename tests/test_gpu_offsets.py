"""pa_norm_rope_write_kv into the last blocks of a pool of 4.9e9 elements: K and V,
both cache types, both pairings, have the bits of the same call into a small
pool."""
from __future__ import annotations

import pytest
import torch

from tests import test_gpu_norm_rope as tn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fp8", [False, True])
def test_writes_past_32_bits(pa_lib, fp8):
    from paged_kv_cache_42_gb300 import binding
    binding.get_device_error(True)
    blocks, small = 300000, 12
    dtype = torch.uint8 if fp8 else torch.bfloat16
    big = [torch.empty(blocks, 8, 16, 128, dtype=dtype, device="cuda") for _ in "kv"]
    for T, norm, inter, rot in ((50, True, False, 128), (50, True, True, 96), (50, False, False, 0),
                                (1, True, False, 64)):
        s = tn.make(T, 32, 8, 128, rot, 17 + rot, fp8=fp8)
        slots = torch.randperm(small * 16, generator=torch.Generator().manual_seed(T))[:T]
        pos, cs = (s["pos"].cuda(), s["cs"].cuda()) if rot else (None, None)
        kw = {"q_weight": s["qw"].cuda() if norm else None,
              "k_weight": s["kw"].cuda() if norm else None, "interleaved": inter}
        few = [torch.zeros(small, 8, 16, 128, dtype=dtype, device="cuda") for _ in "kv"]
        outs = []
        for caches, first in ((few, 0), (big, blocks - small)):
            for c in caches:
                c[first:first + small].zero_()
            args = (s["q"], s["k"], s["v"], pos, cs, (slots + first * 16).cuda(), *caches)
            outs.append(binding.norm_rope_write_kv_fp8(*args, 0.5, 0.25, **kw) if fp8 else
                        binding.norm_rope_write_kv(*args, **kw))
        assert torch.equal(outs[0], outs[1])
        for a, b in zip(few, big):
            assert a.view(torch.uint8).any()
            assert torch.equal(a.view(torch.uint8), b[blocks - small:].view(torch.uint8))
    assert binding.get_device_error(True)[0] == 0
    del big
    torch.cuda.empty_cache()
