"""pa_evict_kv at the lengths where its select changes form: 4, 8, 16 or 32 keys
a thread or none kept, one CTA per head or a cluster of two or four, with
weights that tie across threads, warps and CTAs."""
from __future__ import annotations

import pytest
import torch

from tests import bounded_ref as ref
from tests import test_gpu_evict as te

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("ties", [2, 64, 2 ** 20])
@pytest.mark.parametrize("candidates", [2047, 2048, 2049, 4095, 4096, 4097, 8192, 8193])
def test_around_the_keys_of_a_thread(pa_lib, candidates, ties):
    keep, recent, sinks = 1000, 37, 5
    L = candidates + recent + sinks
    b = ref.Batch([(L, 0), (L - 1, 0), (keep + 1, 0), (keep, 0)], 2, 2, 64, candidates, fp8=True,
                  extra_blocks=4 * 63)
    g = torch.Generator().manual_seed(candidates + ties)
    w = torch.randint(0, ties, (4, 2, b.mb * 16), generator=g).float()
    te.check(b, w, keep, recent, sinks)


@pytest.mark.parametrize("L,hkv", [(10000, 4), (17000, 3), (33500, 4), (66000, 2)])
@pytest.mark.parametrize("ties", [3, 1000])
def test_ties_across_the_ctas_of_a_cluster(pa_lib, L, hkv, ties):
    b = ref.Batch([(L, 0), (L // 2 + 3, 0), (3001, 0)], hkv, hkv, 64, L, fp8=True,
                  extra_blocks=3 * 188)
    g = torch.Generator().manual_seed(L + ties)
    w = torch.randint(0, ties, (3, hkv, b.mb * 16), generator=g).float() - 1
    te.check(b, w, 3000, 800, 16)


def test_many_heads_of_middling_length(pa_lib):
    """512 rows of up to 4096 keys: one CTA each, eight keys a thread."""
    lens = [4096 - 50 * i for i in range(16)]
    b = ref.Batch([(x, 0) for x in lens], 8, 8, 64, 5, extra_blocks=16 * 32)
    w = torch.rand(16, 8, b.mb * 16, generator=torch.Generator().manual_seed(2))
    te.check(b, (w * 512).round() / 512, 500, 250, 4)
