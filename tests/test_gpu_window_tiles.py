"""Which tiles a windowed call over an E4M3 cache takes: the work of its decodes
decides, not prompt chunks (they run elsewhere) nor sinks past the sequences.
The two groupings are not bit-identical, so a batch below the limits gives the
same bits with the token-major tiles forbidden, and one above does not."""
from __future__ import annotations

import pytest
import torch

from tests import bounded_ref as ref
from tests import test_gpu_window as tw

pytestmark = pytest.mark.gpu


def both(b, window, sinks):
    from paged_kv_cache_42_gb300 import binding
    a = tw.run(b, window, sinks)
    binding.set_option("decode_token_major", 0)
    try:
        return a, tw.run(b, window, sinks)
    finally:
        binding.set_option("decode_token_major", 1)


@pytest.mark.parametrize("hq", [32, 64])
@pytest.mark.parametrize("spans,window,sinks", [
    ([(700 + i, 1) for i in range(8)] + [(200, 512)], 300, 4),      # one long chunk
    ([(1100, 300)] * 3 + [(900, 1)] * 3, 1000, 0),                  # more chunk than decode
    ([(600 + i, 1) for i in range(8)], 16, 2 ** 30),                # every key is a sink
    ([(600 + i, 1) for i in range(8)], 500, 2 ** 31 - 1)])
def test_little_work_takes_the_other_tiles(pa_lib, spans, window, sinks, hq):
    b = ref.Batch(spans, hq, 8, 128, 3, fp8=True)
    a, e = both(b, window, sinks)
    assert torch.equal(a, e)
    tw.check(b, window, min(sinks, 10 ** 6))


@pytest.mark.parametrize("hq", [32, 64])
def test_many_decodes_take_token_major_tiles(pa_lib, hq):
    b = ref.Batch([(400 + i, 1) for i in range(120)] + [(64, 40)], hq, 8, 128, 3, fp8=True)
    a, e = both(b, 200, 4)
    assert not torch.equal(a, e)
    tw.check(b, 200, 4)
