"""pa_attention_shared on the GPU: groups of requests with a prefix each, against plain
attention in 64 bits, over every cache format."""
from __future__ import annotations

import pytest
import torch

from tests import shared_ref as sr

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def sharing_whatever_it_saves(pa_lib):
    """These batches are small: by default they would attend without sharing."""
    from paged_kv_cache_42_gb300 import binding
    binding.set_option("shared_min_kb", 0)
    yield
    binding.set_option("shared_min_kb", 24576)

SHAPES = [(4, 2, 64), (16, 2, 64), (1, 1, 64), (2, 2, 128), (8, 4, 128), (32, 8, 128), (64, 8, 128),
          (8, 1, 128)]
LAYOUTS = {
    "one group": dict(groups=[(128, [(5, 1), (60, 1), (0, 1), (16, 1)])]),
    "two pairs": dict(groups=[(32, [(3, 1), (20, 1)]), (48, [(1, 1), (31, 1)])]),
    # no prefix; one request; no request; one block; a ragged key tile; several tiles
    "uneven": dict(groups=[(0, [(7, 1), (90, 1)]), (64, [(9, 1)]), (80, []), (16, [(0, 1), (2, 1), (40, 1)]),
                           (144, [(100, 1), (11, 1)]), (1040, [(33, 1), (0, 1), (300, 1)])],
                   before=[(50, 1), (0, 1)], after=[(129, 1)]),
    # spans of several tokens, none, prompt chunks, contexts that end inside the prefix
    "spans": dict(groups=[(112, [(4, 3), (0, 15), (9, 0), (30, 1), (0, 16), (64, 40)]),
                          (256, [(-1, 1), (-200, 2), (3, 1), (50, 2), (-130, 20)])],
                  before=[(20, 33)], after=[(77, 2)]),
    # left alone: one sharing token beside requests that do not share
    "alone": dict(groups=[(64, [(-3, 1), (10, 1), (0, 0)]), (64, [(5, 2)])]),
    # more tokens than a pair of tiles holds
    "many": dict(groups=[(160, [(i % 37, 1) for i in range(140)]), (32, [(i % 5, 1) for i in range(70)])]),
    "long": dict(groups=[(5008, [(100, 1), (0, 1), (700, 1)]), (2960, [(40, 1), (41, 2)])]),
}


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "rows"])
@pytest.mark.parametrize("name", list(LAYOUTS))
@pytest.mark.parametrize("hq,hkv,d", SHAPES)
def test_against_the_definition(pa_lib, name, hq, hkv, d, fmt):
    from paged_kv_cache_42_gb300 import binding
    if name == "long" and hkv == 8 and hq == 64 and fmt != "rows":
        pytest.skip("the reference of the largest shape, once")
    binding.get_device_error(True)
    b = sr.Batch(hq=hq, hkv=hkv, d=d, seed=3, fmt=fmt, trailing_tokens=3, **LAYOUTS[name])
    g = b.gpu()
    want, tol = b.want()
    out = torch.full(b.q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    b.run(g, out=out)
    got = out.cpu().double()
    mine = ~torch.isnan(want)
    err = ((got - want).abs() / tol)[mine]
    assert (err <= 1).all(), (float(err.max()), (err > 1).float().mean())
    assert (got[~mine] == 7).all()
    assert binding.get_device_error(True)[0] == 0
    again = torch.full_like(out, 7.0)
    b.run(g, out=again, workspace=torch.randint(
        0, 256, (binding.shared_workspace_size(len(b.spans), len(b.q), hq, hkv, d, len(b.groups),
                                               b.max_prefix),), dtype=torch.uint8, device="cuda"))
    assert torch.equal(again, out)
