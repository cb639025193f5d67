"""pa_attention_weights against the 64-bit softmax.

Tolerance: a weight p = exp(s - lse) has the relative error of its exponent's
absolute one: s is a binary32 dot product of head_dim terms (|s| <= 40 in these
inputs, scaled in base 2: error <= 2^-23 x 64), the exponential 2^-21, lse and
the sum of up to rows terms 2^-20. 2^-16 of the key's total covers them."""
from __future__ import annotations

import pytest
import torch

from tests import bounded_ref as ref

pytestmark = pytest.mark.gpu
REL = 2.0 ** -16


def run(b, weights, out=None, **kw):
    from paged_kv_cache_42_gb300 import binding
    g = b.gpu()
    w = weights.cuda()
    o = None if out is None else out.cuda()
    args = (g["q"], g["k"], g["tables"], g["seq_lens"], g["qsl"], b.scale)
    kw = {"max_query_len": b.max_q, "max_seq_len": b.max_len, "out": o, **kw}
    got = binding.attention_weights_fp8(*args, b.k_scale, w, **kw) if b.fp8 else \
        binding.attention_weights(*args, w, **kw)
    torch.cuda.synchronize()
    return got


def check(b, seed=0, width=None, in_place=False):
    from paged_kv_cache_42_gb300 import binding
    binding.get_device_error(True)
    R, width = len(b.spans), width or b.mb * 16 + 3
    gen = torch.Generator().manual_seed(seed)
    w = torch.rand(R, b.hkv, width, generator=gen) * 3
    out = w.clone() if in_place else torch.full_like(w, -7.0)
    want = ref.attention_weights(b.q, b.k, b.tables, b.seq_lens, b.qsl, b.scale, w, out, b.k_scale)
    got = run(b, w, None if in_place else out).cpu()
    assert binding.get_device_error(True)[0] == 0
    err = (got.double() - want).abs()
    assert (err <= REL * want.abs()).all(), float((err / want.abs().clamp(min=1e-30)).max())
    for r, (c, n) in enumerate(b.spans):  # untouched entries, bit for bit
        a = 0 if n == 0 else c + n
        assert torch.equal(got[r, :, a:], out[r, :, a:])


EDGES = [0, 1, 14, 15, 16, 31, 200, 254, 255, 256, 1030]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (4, 2), (8, 2), (16, 2), (3, 3)])
def test_decodes(pa_lib, hq, hkv, d, fp8):
    b = ref.Batch([(c, 1) for c in EDGES] + [(40, 0)], hq, hkv, d, hq + d, fp8=fp8, pad_blocks=1,
                  q_scale=2.0)
    check(b)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("hq,hkv,d", [(2, 2, 64), (4, 2, 128), (8, 2, 128), (16, 2, 64)])
def test_spans_and_chunks(pa_lib, hq, hkv, d, fp8):
    """Every length from a verify span to a chunk of more than a row tile, beside
    decodes: both forms in one call, and tokens behind the last span."""
    spans = [(33, 1), (0, 2), (100, 3), (7, 8), (0, 9), (250, 16), (0, 1), (129, 33), (0, 128),
             (77, 129), (5, 0), (300, 300)]
    b = ref.Batch(spans, hq, hkv, d, hq * d, fp8=fp8, q_scale=2.0, trailing_tokens=5)
    b.q[-5:] = float("nan")  # rows of no request
    check(b)


@pytest.mark.parametrize("fp8", [False, True])
def test_long_context_parts(pa_lib, fp8):
    """More than 16 key tiles: the row statistics are joined from parts."""
    b = ref.Batch([(4000, 20), (2047, 2), (2000, 100), (6000, 1)], 8, 2, 128, 5, fp8=fp8)
    check(b)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("hq,hkv,d,spans", [
    (8, 1, 64, [(0, 700)]), (4, 4, 128, [(1500, 600)]), (16, 2, 128, [(3000, 260), (0, 30)]),
    (64, 8, 64, [(100, 1000), (700, 333)]), (1, 1, 128, [(0, 3001)])])
def test_pairs_in_parts(pa_lib, hq, hkv, d, spans, fp8):
    """Few pairs over many tiles: both passes cut them into parts, joined by the
    warp that finishes last; repeated, since which one that is may change."""
    b = ref.Batch(spans, hq, hkv, d, hq + d, fp8=fp8)
    check(b)
    w = torch.rand(len(spans), hkv, b.mb * 16)
    one = run(b, w, torch.zeros_like(w))
    for _ in range(5):
        assert torch.equal(one, run(b, w, torch.zeros_like(w)))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("hq,spans", [(8, [(41500, 1), (300, 1)]), (1, [(50000, 2), (9, 8)]),
                                      (4, [(41000, 2), (700, 70)])])
def test_longer_than_a_cluster_holds(pa_lib, hq, spans, fp8):
    """Scores that outgrow eight CTAs' shared memory go through global memory."""
    check(ref.Batch(spans, hq, 1, 64, hq, fp8=fp8))


def test_in_place_and_sharp(pa_lib):
    """Accumulation in place; queries sharp enough to give one key nearly all."""
    b = ref.Batch([(500, 1), (90, 40), (1, 1)], 8, 2, 128, 6, q_scale=6.0)
    check(b, in_place=True)


def test_no_new_token_and_first_token(pa_lib):
    b = ref.Batch([(0, 1), (64, 0)], 4, 4, 64, 7)
    check(b)
    b = ref.Batch([(64, 0), (3, 0)], 4, 4, 64, 7)
    b.q = torch.zeros(1, 4, 64).bfloat16()  # one padded row, no span
    b.max_q = 1
    check(b)


def test_negative_and_zero_scale(pa_lib):
    for scale in (-0.1, 0.0):
        b = ref.Batch([(90, 1), (40, 50)], 8, 2, 64, 8)
        b.scale = scale
        check(b)


def test_repeatable_and_permuted_blocks(pa_lib):
    b = ref.Batch([(900, 1), (300, 200)], 8, 2, 128, 9)
    w = torch.rand(2, 2, b.mb * 16)
    one = run(b, w, torch.zeros_like(w))
    assert torch.equal(one, run(b, w, torch.zeros_like(w)))
    perm = torch.randperm(len(b.k), generator=torch.Generator().manual_seed(1))
    k2 = torch.empty_like(b.k)
    k2[perm] = b.k
    b.k = k2
    b.tables = torch.where(b.tables >= 0, perm[b.tables.clamp(min=0).long()].int(), -1)
    assert torch.equal(one, run(b, w, torch.zeros_like(w)))


def test_errors_are_reported(pa_lib):
    from paged_kv_cache_42_gb300 import binding
    binding.get_device_error(True)
    b = ref.Batch([(100, 1), (50, 30), (60, 1)], 4, 2, 64, 10)
    w = torch.rand(3, 2, b.mb * 16)
    keep = b.tables.clone()
    for r in (0, 1):
        b.tables[r, 0] = len(b.k)
        run(b, w.clone())
        assert binding.get_device_error(True)[0] == 2
        b.tables = keep.clone()
    got = run(b, w[:, :, :90].contiguous(), torch.full((3, 2, 90), -7.0)).cpu()  # 101 keys, 90 wide
    assert binding.get_device_error(True) == (3, 0)
    assert (got[0] == -7).all() and (got[1, :, :80] != -7).all()
    run(b, w.clone(), max_query_len=8)
    assert binding.get_device_error(True) == (3, 1)
    # spans that overlap more often than the batch has tokens: refused on the device
    b2 = ref.Batch([(0, 40)], 4, 2, 64, 11)
    g = b2.gpu()
    n = 9
    qsl = torch.tensor([0, 40] * 5, dtype=torch.int32).cuda()
    wide = torch.zeros(n, 2, 48, device="cuda")
    binding.attention_weights(g["q"], g["k"], g["tables"].repeat(n, 1), g["seq_lens"].repeat(n),
                              qsl, b2.scale, wide, max_query_len=40, max_seq_len=40)
    assert binding.get_device_error(True)[0] == 4


def test_refused(pa_lib):
    from paged_kv_cache_42_gb300 import binding
    b = ref.Batch([(20, 1)], 4, 2, 64, 12)
    w = torch.rand(1, 2, 32)
    small = torch.empty(256, dtype=torch.uint8, device="cuda")
    with pytest.raises(binding.PagedAttentionError):
        run(b, w, workspace=small)
    with pytest.raises(ValueError):
        run(b, w[:, :1])
    with pytest.raises(TypeError):
        run(b, w.double())
    with pytest.raises(ValueError):
        run(b, w, torch.zeros(1, 2, 33))
    b.scale = float("nan")
    with pytest.raises(binding.PagedAttentionError):
        run(b, w)
