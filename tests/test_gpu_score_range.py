"""Attention whose scale is negative or zero, and scores far outside the usual
range, over decodes, short spans and prompt chunks.

Tolerances: for ordinary scores those of tests/test_gpu_window.py (the weights'
and the output's rounding). Where one key outweighs every other by more than
binary32 holds, its weight is 1 and the output is its V row, exactly."""
from __future__ import annotations

import pytest
import torch

from tests import bounded_ref as ref
from tests import test_gpu_window as tw

pytestmark = pytest.mark.gpu

SPANS = [(300, 1), (0, 1), (37, 5), (0, 300), (1000, 200), (130, 16), (15, 0)]


def attend(b, **kw):
    """pa_attention[_fp8] on a batch, on the CPU."""
    from paged_kv_cache_42_gb300 import binding
    g = b.gpu()
    args = (g["q"], g["k"], g["v"], g["tables"], g["seq_lens"], g["qsl"], b.scale)
    kw = {"max_query_len": b.max_q, "max_seq_len": b.max_len, **kw}
    got = binding.attention_fp8(*args, b.k_scale, b.v_scale, **kw) if b.fp8 else \
        binding.attention(*args, **kw)
    torch.cuda.synchronize()
    assert binding.get_device_error(True)[0] == 0
    return got.cpu()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("hq,hkv,d", [(4, 2, 64), (8, 2, 128), (16, 2, 128), (32, 8, 128), (8, 8, 64)])
@pytest.mark.parametrize("scale", [-0.1, 0.0])
@pytest.mark.parametrize("window,sinks", [(10 ** 6, 0), (40, 0), (200, 20)])
def test_scale_of_any_sign(pa_lib, scale, window, sinks, hq, hkv, d, fp8):
    b = ref.Batch(SPANS, hq, hkv, d, 7 + window % 97, fp8=fp8)
    b.scale = scale
    if window > b.max_len:
        want, tol = tw.want_and_tol(b, window, sinks)
        err = (attend(b).double() - want).abs()
        assert (err <= tol).all(), (float(err.max()), float((err / tol).max()))
    tw.check(b, window, sinks)


def test_cascade_with_a_negative_scale(pa_lib):
    from paged_kv_cache_42_gb300 import binding
    b = ref.Batch([(64 + 50 * r, 1 + r % 3) for r in range(8)], 16, 4, 128, 19)
    b.tables[:, :4] = b.tables[0, :4]
    b.scale = -0.1
    want, tol = tw.want_and_tol(b, 10 ** 6, 0)
    g = b.gpu()
    got = binding.attention_cascade(g["q"], g["k"], g["v"], g["tables"], g["seq_lens"], g["qsl"],
                                    b.scale, common_prefix_len=64, max_query_len=b.max_q,
                                    max_seq_len=b.max_len)
    err = (got.cpu().double() - want).abs()
    assert (err <= tol).all(), (float(err.max()), float((err / tol).max()))


def steep(b, rising):
    """Scores of -1e32 and less that differ by 1e29 and more from key to key,
    falling or rising with the position; one or two bits each, exact in bf16."""
    b.q.fill_(2.0 ** 50)
    for r, (c, n) in enumerate(b.spans):
        i = torch.arange(c + n)
        j = c + n - 1 - i if rising else i
        val = -(2.0 ** 50) * (1.0 + (j % 128) / 128.0) * 2.0 ** (j // 128)
        b.k[b.tables[r].long()[i // 16], :, i % 16] = val.bfloat16()[:, None, None]


@pytest.mark.parametrize("rising", [False, True])
@pytest.mark.parametrize("hq,hkv,d", [(4, 2, 64), (4, 2, 128), (8, 1, 128), (1, 1, 64)])
def test_chunks_with_scores_below_any_sentinel(pa_lib, hq, hkv, d, rising):
    """The rows of a chunk see windows of 30 keys, most of them in none of their
    work item's first key tiles."""
    b = ref.Batch([(0, 300), (4, 150), (700, 260), (90, 1)], hq, hkv, d, 3)
    steep(b, rising)
    full = attend(b)
    got = tw.run(b, 30, 0)
    for r, (c, n) in enumerate(b.spans):
        p = torch.arange(c, c + n)
        rows = slice(int(b.qsl[r]), int(b.qsl[r + 1]))
        for out, key in ((full, p * rising), (got, p if rising else (p - 29).clamp(min=0))):
            v = b.v[b.tables[r].long()[key // 16], :, key % 16]
            assert torch.equal(out[rows], v.repeat_interleave(hq // hkv, 1)), r


def add_weights(b, **kw):
    """One step's weights over zeros, in place: [R, Hkv, width] on the CPU."""
    from paged_kv_cache_42_gb300 import binding
    g = b.gpu()
    w = torch.zeros(len(b.spans), b.hkv, b.mb * 16, device="cuda")
    args = (g["q"], g["k"], g["tables"], g["seq_lens"], g["qsl"], b.scale)
    kw = {"max_query_len": b.max_q, "max_seq_len": b.max_len, **kw}
    got = binding.attention_weights_fp8(*args, b.k_scale, w, **kw) if b.fp8 else \
        binding.attention_weights(*args, w, **kw)
    torch.cuda.synchronize()
    assert binding.get_device_error(True)[0] == 0
    return got.cpu()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("hq,hkv,d,scale", [(4, 2, 64, -0.1), (8, 2, 128, 0.0), (16, 2, 128, -0.1),
                                            (16, 2, 64, 0.0), (4, 4, 128, 1.5)])
def test_weights_with_a_scale_of_any_sign_and_size(pa_lib, hq, hkv, d, scale, fp8):
    """The relative error of a weight is the absolute one of its exponent: with
    |score| up to 6 sqrt(d) x 1.5 x log2 e < 150, 2^-23 x 150 for the product and
    as much for the log-sum-exp, below 2^-14 with the exponentials'."""
    spans = [(300, 1), (37, 5), (0, 300), (1000, 200), (130, 16)]
    b = ref.Batch(spans, hq, hkv, d, 31, fp8=fp8)
    b.scale = scale
    zero = torch.zeros(len(spans), hkv, b.mb * 16)
    want = ref.attention_weights(b.q, b.k, b.tables, b.seq_lens, b.qsl, scale, zero, zero, b.k_scale)
    got = add_weights(b)
    tiny = 2.0 ** -120  # weights below binary32's range
    assert ((got.double() - want).abs() <= want * 2.0 ** -14 + tiny).all()


@pytest.mark.parametrize("where", ["key", "query"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("hq,hkv,d,c,n", [(4, 2, 64, 100, 1), (8, 2, 128, 100, 2), (8, 2, 128, 100, 300),
                                          (4, 1, 64, 5, 140), (8, 1, 128, 3000, 200)])
def test_a_bad_row_spoils_the_keys_it_sees(pa_lib, hq, hkv, d, c, n, value, where):
    """A NaN or an infinity in a new token's query spoils the weights of all keys
    the token sees; one in a key those of every key that a row seeing it sees.
    Other KV heads, and keys seen by good rows only, keep theirs."""
    b = ref.Batch([(c, n), (50, min(n, 40))], hq, hkv, d, 9)
    b.q[..., 3] = b.q[..., 3].abs() + 0.5  # an infinite key scores plus infinity
    clean = add_weights(b)
    at = c + n // 2  # position of the token, and of the key
    if where == "query":
        b.q[n // 2, 0, 3] = value  # a query head of KV head 0
    else:
        b.k[b.tables[0, at // 16], 0, at % 16, 3] = value
    got = add_weights(b)
    last = at if where == "query" else c + n - 1  # keys up to here are seen by a bad row
    assert torch.isnan(got[0, 0, :last + 1]).all()
    want = clean.clone()
    want[0, 0, :last + 1] = got[0, 0, :last + 1]
    assert torch.equal(got.view(torch.int32), want.view(torch.int32))
