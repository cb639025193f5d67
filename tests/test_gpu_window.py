"""pa_attention_window against the 64-bit definition.

Tolerance of one output element o = sum_i p_i v_i: the output's rounding,
2^-8 |o|; the rounding of the weights the products take, at most 2^-8 p_i each
for bf16 weights and 2^-7 for the two E4M3 terms of the tensor-core kernels
(2^-8 for the second term's rounding, as much again for the products of the
split queries), so 2^-7 sum_i p_i |v_i| covers both; and E4M3's smallest step,
2^-10 of 256 p against a reference up to 2^4 above the maximum: 2^-12 of the
largest |v|."""
from __future__ import annotations

import pytest
import torch

from tests import bounded_ref as ref

pytestmark = pytest.mark.gpu


def hide(b, window, sinks):
    """Everything a windowed call must not read or must not let through: the
    table entries of blocks no token attends to, and the slots of keys that no
    token of the request attends to."""
    bad = [-1, 10 ** 9, -(10 ** 9)]
    for r, (c, n) in enumerate(b.spans):
        L = c + n
        if n == 0:
            b.tables[r] = 10 ** 9
            continue
        see = ref.visible(c, n, window, sinks).any(0)
        p = torch.arange(L)[~see]
        slot = b.tables[r].long()[p // 16]
        for x in (b.k, b.v):
            x[slot, :, p % 16] = 0x7f if b.fp8 else float("nan")
        for i in range((L + 15) // 16):
            if not see[16 * i:16 * i + 16].any():
                b.tables[r, i] = bad[i % 3]


def run(b, window, sinks, **kw):
    from paged_kv_cache_42_gb300 import binding
    g = b.gpu()
    out = torch.full_like(g["q"], 7.0)
    args = (g["q"], g["k"], g["v"], g["tables"], g["seq_lens"], g["qsl"], b.scale)
    kw = {"window": window, "sinks": sinks, "max_query_len": b.max_q, "max_seq_len": b.max_len,
          "out": out, **kw}
    got = binding.attention_window_fp8(*args, b.k_scale, b.v_scale, **kw) if b.fp8 else \
        binding.attention_window(*args, **kw)
    torch.cuda.synchronize()
    return got.cpu()


def want_and_tol(b, window, sinks):
    tables = b.tables.clamp(0, len(b.k) - 1)  # entries that are not read point anywhere
    args = (b.q, b.k, b.v, tables, b.seq_lens, b.qsl, b.scale, window, sinks)
    want = ref.window_attention(*args, b.k_scale, b.v_scale)
    v = ref.values(b.v, b.v_scale)
    size = ref.window_attention(b.q, b.k, v.abs(), *args[3:], b.k_scale)
    top = v.nan_to_num().abs().max()
    return want, want.abs() * 2.0 ** -8 + size * 2.0 ** -7 + top * 2.0 ** -12


def check(b, window, sinks):
    from paged_kv_cache_42_gb300 import binding
    binding.get_device_error(True)
    hide(b, window, sinks)
    want, tol = want_and_tol(b, window, sinks)
    got = run(b, window, sinks)
    assert binding.get_device_error(True)[0] == 0
    n = int(b.qsl[-1])
    assert torch.isfinite(got[:n].float()).all()
    err = (got.double() - want).abs()[:n]
    assert (err <= tol[:n]).all(), (float(err.max()), float((err / tol[:n]).max()))
    assert (got[n:] == 7).all()


LENS = [1, 2, 15, 16, 17, 33, 63, 64, 65, 200, 257, 1000]
SHAPES = [(1, 1, 64), (4, 2, 64), (8, 2, 64), (8, 1, 64), (2, 2, 128), (4, 2, 128), (8, 2, 128),
          (16, 2, 128), (8, 8, 128), (32, 8, 128), (64, 8, 128)]


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (15, 0), (16, 4), (17, 16), (50, 17),
                                          (64, 100), (333, 40)])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("hq,hkv,d", SHAPES)
def test_decodes(pa_lib, hq, hkv, d, fp8, window, sinks):
    b = ref.Batch([(L - 1, 1) for L in LENS] + [(30, 0)], hq, hkv, d, window + d, fp8=fp8,
                  pad_blocks=2)
    check(b, window, sinks)


@pytest.mark.parametrize("window,sinks", [(1, 0), (5, 3), (16, 16), (100, 4), (129, 0), (200, 130)])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("hq,hkv,d", [(2, 2, 64), (16, 2, 64), (4, 2, 128), (8, 2, 128),
                                      (16, 2, 128), (32, 8, 128)])
def test_mixed_batches(pa_lib, hq, hkv, d, fp8, window, sinks):
    """Decodes, short spans, chunks from one row tile to several, and rows
    behind the last span."""
    spans = [(99, 1), (0, 1), (700, 1), (40, 5), (0, 16), (300, 15), (513, 33), (0, 130),
             (129, 300), (20, 0), (1000, 64)]
    b = ref.Batch(spans, hq, hkv, d, 7 * window + d, fp8=fp8, trailing_tokens=4)
    check(b, window, sinks)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 64), (32, 8, 128), (64, 8, 128)])
def test_long_sequences(pa_lib, hq, hkv, d, fp8):
    """Windows and sinks of many tiles, split over many workers."""
    b = ref.Batch([(9000, 1), (20000, 1), (5000, 1)], hq, hkv, d, d, fp8=fp8)
    check(b, 3001, 70)


@pytest.mark.parametrize("hq,n,L,window", [(8, 220, 400, 250), (32, 220, 400, 250),
                                           (64, 220, 400, 250), (32, 300, 900, 700),
                                           (32, 3, 30000, 20000)])
def test_token_major_tiles(pa_lib, hq, n, L, window):
    """E4M3 over eight KV heads with enough blocks for the token-major kernel:
    one and two CTAs per SM, and few tokens over many workers."""
    check(ref.Batch([(L + 3 * i, 1) for i in range(n)], hq, 8, 128, hq + n, fp8=True), window, 5)


def test_wide_chunk_overlaps_decodes(pa_lib):
    """A batch on the overlapped path: many decodes beside a long chunk."""
    b = ref.Batch([(900 + 7 * i, 1) for i in range(96)] + [(1000, 300)], 16, 4, 128, 3)
    check(b, 500, 4)


@pytest.mark.parametrize("fp8", [False, True])
def test_window_of_everything_is_attention(pa_lib, fp8):
    from paged_kv_cache_42_gb300 import binding
    b = ref.Batch([(99, 1), (700, 1), (40, 5), (129, 300)], 32, 8, 128, 4, fp8=fp8)
    g = b.gpu()
    args = (g["q"], g["k"], g["v"], g["tables"], g["seq_lens"], g["qsl"], b.scale)
    kw = {"max_query_len": b.max_q, "max_seq_len": b.max_len}
    whole = binding.attention_fp8(*args, b.k_scale, b.v_scale, **kw) if fp8 else \
        binding.attention(*args, **kw)
    for window, sinks in ((b.max_len, 0), (2 ** 31 - 1, 2 ** 31 - 1)):
        assert torch.equal(run(b, window, sinks), whole.cpu())
    # sinks that reach every window hide nothing either
    want, tol = want_and_tol(b, 10, 2 ** 31 - 1)
    got = run(b, 10, 2 ** 31 - 1)
    assert ((got.double() - want).abs() <= tol).all()


def test_repeatable_planned_and_self_planned(pa_lib):
    from paged_kv_cache_42_gb300 import binding
    for fp8 in (False, True):
        b = ref.Batch([(999, 1), (12, 1), (3000, 1)], 32, 8, 128, 5, fp8=fp8)
        one = run(b, 700, 4)
        assert torch.equal(one, run(b, 700, 4))
        binding.set_option("decode_self_plan", 0)
        try:
            assert torch.equal(one, run(b, 700, 4))
        finally:
            binding.set_option("decode_self_plan", 1)


def test_both_split_kernels_and_worker_counts(pa_lib):
    from paged_kv_cache_42_gb300 import binding
    for fp8 in (False, True):
        b = ref.Batch([(4000, 1), (77, 1)], 8, 2, 128, 6, fp8=fp8)
        want, tol = want_and_tol(b, 2000, 33)
        for tc in (0, 2):
            for workers in (1, 3, 0):
                binding.set_option("decode_tc", tc)
                binding.set_option("decode_max_workers", workers)
                try:
                    got = run(b, 2000, 33)
                finally:
                    binding.set_option("decode_tc", 1)
                    binding.set_option("decode_max_workers", 0)
                assert ((got.double() - want).abs() <= tol).all()


def test_bad_blocks_inside_the_window_are_reported(pa_lib):
    from paged_kv_cache_42_gb300 import binding
    binding.get_device_error(True)
    b = ref.Batch([(300, 1), (100, 40)], 8, 2, 128, 7)
    b.tables[0, 17] = len(b.k)
    run(b, 50, 4)
    assert binding.get_device_error(True)[0] == 2


def test_refused(pa_lib):
    from paged_kv_cache_42_gb300 import binding
    b = ref.Batch([(30, 1)], 4, 2, 64, 8)
    for window, sinks in ((0, 0), (-1, 0), (4, -1)):
        with pytest.raises(binding.PagedAttentionError):
            run(b, window, sinks)
    with pytest.raises(ValueError):
        run(b, 4, 0, out=torch.empty(2, 4, 64, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(TypeError):
        b.k = b.k.float()
        run(b, 4, 0)
