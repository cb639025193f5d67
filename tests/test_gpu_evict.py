"""pa_evict_kv: which tokens stay, and that exactly their rows arrive."""
from __future__ import annotations

import math

import pytest
import torch

from tests import bounded_ref as ref

pytestmark = pytest.mark.gpu


def run(b, weights, keep, recent, sinks, new_width=None):
    from paged_kv_cache_42_gb300 import binding
    R, nnew = len(b.spans), (keep + 15) // 16
    g = b.gpu()
    new_tables = b.free[:R * nnew].view(R, nnew).contiguous()
    kept = torch.full((R, b.hkv, keep), -7, dtype=torch.int32, device="cuda")
    nw = torch.full((R, b.hkv, new_width or keep), -7.0, device="cuda")
    out = binding.evict_kv(g["k"], g["v"], g["tables"], g["seq_lens"], weights.cuda(),
                           new_tables.cuda(), keep=keep, recent=recent, sinks=sinks,
                           max_seq_len=b.max_len, kept=kept, new_weights=nw)
    torch.cuda.synchronize()
    return new_tables, [x.cpu() for x in out], g["k"].cpu(), g["v"].cpu()


def check(b, weights, keep, recent, sinks, new_width=None):
    from paged_kv_cache_42_gb300 import binding
    binding.get_device_error(True)
    tables, (lens, kept, nw), k, v = run(b, weights, keep, recent, sinks, new_width)
    assert binding.get_device_error(True)[0] == 0
    want_lens, want = ref.evict(weights, b.seq_lens, keep, recent, sinks)
    assert lens.tolist() == want_lens
    want_k, want_v = b.k.clone(), b.v.clone()
    n = torch.arange(keep)
    for r in range(len(b.spans)):
        for h in range(b.hkv):
            if (r, h) not in want:
                assert (kept[r, h] == -7).all() and (nw[r, h] == -7).all()
                continue
            ids = torch.tensor(want[r, h])
            assert torch.equal(kept[r, h].long(), ids), (r, h)
            assert torch.equal(nw[r, h, :keep].view(torch.int32),
                               weights[r, h, ids].contiguous().view(torch.int32))
            assert (nw[r, h, keep:] == -7).all()
            src, dst = b.tables[r].long()[ids // 16], tables[r].long()[n // 16]
            want_k[dst, h, n % 16] = b.k[src, h, ids % 16]
            want_v[dst, h, n % 16] = b.v[src, h, ids % 16]
    assert torch.equal(k.view(torch.uint8), want_k.view(torch.uint8))
    assert torch.equal(v.view(torch.uint8), want_v.view(torch.uint8))


@pytest.mark.parametrize("d,fp8", [(64, False), (128, False), (64, True), (128, True)])
@pytest.mark.parametrize("keep,recent,sinks", [(1, 0, 0), (1, 1, 0), (16, 4, 4), (17, 0, 1),
                                               (33, 33, 0), (100, 60, 4), (129, 0, 129)])
def test_lengths_and_layouts(pa_lib, d, fp8, keep, recent, sinks):
    lens = [keep - 1, keep, keep + 1, keep + 17, 3 * keep + 40, 515]
    b = ref.Batch([(max(0, x), 0) for x in lens], 2, 2, d, keep + d, fp8=fp8,
                  extra_blocks=6 * ((keep + 15) // 16), pad_blocks=2)
    w = torch.rand(6, 2, b.mb * 16, generator=torch.Generator().manual_seed(keep))
    check(b, w, keep, recent, sinks, new_width=keep + 5)


def test_ties_signs_and_nan(pa_lib):
    """Equal weights go to the lowest position, -0 equals 0, a NaN goes first."""
    b = ref.Batch([(700, 0)] * 6, 1, 1, 64, 3, extra_blocks=6 * 13)
    g = torch.Generator().manual_seed(4)
    w = torch.zeros(6, 1, b.mb * 16)
    w[1] = torch.randint(0, 3, (1, w.shape[2]), generator=g).float()
    w[2] = -torch.rand(1, w.shape[2], generator=g)
    w[3, :, ::2] = -0.0
    w[4] = torch.rand(1, w.shape[2], generator=g)
    w[4, :, 100:600] = math.nan
    w[5] = torch.rand(1, w.shape[2], generator=g) * 1e-41  # below the normal range
    w[5, :, 300:310] = math.inf
    check(b, w, 200, 13, 5)


@pytest.mark.parametrize("L", [40960 + 77, 70001])
def test_longer_than_shared_memory(pa_lib, L):
    b = ref.Batch([(L, 0), (5000, 0)], 1, 1, 64, 8, fp8=True, extra_blocks=2 * 260)
    w = torch.randn(2, 1, b.mb * 16, generator=torch.Generator().manual_seed(5)).exp()
    w = (w * 64).round() / 64
    check(b, w, 4097, 1000, 16)


def test_shared_source_blocks(pa_lib):
    """Two requests may keep the same prefix blocks: they are only read."""
    b = ref.Batch([(320, 0), (320, 0)], 4, 4, 128, 11, extra_blocks=2 * 7)
    b.tables[1, :20] = b.tables[0, :20]
    w = torch.rand(2, 4, b.mb * 16, generator=torch.Generator().manual_seed(6))
    check(b, w, 100, 20, 4)


def test_bad_lengths_and_blocks_are_reported(pa_lib):
    from paged_kv_cache_42_gb300 import binding
    binding.get_device_error(True)
    b = ref.Batch([(100, 0), (90, 0)], 2, 2, 64, 12, extra_blocks=4)
    w = torch.rand(2, 2, b.mb * 16, generator=torch.Generator().manual_seed(7))
    b.seq_lens[0] = b.mb * 16 + 1  # more than its table holds
    b.max_len = 10 ** 4
    _, (lens, kept, _), k, _ = run(b, w, 20, 4, 2)
    assert binding.get_device_error(True) == (3, 0)
    assert (kept[0] == -7).all() and lens[1] == 20 and (kept[1] != -7).all()
    b.seq_lens[0] = 100
    bad = b.tables[1, 0].item()
    b.tables[1, 0] = len(b.k)  # holds the first tokens of request 1
    run(b, w, 20, 4, 2)
    assert binding.get_device_error(True)[0] == 2
    b.tables[1, 0] = bad
    check(b, w, 20, 4, 2)


def test_refused(pa_lib):
    from paged_kv_cache_42_gb300 import binding
    b = ref.Batch([(100, 0)], 2, 2, 64, 13, extra_blocks=4)
    g = b.gpu()
    w = torch.rand(1, 2, b.mb * 16, device="cuda")
    nt = g["free"][:2].view(1, 2).contiguous()

    def call(**kw):
        a = dict(keep=20, recent=4, sinks=2, max_seq_len=100)
        pos = dict(k=g["k"], v=g["v"], t=g["tables"], s=g["seq_lens"], w=w, n=nt)
        for n in list(kw):
            (pos if n in pos else a)[n] = kw[n]
        return binding.evict_kv(pos["k"], pos["v"], pos["t"], pos["s"], pos["w"], pos["n"], **a)

    call()
    for kw, exc in (({"keep": 0}, binding.PagedAttentionError),
                    ({"recent": 19}, binding.PagedAttentionError),
                    ({"sinks": -1}, binding.PagedAttentionError),
                    ({"keep": 33}, binding.PagedAttentionError),  # three blocks, two given
                    ({"new_seq_lens": g["seq_lens"]}, binding.PagedAttentionError),
                    ({"w": w[0]}, ValueError), ({"w": w.double()}, TypeError),
                    ({"k": g["k"].float(), "v": g["v"].float()}, TypeError),
                    ({"kept": torch.empty(1, 2, 21, dtype=torch.int32, device="cuda")}, ValueError),
                    ({"new_weights": w[:, :, :19].contiguous()}, binding.PagedAttentionError)):
        with pytest.raises(exc):
            call(**kw)
    torch.cuda.synchronize()
