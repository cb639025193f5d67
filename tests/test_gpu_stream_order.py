"""Attention reads what the work enqueued before it on its stream has written:
queries, lengths, tables and cache rows made by other kernels right before the
call, by pa_norm_rope_write_kv and by pa_evict_kv. Nothing waits on the host
between the calls; results are those of a run that does, bit for bit."""
from __future__ import annotations

import pytest
import torch

from tests import bounded_ref as ref

pytestmark = pytest.mark.gpu

CASES = {  # spans, hq, hkv, d, fp8: one per split-KV kernel, and a planned batch
    "cuda-core": ([(400 + 9 * i, 1) for i in range(24)], 8, 8, 64, False),
    "tensor-core": ([(900 + 13 * i, 1) for i in range(24)], 32, 8, 128, False),
    "tensor-core e4m3": ([(900 + 13 * i, 1) for i in range(24)], 16, 4, 128, True),
    "token-major e4m3": ([(900 + 13 * i, 1) for i in range(24)], 32, 8, 128, True),
    "mixed": ([(900 + 13 * i, 1) for i in range(20)] + [(40, 200), (7, 3)], 32, 8, 128, False),
    "mixed e4m3": ([(900 + 13 * i, 1) for i in range(20)] + [(40, 200), (7, 3)], 32, 8, 128, True),
}


def attention(b, q, k, v, tables, lens, qsl, out, ws, prefix=0, max_len=None):
    from paged_kv_cache_42_gb300 import binding
    kw = {"max_query_len": b.max_q, "max_seq_len": max_len or b.max_len, "out": out, "workspace": ws}
    args = (q, k, v, tables, lens, qsl, b.scale)
    if prefix:
        return binding.attention_cascade(*args, common_prefix_len=prefix, **kw)
    return binding.attention_fp8(*args, b.k_scale, b.v_scale, **kw) if b.fp8 else \
        binding.attention(*args, **kw)


def rounds(step, n, reps=4):
    """The results of n different rounds, synchronised, then the same back to
    back, eager and in one captured graph."""
    want = []
    for i in range(n):
        want.append([t.clone() for t in step(i)])
        torch.cuda.synchronize()
    for _ in range(reps):
        got = [[t.clone() for t in step(i)] for i in range(n)]
        torch.cuda.synchronize()
        for a, e in zip(got, want):
            for x, y in zip(a, e):
                assert torch.equal(x, y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [[t.clone() for t in step(i)] for i in range(n)]
    for _ in range(reps):
        graph.replay()
        torch.cuda.synchronize()
        for a, e in zip(got, want):
            for x, y in zip(a, e):
                assert torch.equal(x, y)


@pytest.mark.parametrize("name,prefix", [(n, 0) for n in CASES] + [("cuda-core", 64),
                                                                   ("tensor-core", 64)])
def test_inputs_made_right_before(pa_lib, name, prefix):
    from paged_kv_cache_42_gb300 import binding
    spans, hq, hkv, d, fp8 = CASES[name]
    binding.get_device_error(True)
    b = ref.Batch(spans, hq, hkv, d, 5, fp8=fp8)
    if prefix:
        b.tables[:, :prefix // 16] = b.tables[0, :prefix // 16]
    g = b.gpu()
    gen = torch.Generator().manual_seed(1)
    qs = torch.randn((3,) + tuple(b.q.shape), generator=gen).bfloat16().cuda()
    lens = [g["seq_lens"] - 16 * i for i in range(3)]  # contexts stay within the tables
    lens = [torch.where(g["seq_lens"] > 500, x, g["seq_lens"]).int() for x in lens]
    rolled = [torch.roll(g["k"], i, 1) for i in range(3)]
    q, k, sl, tb = (torch.empty_like(x) for x in (g["q"], g["k"], g["seq_lens"], g["tables"]))
    out = torch.empty_like(q)
    ws = torch.empty(binding.cascade_workspace_size(len(spans), len(q), hq, hkv, d),
                     dtype=torch.uint8, device="cuda")

    def step(i):
        sl.copy_(lens[i])
        tb.copy_(g["tables"])
        k.copy_(rolled[i])
        q.copy_(qs[i])
        return [attention(b, q, k, g["v"], tb, sl, g["qsl"], out, ws, prefix)]
    rounds(step, 3)
    assert binding.get_device_error(True)[0] == 0


@pytest.mark.parametrize("name", ["cuda-core", "tensor-core", "tensor-core e4m3", "token-major e4m3"])
def test_behind_norm_rope_and_evict(pa_lib, name):
    """Write, attention, weights, eviction, and attention over what is left."""
    from paged_kv_cache_42_gb300 import binding
    spans, hq, hkv, d, fp8 = CASES[name]
    binding.get_device_error(True)
    R, keep = len(spans), 200
    nnew = (keep + 15) // 16
    b = ref.Batch(spans, hq, hkv, d, 6, fp8=fp8, extra_blocks=R * nnew)
    g = b.gpu()
    slots = torch.tensor([int(b.tables[r, c // 16]) * 16 + c % 16 for r, (c, _) in enumerate(spans)],
                         device="cuda")
    gen = torch.Generator().manual_seed(3)
    xs = torch.randn(3, R, (hq + 2 * hkv) * d, generator=gen).bfloat16().cuda()
    nt = g["free"].view(R, nnew).contiguous()
    qo = torch.empty(R, hq, d, dtype=torch.bfloat16, device="cuda")
    out, out2 = torch.empty_like(qo), torch.empty_like(qo)
    w = torch.zeros(R, hkv, b.mb * 16, device="cuda")
    new_lens = torch.empty(R, dtype=torch.int32, device="cuda")
    kept = torch.empty(R, hkv, keep, dtype=torch.int32, device="cuda")
    nw = torch.empty(R, hkv, keep, device="cuda")
    ws = torch.empty(binding.workspace_size(R, R, hq, hkv, d), dtype=torch.uint8, device="cuda")
    ws2 = torch.empty(binding.weights_workspace_size(R, R, hq, hkv, d, 1, b.max_len),
                      dtype=torch.uint8, device="cuda")

    def step(i):
        q, k, v = (xs[i][:, a * d:e * d].unflatten(1, (-1, d))
                   for a, e in ((0, hq), (hq, hq + hkv), (hq + hkv, hq + 2 * hkv)))
        args = (q, k, v, None, None, slots, g["k"], g["v"])
        if fp8:
            binding.norm_rope_write_kv_fp8(*args, b.k_scale, b.v_scale, out=qo)
        else:
            binding.norm_rope_write_kv(*args, out=qo)
        attention(b, qo, g["k"], g["v"], g["tables"], g["seq_lens"], g["qsl"], out, ws)
        w.zero_()
        wa = (qo, g["k"], g["tables"], g["seq_lens"], g["qsl"], b.scale)
        kw = {"max_query_len": 1, "max_seq_len": b.max_len, "workspace": ws2}
        if fp8:
            binding.attention_weights_fp8(*wa, b.k_scale, w, **kw)
        else:
            binding.attention_weights(*wa, w, **kw)
        binding.evict_kv(g["k"], g["v"], g["tables"], g["seq_lens"], w, nt, keep=keep, recent=50,
                         sinks=4, max_seq_len=b.max_len, new_seq_lens=new_lens, kept=kept,
                         new_weights=nw)
        attention(b, qo, g["k"], g["v"], nt, new_lens, g["qsl"], out2, ws, max_len=keep)
        return [out, w, new_lens, kept, nw, out2]
    rounds(step, 3)
    assert binding.get_device_error(True)[0] == 0


@pytest.mark.parametrize("name", CASES)
def test_write_overlap_gives_the_same_bits(pa_lib, name):
    """pa_write_kv and attention directly behind it, with the option and without."""
    from paged_kv_cache_42_gb300 import binding
    spans, hq, hkv, d, fp8 = CASES[name]
    b = ref.Batch(spans, hq, hkv, d, 8, fp8=fp8)
    g = b.gpu()
    T = len(b.q)
    slots = torch.tensor([int(b.tables[r, p // 16]) * 16 + p % 16 for r, (c, n) in enumerate(spans)
                          for p in range(c, c + n)], device="cuda")
    gen = torch.Generator().manual_seed(4)
    kv = torch.randn(3, 2, T, hkv, d, generator=gen).bfloat16().cuda()
    out = torch.empty_like(g["q"])
    ws = torch.empty(binding.workspace_size(len(spans), T, hq, hkv, d), dtype=torch.uint8,
                     device="cuda")

    def step(i):
        if fp8:
            binding.write_kv_fp8(kv[i, 0], kv[i, 1], slots, g["k"], g["v"], b.k_scale, b.v_scale)
        else:
            binding.write_kv(kv[i, 0], kv[i, 1], slots, g["k"], g["v"])
        return attention(b, g["q"], g["k"], g["v"], g["tables"], g["seq_lens"], g["qsl"], out, ws)
    want = [step(i).clone() for i in range(3)]
    torch.cuda.synchronize()
    binding.set_option("write_overlap", 1)
    try:
        for _ in range(5):
            for i in range(3):
                assert torch.equal(step(i), want[i])
        torch.cuda.synchronize()
    finally:
        binding.set_option("write_overlap", 0)
