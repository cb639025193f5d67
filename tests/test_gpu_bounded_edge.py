"""What a user may do with the bounded-cache operators besides one plain call:
caches past 32-bit offsets, two streams at once, captured and replayed steps,
the attention of the next step right behind them."""
from __future__ import annotations

import pytest
import torch

from tests import bounded_ref as ref

pytestmark = pytest.mark.gpu


def spread(b, blocks):
    """The batch's blocks moved to the top of a pool of `blocks`: (k, v, tables,
    free ids) on the GPU, the rest of the pool uninitialised."""
    n = len(b.k)
    k = torch.empty((blocks,) + b.k.shape[1:], dtype=b.k.dtype, device="cuda")
    v = torch.empty_like(k)
    k[blocks - n:] = b.k.cuda()
    v[blocks - n:] = b.v.cuda()
    return k, v, torch.where(b.tables >= 0, b.tables + (blocks - n), -1).cuda(), b.free + (blocks - n)


@pytest.mark.parametrize("fp8", [False, True])
def test_offsets_past_32_bits(pa_lib, fp8):
    """300000 blocks of 8 heads x 16 x 128: 4.9e9 elements a cache."""
    from paged_kv_cache_42_gb300 import binding
    binding.get_device_error(True)
    b = ref.Batch([(300, 1), (40, 20), (0, 1)], 32, 8, 128, 3, fp8=fp8, extra_blocks=9)
    blocks = 300000
    k, v, tables, free = spread(b, blocks)
    q, sl, qsl = b.q.cuda(), b.seq_lens.cuda(), b.qsl.cuda()
    kw = {"max_query_len": b.max_q, "max_seq_len": b.max_len}
    args = (q, k, v, tables, sl, qsl, b.scale)
    got = (binding.attention_window_fp8(*args, b.k_scale, b.v_scale, window=50, sinks=4, **kw) if fp8
           else binding.attention_window(*args, window=50, sinks=4, **kw))
    want = ref.window_attention(b.q, b.k, b.v, b.tables, b.seq_lens, b.qsl, b.scale, 50, 4,
                                b.k_scale, b.v_scale)
    assert (got.cpu().double() - want).abs().max() < 2e-2
    w = torch.rand(3, 8, b.mb * 16)
    out = torch.zeros_like(w).cuda()
    args = (q, k, tables, sl, qsl, b.scale)
    (binding.attention_weights_fp8(*args, b.k_scale, w.cuda(), out=out, **kw) if fp8 else
     binding.attention_weights(*args, w.cuda(), out=out, **kw))
    want = ref.attention_weights(b.q, b.k, b.tables, b.seq_lens, b.qsl, b.scale, w,
                                 torch.zeros_like(w), b.k_scale)
    assert ((out.cpu().double() - want).abs() <= want * 2.0 ** -16).all()
    new_tables = free[:9].view(3, 3).contiguous().cuda()
    lens, kept, _ = binding.evict_kv(k, v, tables, sl, w.cuda(), new_tables, keep=40, recent=8,
                                     sinks=2, max_seq_len=b.max_len)
    want_lens, want = ref.evict(w, b.seq_lens, 40, 8, 2)
    assert lens.tolist() == want_lens
    n = torch.arange(40)
    for (r, h), ids in want.items():
        assert kept[r, h].tolist() == ids
        ids = torch.tensor(ids)
        src, dst = b.tables[r].long()[ids // 16], new_tables.cpu()[r].long()[n // 16]
        assert torch.equal(k[dst.cuda(), h, (n % 16).cuda()].cpu().view(torch.uint8),
                           b.k[src, h, ids % 16].view(torch.uint8))
    slots = (torch.arange(3) + (blocks * 16 - 3)).cuda()
    x = torch.randn(3, 8, 128).bfloat16().cuda()
    if fp8:
        binding.norm_rope_write_kv_fp8(x, x, x, None, None, slots, k, v, 0.5, 0.25)
    else:
        binding.norm_rope_write_kv(x, x, x, None, None, slots, k, v)
        assert torch.equal(v[blocks - 1, :, 13:].transpose(0, 1), x)
    assert binding.get_device_error(True)[0] == 0
    del k, v
    torch.cuda.empty_cache()


def test_two_streams_at_once(pa_lib):
    """Calls that overlap on the GPU, each with its own workspace and outputs."""
    from paged_kv_cache_42_gb300 import binding
    spans = [[(1500, 1), (90, 130), (700, 1)], [(400, 260), (33, 1)]]
    bs = [ref.Batch(s, 16, 4, 128, 20 + i, extra_blocks=24) for i, s in enumerate(spans)]
    gs = [b.gpu() for b in bs]
    ws = [torch.rand(len(b.spans), 4, b.mb * 16, device="cuda") for b in bs]

    def calls(i):
        b, g = bs[i], gs[i]
        kw = {"max_query_len": b.max_q, "max_seq_len": b.max_len}
        args = (g["q"], g["k"], g["v"], g["tables"], g["seq_lens"], g["qsl"], b.scale)
        a = binding.attention_window(*args, window=300, sinks=4, **kw)
        o = binding.attention_weights(g["q"], g["k"], g["tables"], g["seq_lens"], g["qsl"], b.scale,
                                      ws[i], out=torch.zeros_like(ws[i]), **kw)
        R = len(b.spans)
        kept = torch.zeros(R, 4, 100, dtype=torch.int32, device="cuda")
        nw = torch.zeros(R, 4, 100, device="cuda")
        e = binding.evict_kv(g["k"], g["v"], g["tables"], g["seq_lens"], ws[i],
                             g["free"][:R * 7].view(R, 7).contiguous(), keep=100, recent=20, sinks=4,
                             max_seq_len=b.max_len, kept=kept, new_weights=nw)
        return a, o, *e

    alone = []
    for i in (0, 1):
        alone.append([t.clone() for t in calls(i)])
        torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in bs]
    for _ in range(4):
        got = [None, None]
        for i in (0, 1):
            streams[i].wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(streams[i]):
                got[i] = calls(i)
        torch.cuda.synchronize()
        for i in (0, 1):
            for x, y in zip(got[i], alone[i]):
                assert torch.equal(x, y)
    assert binding.get_device_error(True)[0] == 0


@pytest.mark.parametrize("fp8", [False, True])
def test_captured_step_follows_its_inputs(pa_lib, fp8):
    """Write, windowed attention, weights and eviction in one graph; lengths,
    tables and values change between replays (within the captured bounds), padding
    tokens among them."""
    from paged_kv_cache_42_gb300 import binding
    binding.get_device_error(True)
    hq, hkv, d, R, T = 16, 2, 128, 3, 8
    batches = [ref.Batch(s, hq, hkv, d, 30 + i, fp8=fp8, extra_blocks=12)
               for i, s in enumerate([[(300, 1), (40, 5), (0, 2)], [(17, 3), (120, 1), (301, 1)],
                                      [(64, 0), (64, 1), (99, 6)]])]
    blocks = max(len(b.k) for b in batches)
    dtype = torch.uint8 if fp8 else torch.bfloat16
    kc = torch.zeros(blocks, hkv, 16, d, dtype=dtype, device="cuda")
    vc = torch.zeros_like(kc)
    tables = torch.zeros(R, 20, dtype=torch.int32, device="cuda")
    sl, qsl = torch.zeros(R, dtype=torch.int32).cuda(), torch.zeros(R + 1, dtype=torch.int32).cuda()
    x = torch.zeros(T, (hq + 2 * hkv) * d, dtype=torch.bfloat16, device="cuda")
    q, k, v = (x[:, a * d:e * d].unflatten(1, (-1, d))
               for a, e in ((0, hq), (hq, hq + hkv), (hq + hkv, hq + 2 * hkv)))
    slots, w = torch.full((T,), -1).cuda(), torch.zeros(R, hkv, 320, device="cuda")
    nt = torch.zeros(R, 4, dtype=torch.int32, device="cuda")
    qo, at, wo = torch.zeros_like(q.contiguous()), torch.zeros_like(q.contiguous()), torch.zeros_like(w)
    lens = torch.zeros(R, dtype=torch.int32, device="cuda")
    kept = torch.zeros(R, hkv, 60, dtype=torch.int32, device="cuda")
    nw = torch.zeros(R, hkv, 60, device="cuda")
    kw = {"max_query_len": 8, "max_seq_len": 320}
    ws1 = torch.empty(binding.workspace_size(R, T, hq, hkv, d), dtype=torch.uint8, device="cuda")
    ws2 = torch.empty(binding.weights_workspace_size(R, T, hq, hkv, d, 8, 320), dtype=torch.uint8,
                      device="cuda")

    def load(b, seed):
        g = torch.Generator().manual_seed(seed)
        n = int(b.qsl[-1])
        kc.zero_(), vc.zero_()
        kc[:len(b.k)] = torch.where(b.k != b.k, 0, b.k) if not fp8 else b.k.masked_fill(b.k == 0x7f, 0)
        vc[:len(b.v)] = torch.where(b.v != b.v, 0, b.v) if not fp8 else b.v.masked_fill(b.v == 0x7f, 0)
        tables.fill_(-1)
        tables[:, :b.mb] = b.tables
        sl.copy_(b.seq_lens), qsl.copy_(b.qsl)
        x.copy_(torch.randn(x.shape, generator=g).bfloat16())
        slots.fill_(-1)
        s = [int(b.tables[r, p // 16]) * 16 + p % 16
             for r, (c, m) in enumerate(b.spans) for p in range(c, c + m)]
        slots[:n] = torch.tensor(s)
        w.copy_(torch.rand(w.shape, generator=g))
        nt.copy_(b.free[:12].view(3, 4))
        for o in (qo, at, wo, kept, nw, lens):
            o.fill_(5)

    def step():
        if fp8:
            binding.norm_rope_write_kv_fp8(q, k, v, None, None, slots, kc, vc, 0.0113, 0.0127, out=qo)
            binding.attention_window_fp8(qo, kc, vc, tables, sl, qsl, 0.1, 0.0113, 0.0127, window=70,
                                         sinks=3, out=at, workspace=ws1, **kw)
            binding.attention_weights_fp8(qo, kc, tables, sl, qsl, 0.1, 0.0113, w, out=wo,
                                          workspace=ws2, **kw)
        else:
            binding.norm_rope_write_kv(q, k, v, None, None, slots, kc, vc, out=qo)
            binding.attention_window(qo, kc, vc, tables, sl, qsl, 0.1, window=70, sinks=3, out=at,
                                     workspace=ws1, **kw)
            binding.attention_weights(qo, kc, tables, sl, qsl, 0.1, w, out=wo, workspace=ws2, **kw)
        binding.evict_kv(kc, vc, tables, sl, wo, nt, keep=60, recent=20, sinks=4, max_seq_len=320,
                         new_seq_lens=lens, kept=kept, new_weights=nw)

    outs = (qo, at, wo, lens, kept, nw, kc, vc)
    want = []
    for i, b in enumerate(batches):
        load(b, i)
        step()
        torch.cuda.synchronize()
        want.append([t.clone() for t in outs])
        n = int(b.qsl[-1])
        assert (qo[n:] == 5).all() and (at[n:] == 5).all()
    assert binding.get_device_error(True)[0] == 0
    graph = torch.cuda.CUDAGraph()
    load(batches[0], 0)
    with torch.cuda.graph(graph):
        step()
    for i in (1, 0, 2, 1):
        load(batches[i], i)
        graph.replay()
        torch.cuda.synchronize()
        for x_, y in zip(outs, want[i]):
            assert torch.equal(x_.view(torch.uint8), y.view(torch.uint8))
    assert binding.get_device_error(True)[0] == 0


def test_attention_right_behind(pa_lib):
    """The split-KV grid of the next call may start as soon as the last grid of
    these ends; many rounds without a synchronise, each from new queries."""
    from paged_kv_cache_42_gb300 import binding
    b = ref.Batch([(700 + 13 * i, 1) for i in range(24)], 32, 8, 128, 40)
    g = b.gpu()
    R = len(b.spans)
    slots = torch.tensor([int(b.tables[r, c // 16]) * 16 + c % 16
                          for r, (c, _) in enumerate(b.spans)]).cuda()
    gen = torch.Generator().manual_seed(3)
    xs = torch.randn(6, R, 48 * 128, generator=gen).bfloat16().cuda()
    ws = torch.empty(binding.workspace_size(R, R, 32, 8, 128), dtype=torch.uint8, device="cuda")
    kw = {"max_query_len": 1, "max_seq_len": b.max_len}
    w = torch.zeros(R, 8, b.mb * 16, device="cuda")
    qo = torch.empty(R, 32, 128, dtype=torch.bfloat16, device="cuda")

    def one(i, out):
        q, k, v = (xs[i][:, a * 128:e * 128].unflatten(1, (-1, 128))
                   for a, e in ((0, 32), (32, 40), (40, 48)))
        binding.norm_rope_write_kv(q, k, v, None, None, slots, g["k"], g["v"], out=qo)
        binding.attention(qo, g["k"], g["v"], g["tables"], g["seq_lens"], g["qsl"], b.scale,
                          out=out, workspace=ws, **kw)
        return out

    want = []
    for i in range(6):
        want.append(one(i, torch.empty_like(qo)).clone())
        torch.cuda.synchronize()
    for _ in range(5):
        got = [one(i, torch.empty_like(qo)) for i in range(6)]
        binding.attention_weights(qo, g["k"], g["tables"], g["seq_lens"], g["qsl"], b.scale, w, **kw)
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(x, y)


def test_memory_of_the_calls_stream(pa_lib, monkeypatch):
    """What a call on another stream allocates comes from that stream."""
    from paged_kv_cache_42_gb300 import binding
    b = ref.Batch([(300, 1), (40, 20)], 8, 2, 64, 11, extra_blocks=6)
    g = b.gpu()
    kw = {"max_query_len": b.max_q, "max_seq_len": b.max_len}
    w = torch.rand(2, 2, b.mb * 16, device="cuda")
    slots = torch.full((21,), -1, dtype=torch.int64, device="cuda")
    kv = torch.zeros(21, 2, 64, dtype=torch.bfloat16, device="cuda")
    new_tables = g["free"].view(2, 3).contiguous()
    side, at = torch.cuda.Stream(), []
    torch.cuda.synchronize()
    empty = torch.empty

    def spy(*args, **kwargs):
        at.append(torch.cuda.current_stream() == side)
        return empty(*args, **kwargs)
    monkeypatch.setattr(torch, "empty", spy)
    args = (g["q"], g["k"], g["v"], g["tables"], g["seq_lens"], g["qsl"], b.scale)
    got = binding.attention_window(*args, window=50, sinks=4, **kw, stream=side)
    binding.norm_rope_write_kv(g["q"], kv, kv, None, None, slots, g["k"], g["v"], stream=side)
    binding.attention_weights(g["q"], g["k"], g["tables"], g["seq_lens"], g["qsl"], b.scale, w,
                              **kw, stream=side)
    binding.evict_kv(g["k"], g["v"], g["tables"], g["seq_lens"], w, new_tables, keep=40, recent=8,
                     max_seq_len=b.max_len, stream=side)
    monkeypatch.undo()
    torch.cuda.synchronize()
    assert at == [True] * 7
    want = ref.window_attention(b.q, b.k, b.v, b.tables, b.seq_lens, b.qsl, b.scale, 50, 4)
    assert (got.cpu().double() - want).abs().max() < 2e-2


@pytest.mark.parametrize("d", [64, 128])
def test_decodes_with_scores_below_any_sentinel(pa_lib, d):
    """Scores of -1e31 and less: key i of a request scores i + 1 times the first
    key's, so the first key the token sees takes the whole weight."""
    from paged_kv_cache_42_gb300 import binding
    b = ref.Batch([(0, 1), (4, 1), (100, 1), (700, 1)], 4, 2, d, 3)
    b.q.fill_(2.0 ** 50)
    for r, (c, n) in enumerate(b.spans):
        i = torch.arange(c + n)
        # one or two bits each: exact in bf16, falling with the position
        val = -(2.0 ** 50) * (1.0 + (i % 128) / 128.0) * 2.0 ** (i // 128)
        b.k[b.tables[r].long()[i // 16], :, i % 16] = val.bfloat16()[:, None, None]
    g = b.gpu()
    kw = {"max_query_len": 1, "max_seq_len": b.max_len}
    out = torch.full((4, 2, b.mb * 16), -7.0, device="cuda")
    zero = torch.zeros_like(out)
    binding.attention_weights(g["q"], g["k"], g["tables"], g["seq_lens"], g["qsl"], b.scale, zero,
                              out=out, **kw)
    got = binding.attention_window(g["q"], g["k"], g["v"], g["tables"], g["seq_lens"], g["qsl"],
                                   b.scale, window=30, **kw).cpu()
    for r, (c, n) in enumerate(b.spans):
        L = c + n
        want = torch.zeros(2, L)
        want[:, 0] = 2.0  # both query heads of the KV head
        assert torch.equal(out[r, :, :L].cpu(), want)
        first = max(0, L - 30)
        v = b.v[b.tables[r, first // 16], :, first % 16]
        assert torch.equal(got[r], v.repeat_interleave(2, 0))


def test_lengths_of_an_eviction_that_cuts_nothing(pa_lib):
    """Attention right behind an eviction reads the lengths it wrote, also where
    no request is longer than `keep` (a single grid then, and no rows moved)."""
    from paged_kv_cache_42_gb300 import binding
    b = ref.Batch([(5 + 7 * i % 90, 1) for i in range(500)], 8, 8, 64, 41)
    g = b.gpu()
    R, keep = len(b.spans), 128
    kw = {"max_query_len": 1, "max_seq_len": b.max_len}
    args = (g["q"], g["k"], g["v"], g["tables"])
    ws = torch.empty(binding.workspace_size(R, R, 8, 8, 64), dtype=torch.uint8, device="cuda")
    want = binding.attention(*args, g["seq_lens"], g["qsl"], b.scale, workspace=ws, **kw)
    w = torch.rand(R, 8, b.mb * 16, device="cuda")
    new_tables = torch.zeros(R, 8, dtype=torch.int32, device="cuda")
    new_lens = torch.empty(R, dtype=torch.int32, device="cuda")
    kept = torch.empty(R, 8, keep, dtype=torch.int32, device="cuda")
    new_w = torch.empty(R, 8, keep, device="cuda")
    torch.cuda.synchronize()
    binding.get_device_error(True)
    for _ in range(50):
        out = torch.empty_like(want)
        new_lens.fill_(1)  # a length that every request may have
        binding.evict_kv(g["k"], g["v"], g["tables"], g["seq_lens"], w, new_tables, keep=keep,
                         recent=8, max_seq_len=b.max_len, new_seq_lens=new_lens, kept=kept,
                         new_weights=new_w)
        binding.attention(*args, new_lens, g["qsl"], b.scale, workspace=ws, out=out, **kw)
        assert torch.equal(out, want)
    assert binding.get_device_error(True)[0] == 0


@pytest.mark.parametrize("fp8", [False, True])
def test_two_graphs_share_a_workspace(pa_lib, fp8):
    """Captured windows and weights of two batches, one workspace, replayed in
    turn: no call depends on what another left there."""
    from paged_kv_cache_42_gb300 import binding
    batches = [ref.Batch([(900, 300), (40, 1), (0, 20)], 32, 8, 128, 50, fp8=fp8),
               ref.Batch([(33, 1), (2100, 1), (5, 130), (16, 0), (700, 3)], 32, 8, 128, 51, fp8=fp8)]
    size = max(max(binding.workspace_size(len(b.spans), len(b.q), 32, 8, 128),
                   binding.weights_workspace_size(len(b.spans), len(b.q), 32, 8, 128, b.max_q,
                                                  b.max_len)) for b in batches)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    steps, alive = [], []
    for b in batches:
        g = b.gpu()
        o = torch.zeros_like(g["q"])
        w = torch.zeros(len(b.spans), 8, b.mb * 16, device="cuda")
        wo = torch.zeros_like(w)

        def step(b=b, g=g, o=o, w=w, wo=wo):
            kw = {"max_query_len": b.max_q, "max_seq_len": b.max_len, "workspace": ws}
            meta = (g["tables"], g["seq_lens"], g["qsl"], b.scale)
            if fp8:
                binding.attention_window_fp8(g["q"], g["k"], g["v"], *meta, b.k_scale, b.v_scale,
                                             window=200, sinks=4, out=o, **kw)
                binding.attention_weights_fp8(g["q"], g["k"], *meta, b.k_scale, w, out=wo, **kw)
            else:
                binding.attention_window(g["q"], g["k"], g["v"], *meta, window=200, sinks=4, out=o,
                                         **kw)
                binding.attention_weights(g["q"], g["k"], *meta, w, out=wo, **kw)
        step()
        torch.cuda.synchronize()
        want = o.clone(), wo.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        steps.append((graph, o, wo, want))
        alive.append(step)  # the graph's inputs
    for i in (0, 1, 1, 0, 0, 1):
        graph, o, wo, want = steps[i]
        o.zero_()
        wo.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want[0]) and torch.equal(wo, want[1])
    for i in (0, 1) * 4:  # and with nothing between the replays
        steps[i][0].replay()
    torch.cuda.synchronize()
    for _, o, wo, want in steps:
        assert torch.equal(o, want[0]) and torch.equal(wo, want[1])
