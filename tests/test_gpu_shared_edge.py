"""pa_attention_shared beside one plain call: other calls' results, wrong metadata,
captured and replayed steps, two streams, results in host memory."""
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


def close(got, b):
    want, tol = b.want()
    mine = ~torch.isnan(want)
    assert ((got.cpu().double() - want).abs() <= tol)[mine].all()


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "rows"])
def test_no_groups_is_the_plain_call(pa_lib, fmt):
    b = sr.Batch([], 32, 8, 128, 4, fmt=fmt, before=[(100, 1), (33, 1), (0, 20), (7, 2)])
    g = b.gpu()
    assert torch.equal(b.run(g), b.plain(g))
    # prefixes of nothing: one launch order or another, the same result
    b = sr.Batch([(0, [(100, 1), (33, 1)])], 32, 8, 128, 4, fmt=fmt)
    g = b.gpu()
    assert torch.equal(b.run(g), b.plain(g))
    close(b.run(g, max_prefix_len=64), b)


def test_against_the_cascade(pa_lib):
    """One group that is the whole batch: both stay within the tolerances."""
    from paged_kv_cache_42_gb300 import binding
    b = sr.Batch([(1024, [(i * 3 % 200, 1) for i in range(60)])], 32, 8, 128, 6)
    g = b.gpu()
    c = binding.attention_cascade(g["q"], g["k"], g["v"], g["tables"], g["seq_lens"], g["qsl"],
                                  b.scale, common_prefix_len=1024, max_query_len=1,
                                  max_seq_len=b.max_len)
    close(c, b)
    close(b.run(g), b)


def test_a_larger_bound_changes_nothing_but_the_order(pa_lib):
    b = sr.Batch([(256, [(9, 1), (40, 1)]), (64, [(3, 1), (4, 1), (50, 1)])], 16, 4, 128, 2, fmt="rows")
    g = b.gpu()
    close(b.run(g, max_prefix_len=100000), b)
    close(b.run(g, max_seq_len=100000, max_query_len=15), b)


@pytest.mark.parametrize("hq,hkv,d,fmt", [(8, 2, 64, "bf16"), (32, 8, 128, "rows")])
def test_wrong_groups_attend_on_their_own(pa_lib, hq, hkv, d, fmt):
    """Groups outside the batch and lengths that are none are reported; every request's
    result is right all the same."""
    from paged_kv_cache_42_gb300 import binding
    b = sr.Batch([(64, [(9, 1), (40, 1)]), (64, [(3, 1), (4, 1)])], hq, hkv, d, 2, fmt=fmt)
    g = b.gpu()
    for loc, prefix, err in (
            ([0, 2, 5], [64, 64], (4, 1)),       # five requests of four
            ([-1, 2, 4], [64, 64], (4, 0)),
            ([0, 3, 1], [64, 64], (4, 1)),
            ([0, 2, 4], [64, 72], (6, 1)),       # no multiple of 16
            ([0, 2, 4], [-16, 64], (6, 0)),
            ([0, 2, 4], [80, 64], (6, 0))):      # longer than max_prefix_len
        binding.get_device_error(True)
        g["group_loc"] = torch.tensor(loc, dtype=torch.int32).cuda()
        g["prefix"] = torch.tensor(prefix, dtype=torch.int32).cuda()
        got = b.run(g)
        if loc != [0, 3, 1]:  # (whose first group holds requests of two prefixes)
            close(got, b)
            assert binding.get_device_error(True) == err, loc
        else:
            assert binding.get_device_error(True)[0] in (4, 6)


def test_a_foreign_prefix_is_reported(pa_lib):
    from paged_kv_cache_42_gb300 import binding
    b = sr.Batch([(640, [(9, 1), (40, 1), (7, 1), (1, 1)])], 16, 4, 128, 2)
    g = b.gpu()
    binding.get_device_error(True)
    b.run(g)
    assert binding.get_device_error(True)[0] == 0
    g["tables"][2, 39] = g["tables"][0, 40]
    b.run(g)
    assert binding.get_device_error(True) == (6, 2)


def test_bad_lengths_skip_their_request(pa_lib):
    from paged_kv_cache_42_gb300 import binding
    b = sr.Batch([(64, [(9, 1), (40, 1), (5, 1)])], 8, 2, 64, 2)
    g = b.gpu()
    want, tol = b.want()
    g["seq_lens"][1] = 10 ** 6
    binding.get_device_error(True)
    out = torch.full(b.q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    b.run(g, out=out)
    assert binding.get_device_error(True) == (3, 1)
    got = out.cpu().double()
    assert (got[1] == 7).all()
    for r in (0, 2):
        assert ((got[r] - want[r]).abs() <= tol[r]).all()


def test_spans_that_overlap_stay_in_bounds(pa_lib):
    """query_start_loc that runs back and forth: reported, and nothing else is touched."""
    from paged_kv_cache_42_gb300 import binding
    b = sr.Batch([(16, [(3, 1), (4, 1), (5, 1)]) for _ in range(4)], 4, 2, 64, 2)
    g = b.gpu()
    T = len(b.q)
    qsl = [0] + [T if i % 2 else 0 for i in range(T)]
    g["qsl"] = torch.tensor(qsl, dtype=torch.int32).cuda()
    g["seq_lens"] += T
    binding.get_device_error(True)
    big = torch.full((T + 64, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    b.run(g, out=big[:T], max_query_len=T, max_seq_len=b.max_len + T)
    assert binding.get_device_error(True)[0] in (3, 4)
    assert (big[T:] == 7).all()


@pytest.mark.parametrize("fmt", ["bf16", "rows"])
def test_captured_step_follows_its_groups(pa_lib, fmt):
    """Groups, prefixes, lengths and queries change between replays, within the bounds."""
    from paged_kv_cache_42_gb300 import binding
    layouts = [
        [(128, [(9, 1), (40, 1), (0, 1)]), (64, [(3, 1), (4, 1), (7, 1)])],
        [(16, [(9, 1), (100, 1)]), (112, [(3, 1), (4, 1), (7, 1), (90, 1)])],
        [(0, [(9, 1), (40, 1), (10, 1), (3, 1), (4, 1)]), (96, [(7, 1)])],
    ]
    bs = [sr.Batch(x, 32, 8, 128, 7 + i, fmt=fmt) for i, x in enumerate(layouts)]
    width = max(b.mb for b in bs)
    blocks = max(len(b.k) for b in bs)

    def padded(b):
        g = b.gpu()
        t = torch.full((6, width), -1, dtype=torch.int32, device="cuda")
        t[:, :b.mb] = g["tables"]
        g["tables"] = t
        for n in ("k", "v", "scales"):
            x = torch.zeros((blocks,) + g[n].shape[1:], dtype=g[n].dtype, device="cuda")
            x[:len(g[n])] = g[n]
            g[n] = x
        return g

    gs = [padded(b) for b in bs]
    live = {n: t.clone() for n, t in gs[0].items()}
    bound = dict(max_prefix_len=128, max_query_len=1, max_seq_len=max(b.max_len for b in bs))
    out = torch.zeros_like(live["q"])
    ws = torch.empty(binding.shared_workspace_size(6, 6, 32, 8, 128, 2, 128), dtype=torch.uint8,
                     device="cuda")
    binding.init()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        bs[0].run(live, out=out, workspace=ws, **bound)
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bs[0].run(live, out=out, workspace=ws, **bound)
    for i in (1, 2, 0, 2, 1):
        for n, t in live.items():
            t.copy_(gs[i][n])
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        close(out, bs[i])
    assert binding.get_device_error(True)[0] == 0


def test_two_streams_at_once(pa_lib):
    from paged_kv_cache_42_gb300 import binding
    bs = [sr.Batch([(512, [(i, 1) for i in range(30)]), (64, [(200, 1), (3, 2)])], 32, 8, 128, 1, fmt="rows"),
          sr.Batch([(1024, [(9, 1), (300, 1)])], 16, 4, 128, 2)]
    gs = [b.gpu() for b in bs]
    alone = [b.run(g).clone() for b, g in zip(bs, gs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in bs]
    for _ in range(5):
        got = [b.run(g, stream=s) for b, g, s in zip(bs, gs, streams)]
        torch.cuda.synchronize()
        for x, y in zip(got, alone):
            assert torch.equal(x, y)
    assert binding.get_device_error(True)[0] == 0


@pytest.mark.parametrize("fmt", ["bf16", "rows"])
def test_result_in_host_memory(pa_lib, fmt):
    b = sr.Batch([(128, [(9, 1), (40, 1), (0, 3)]), (64, [(3, 1), (4, 1)])], 32, 8, 128, 7, fmt=fmt,
                 before=[(30, 20)])
    g = b.gpu()
    host = torch.empty(b.q.shape, dtype=torch.bfloat16).pin_memory()
    b.run(g, out=host)
    torch.cuda.synchronize()
    assert torch.equal(host, b.run(g).cpu())


@pytest.mark.parametrize("option,value", [("decode_tc", 0), ("decode_token_major", 0),
                                          ("decode_max_workers", 5), ("decode_tm_ctas_per_sm", 1)])
def test_options(pa_lib, option, value):
    from paged_kv_cache_42_gb300 import binding
    default = {"decode_tc": 1, "decode_token_major": 1, "decode_max_workers": 0,
               "decode_tm_ctas_per_sm": 2}[option]
    b = sr.Batch([(256, [(9, 1), (40, 1), (500, 1)]), (64, [(3, 1), (4, 1)])], 32, 8, 128, 7, fmt="rows",
                 after=[(700, 1)])
    g = b.gpu()
    binding.set_option(option, value)
    try:
        close(b.run(g), b)
        close(b.plain(g), b)
    finally:
        binding.set_option(option, default)


@pytest.mark.parametrize("fmt", ["bf16", "rows"])
def test_offsets_past_32_bits(pa_lib, fmt):
    """300000 blocks of 8 heads x 16 x 128: 4.9e9 elements a cache."""
    from paged_kv_cache_42_gb300 import binding
    binding.get_device_error(True)
    b = sr.Batch([(256, [(9, 1), (40, 1), (33, 20)]), (64, [(3, 1), (4, 1)])], 32, 8, 128, 7, fmt=fmt)
    g = b.gpu()
    n, blocks = len(b.k), 300000
    for name in ("k", "v", "scales"):
        x = torch.empty((blocks,) + g[name].shape[1:], dtype=g[name].dtype, device="cuda")
        x[blocks - n:] = g[name]
        g[name] = x
    g["tables"] = torch.where(g["tables"] >= 0, g["tables"] + (blocks - n), -1)
    close(b.run(g), b)
    close(b.plain(g), b)
    loc = torch.tensor([0, 100, 100, 200], dtype=torch.int32).cuda()
    kw = dict(num_tokens=200)
    if fmt == "rows":
        k, v = binding.read_kv_rows(g["k"], g["v"], g["scales"], g["tables"][:3], loc, **kw)
    else:
        k, v = binding.read_kv(g["k"], g["v"], g["tables"][:3], loc, **kw)
    from tests import bounded_ref as ref
    for x, w in ((k, b.k64), (v, b.v64)):
        assert torch.equal(x[:100].cpu().double(), ref.dense(w, b.tables[0], 100))
        assert torch.equal(x[100:].cpu().double(), ref.dense(w, b.tables[2], 100))
    slots = (torch.arange(3) + (blocks * 16 - 3)).cuda()
    x = torch.randn(3, 8, 128).bfloat16().cuda()
    if fmt == "rows":
        from tests import rows_ref as rr
        codes, by = rr.quantise(x.cpu())
        binding.write_kv_rows(x, x, slots, g["k"], g["v"], g["scales"])
        assert torch.equal(g["v"][blocks - 1, :, 13:].transpose(0, 1).cpu(), codes)
        assert torch.equal(g["scales"][blocks - 1, :, 1, 13:].T.cpu(), by)
        binding.norm_rope_write_kv_rows(x, x, x, None, None, slots - 3, g["k"], g["v"], g["scales"])
        assert torch.equal(g["k"][blocks - 1, :, 10:13].transpose(0, 1).cpu(), codes)
    assert binding.get_device_error(True)[0] == 0
    del g
    torch.cuda.empty_cache()


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "rows"])
def test_batches_that_do_not_share(pa_lib, fmt):
    """Below the limit the call attends without sharing, above it with: the same result."""
    from paged_kv_cache_42_gb300 import binding
    b = sr.Batch([(256, [(9, 1), (40, 1), (0, 3)]), (1040, [(3, 1), (4, 1)])], 32, 8, 128, 7, fmt=fmt,
                 before=[(30, 1)], after=[(5, 20)])
    g = b.gpu()
    outs = []
    for kb in (24576, 0, 2 ** 31 - 1):
        binding.set_option("shared_min_kb", kb)
        outs.append(b.run(g).clone())
        close(outs[-1], b)
    assert torch.equal(outs[0], outs[2])
    # a long prefix is shared whatever the tokens save
    b = sr.Batch([(4096, [(9, 1), (40, 1)])], 8, 2, 64, 7, fmt=fmt)
    g = b.gpu()
    for kb in (2 ** 31 - 1, 0):
        binding.set_option("shared_min_kb", kb)
        close(b.run(g), b)
    assert binding.get_device_error(True)[0] == 0


@pytest.mark.parametrize("fmt", ["fp8", "rows"])
@pytest.mark.parametrize("d", [64, 128])
def test_a_chunks_blocks_outside_the_pool_count_as_zeros(pa_lib, fmt, d):
    """Over E4M3 caches the rows of such a block are keys and values of zero, and only its
    own request's; and so they are in a shared prefix."""
    from paged_kv_cache_42_gb300 import binding
    b = sr.Batch([], 16, 4, d, 9, fmt=fmt, before=[(700, 40), (333, 64), (900, 20)])
    g = b.gpu()
    binding.get_device_error(True)
    clean = b.plain(g)
    empty = int((set(range(len(b.k))) - set(b.tables.flatten().tolist())).pop())
    for t in ("k", "v"):
        g[t][empty] = 0
    g["scales"][empty] = 127
    spots = [(1, 2), (1, 10), (1, 24)]  # first key tile, second, the chunk's last block
    for r, c in spots:
        g["tables"][r, c] = empty
    want = b.plain(g)
    assert binding.get_device_error(True)[0] == 0
    for r, c in spots:
        g["tables"][r, c] = len(b.k) + 5
    got = b.plain(g)
    assert binding.get_device_error(True)[0] == 2
    assert torch.equal(got, want)
    assert torch.equal(got[:40], clean[:40]) and torch.equal(got[104:], clean[104:])

    b = sr.Batch([(640, [(9, 1), (40, 1), (7, 1)])], 16, 4, d, 2, fmt=fmt)
    g = b.gpu()
    empty = int((set(range(len(b.k))) - set(b.tables.flatten().tolist())).pop())
    for t in ("k", "v"):
        g[t][empty] = 0
    g["scales"][empty] = 127
    g["tables"][:, 17] = empty
    want = b.run(g)
    assert binding.get_device_error(True)[0] == 0
    g["tables"][:, 17] = -3
    assert torch.equal(b.run(g), want)
    assert binding.get_device_error(True)[0] == 2


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("group", [1, 2, 4, 8])
def test_many_tokens_of_many_heads(pa_lib, group, d):
    """Merged by a warp per (token, KV head) or part of its query heads."""
    from paged_kv_cache_42_gb300 import binding
    b = sr.Batch([(160, [(i % 37, 1) for i in range(40)]), (1040, [(i % 5, 1) for i in range(30)])],
                 16 * group, 16, d, 4, before=[(70, 1)], trailing_tokens=1)
    g = b.gpu()
    binding.get_device_error(True)
    close(b.run(g), b)
    assert binding.get_device_error(True)[0] == 0


@pytest.mark.parametrize("groups", [[(640, [(9, 1), (40, 1), (7, 1)])], []])
@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_scales_of_another_format_are_ignored(pa_lib, monkeypatch, fmt, groups):
    from paged_kv_cache_42_gb300 import binding
    b = sr.Batch(groups, 32, 8, 128, 2, fmt=fmt, before=[(300, 1), (50, 20)])
    g = b.gpu()
    want = b.run(g).clone()
    pack = binding._pack_sh
    assert pack is not None
    stray = torch.full((len(b.k), 8, 2, 16), 120, dtype=torch.uint8, device="cuda")
    monkeypatch.setattr(binding, "_pack_sh",
                        lambda *a: pack(*a[:3], stray.data_ptr(), *a[4:]))
    assert torch.equal(b.run(g), want)


@pytest.mark.parametrize("fmt", ["bf16", "rows"])
def test_as_many_groups_as_there_may_be(pa_lib, fmt):
    from paged_kv_cache_42_gb300 import binding
    b = sr.Batch([(16 * (1 + i % 3), [(i % 40, 1), (i % 7, 1)] + [(i % 11, 2)] * (i % 5 == 0))
                  for i in range(1024)], 4, 2, 64, 6, fmt=fmt)
    g = b.gpu()
    binding.get_device_error(True)
    close(b.run(g), b)
    assert binding.get_device_error(True)[0] == 0
    for grp in (0, 31, 32, 700, 1023):
        last = int(b.group_loc[grp + 1]) - 1
        keep = int(g["tables"][last, 0])
        other = int(b.group_loc[grp]) - 1 if grp else last + 1  # a request of the next group
        g["tables"][last, 0] = int(g["tables"][other, 0])
        b.run(g)
        assert binding.get_device_error(True) == (6, last)
        g["tables"][last, 0] = keep
    b.run(g)
    assert binding.get_device_error(True)[0] == 0


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_more_tokens_than_the_planner_keeps_on_chip(pa_lib, fmt):
    from paged_kv_cache_42_gb300 import binding
    b = sr.Batch([(32, [(i % 9, 1) for i in range(15)])] * 280, 4, 2, 64, 6, fmt=fmt,
                 after=[(5, 20), (40, 1)])
    assert len(b.q) > 4096
    g = b.gpu()
    binding.get_device_error(True)
    close(b.run(g), b)
    assert binding.get_device_error(True)[0] == 0
