"""The row-scaled cache's operators and shared prefixes together, as a serving loop uses
them: prompts that share a system prompt are written through norm and rotation, decoded in
groups, read back, and moved into another cache. A 64-bit model beside it works on the rows
that the slots hold."""
from __future__ import annotations

import math

import pytest
import torch

from tests import bounded_ref as ref
from tests import rows_ref as rr

pytestmark = pytest.mark.gpu

SCALE = 1 / math.sqrt(128)


def table(n, d):
    inv = 10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)
    a = torch.arange(n, dtype=torch.float64)[:, None] * inv
    return torch.cat([a.cos(), a.sin()], 1).float()


@pytest.mark.parametrize("hq,hkv,d", [(32, 8, 128), (8, 2, 64), (8, 4, 128)])
def test_serving_loop(pa_lib, hq, hkv, d):
    from paged_kv_cache_42_gb300 import binding, host
    binding.get_device_error(True)
    binding.set_option("shared_min_kb", 0)  # share, however little it saves
    g = torch.Generator().manual_seed(5)
    blocks, prefix = 96, 48
    pool = host.BlockPool(blocks)
    kc = torch.randint(0, 256, (blocks, hkv, 16, d), generator=g, dtype=torch.uint8).cuda()
    vc, sc = kc.clone(), torch.full((blocks, hkv, 2, 16), 255, dtype=torch.uint8, device="cuda")
    cs = table(512, d).cuda()
    qw, kw = ((1 + 0.1 * torch.randn(d, generator=g)).bfloat16().cuda() for _ in "qk")
    shared = [int(b) for b in pool.allocate(prefix // 16)]
    own = [[] for _ in range(5)]         # requests 0 .. 3 share the prefix, 4 does not
    length = [prefix] * 4 + [0]
    width = 12

    def table_of(r):
        return (shared if r < 4 else []) + own[r]

    def tables():
        t = torch.full((5, width), -1, dtype=torch.int32)
        for r in range(5):
            t[r, :len(table_of(r))] = torch.tensor(table_of(r), dtype=torch.int32)
        return t

    def project(T):
        x = torch.randn(T, (hq + 2 * hkv) * d, generator=g)
        x = (x * torch.exp2(torch.randint(-2, 3, (T, 1), generator=g).float())).bfloat16().cuda()
        return [x[:, a * d:b * d].unflatten(1, (-1, d)) for a, b in
                ((0, hq), (hq, hq + hkv), (hq + hkv, hq + 2 * hkv))]

    def write(parts, pos, slots):
        q, k, v = parts
        pos, slots = torch.tensor(pos, dtype=torch.int32).cuda(), torch.tensor(slots).cuda()
        qo = binding.norm_rope_write_kv_rows(q, k, v, pos, cs, slots, kc, vc, sc, q_weight=qw,
                                             k_weight=kw)
        want = ref.norm_rope(k.cpu(), kw.cpu(), 1e-6, cs.cpu(), pos.cpu(), False)
        held = rr.values(kc.cpu(), sc.cpu()[:, :, 0])[slots.cpu() // 16, :, slots.cpu() % 16]
        top = want.abs().amax(-1, keepdim=True)
        # half an E4M3 step; its smallest is 2^-9 of a scale, and 2^-e is above top / 448 / 2
        assert ((held - want).abs() <= want.abs() * 2.0 ** -4 + top * 2.0 ** -17).all()
        return qo

    # the system prompt, written once by request 0's program
    write(project(prefix), list(range(prefix)), [shared[p // 16] * 16 + p % 16 for p in range(prefix)])

    def step(new):
        qsl, pos, slots = [0], [], []
        for r in range(5):
            while len(table_of(r)) * 16 < length[r] + new[r]:
                own[r] += [int(b) for b in pool.allocate(1)]
            for j in range(new[r]):
                p = length[r] + j
                pos.append(p)
                slots.append(table_of(r)[p // 16] * 16 + p % 16)
            length[r] += new[r]
            qsl.append(qsl[-1] + new[r])
        q = write(project(qsl[-1]), pos, slots)
        t, sl = tables().cuda(), torch.tensor(length, dtype=torch.int32).cuda()
        ql = torch.tensor(qsl, dtype=torch.int32).cuda()
        bounds = dict(max_query_len=max(new), max_seq_len=max(length))
        outs = [binding.attention_shared_rows(
            q, kc, vc, sc, t, sl, ql, torch.tensor([0, 4], dtype=torch.int32).cuda(),
            torch.tensor([prefix], dtype=torch.int32).cuda(), SCALE, max_prefix_len=prefix, **bounds),
            binding.attention_rows(q, kc, vc, sc, t, sl, ql, SCALE, **bounds)]
        torch.cuda.synchronize()

        class B:  # what rows_ref.attention wants
            pass
        b = B()
        b.hq, b.hkv, b.q, b.qsl, b.seq_lens, b.tables, b.scale = hq, hkv, q.cpu(), qsl, length, tables(), SCALE
        b.spans = [(length[r] - new[r], new[r]) for r in range(5)]
        k64, v64 = rr.values(kc.cpu(), sc.cpu()[:, :, 0]), rr.values(vc.cpu(), sc.cpu()[:, :, 1])
        want, tol = rr.attention(b, k64, v64)
        for o in outs:
            assert ((o.cpu().double() - want).abs() <= tol).all()

    step([5, 20, 1, 17, 30])             # the users' prompts: chunks and short spans
    for i in range(6):
        step([1, 1, 1, 1, 1] if i % 2 else [1, 0, 2, 1, 1])
    # request 1 leaves: its rows go to a bf16 cache of another program
    n = length[1]
    loc = torch.tensor([0, 0, n, n, n, n], dtype=torch.int32).cuda()
    k, v = binding.read_kv_rows(kc, vc, sc, tables().cuda(), loc, num_tokens=n)
    for x, c, i in ((k, kc, 0), (v, vc, 1)):
        want = ref.dense(rr.values(c.cpu(), sc.cpu()[:, :, i]), tables()[1], n)
        assert torch.equal(x.cpu().double(), want)
    kb = torch.zeros(8, hkv, 16, d, dtype=torch.bfloat16, device="cuda")
    vb = torch.zeros_like(kb)
    binding.write_kv(k, v, torch.arange(n).cuda(), kb, vb)
    back = binding.read_kv(kb, vb, torch.arange(8, dtype=torch.int32).cuda()[None],
                           torch.tensor([0, n], dtype=torch.int32).cuda(), num_tokens=n)
    assert torch.equal(back[0], k) and torch.equal(back[1], v)
    # and back into a row-scaled one: codes and scales are the same again
    k2, v2, s2 = torch.zeros_like(kc), torch.zeros_like(vc), torch.zeros_like(sc)
    binding.write_kv_rows(k, v, torch.arange(n).cuda(), k2, v2, s2)
    k3, v3 = binding.read_kv_rows(k2, v2, s2, torch.arange(8, dtype=torch.int32).cuda()[None],
                                  torch.tensor([0, n], dtype=torch.int32).cuda(), num_tokens=n)
    assert torch.equal(k3, k) and torch.equal(v3, v)
    pool.release(own[1])
    binding.set_option("shared_min_kb", 24576)
    assert binding.get_device_error(True)[0] == 0


@pytest.mark.parametrize("overlap", [0, 1])
def test_captured_steps_and_what_comes_before(pa_lib, overlap):
    """Write, attention and reading back in one graph, over inputs that change between
    replays; the option that starts attention beside the write gives the same bits."""
    from paged_kv_cache_42_gb300 import binding
    b = rr.Batch([(40, 1), (700, 1), (31, 1), (16, 1)], 32, 8, 128, 3)
    t = b.gpu()
    new_slots = [int(b.tables[r, (int(b.seq_lens[r]) - 1) // 16]) * 16 + (int(b.seq_lens[r]) - 1) % 16
                 for r in range(4)]
    slots = torch.tensor(new_slots).cuda()
    k_in = torch.zeros(4, 8, 128, dtype=torch.bfloat16, device="cuda")
    v_in, out = k_in.clone(), torch.zeros_like(t["q"])
    loc = torch.tensor([0, 3, 3, 5, 9], dtype=torch.int32).cuda()
    first = (t["seq_lens"] - torch.tensor([3, 0, 2, 4], device="cuda")).int()
    ko = torch.zeros(9, 8, 128, dtype=torch.bfloat16, device="cuda")
    vo = torch.zeros_like(ko)
    ws = torch.empty(binding.workspace_size(4, 4, 32, 8, 128), dtype=torch.uint8, device="cuda")

    def step():
        binding.write_kv_rows(k_in, v_in, slots, t["k"], t["v"], t["scales"])
        binding.attention_rows(t["q"], t["k"], t["v"], t["scales"], t["tables"], t["seq_lens"],
                               t["qsl"], b.scale, max_query_len=1, max_seq_len=b.max_len, out=out,
                               workspace=ws)
        binding.read_kv_rows(t["k"], t["v"], t["scales"], t["tables"], loc, first=first, k_out=ko,
                             v_out=vo)

    binding.set_option("write_overlap", overlap)
    try:
        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        g = torch.Generator().manual_seed(9)
        for i in range(6):
            k_in.copy_(torch.randn(4, 8, 128, generator=g) * 2.0 ** (i - 3))
            v_in.copy_(torch.randn(4, 8, 128, generator=g) * 2.0 ** (3 - i))
            graph.replay()
            torch.cuda.synchronize()
            for c, s, x in ((b.k, 0, k_in), (b.v, 1, v_in)):
                codes, by = rr.quantise_fast(x.cpu().float())
                for r, slot in enumerate(new_slots):
                    c[slot // 16, :, slot % 16] = codes[r]
                    b.scales[slot // 16, :, s, slot % 16] = by[r]
            k64, v64 = rr.values(b.k, b.scales[:, :, 0]), rr.values(b.v, b.scales[:, :, 1])
            want, tol = rr.attention(b, k64, v64)
            assert ((out.cpu().double() - want).abs() <= tol).all()
            for x, c64 in ((ko, k64), (vo, v64)):
                for r in range(4):
                    n = int(loc[r + 1] - loc[r])
                    L = int(b.seq_lens[r])
                    assert torch.equal(x[int(loc[r]):int(loc[r + 1])].cpu().double(),
                                       ref.dense(c64, b.tables[r], L)[L - n:L])
    finally:
        binding.set_option("write_overlap", 0)
    assert binding.get_device_error(True)[0] == 0


def test_work_enqueued_right_before(pa_lib):
    """Each call reads what the kernel before it on the stream has just written."""
    from paged_kv_cache_42_gb300 import binding
    b = rr.Batch([(300, 1), (40, 1)], 32, 8, 128, 3)
    t = b.gpu()
    kw = dict(max_query_len=1, max_seq_len=b.max_len)
    args = (t["q"], t["k"], t["v"], t["scales"], t["tables"], t["seq_lens"], t["qsl"], b.scale)
    good = binding.attention_rows(*args, **kw).clone()
    loc = torch.tensor([0, 200, 240], dtype=torch.int32).cuda()
    kept = binding.read_kv_rows(*args[1:4], t["tables"], loc, num_tokens=240)[0].clone()
    q, k, s, x = (t[n].clone() for n in ("q", "k", "scales", "tables"))
    big = torch.randn(64 << 20, device="cuda")
    for _ in range(5):
        for n, v in (("q", q), ("k", k), ("scales", s), ("tables", x)):
            t[n].copy_(torch.zeros_like(v))
        big.mul_(1.0)
        for n, v in (("q", q), ("k", k), ("scales", s), ("tables", x)):
            t[n].copy_(v)
        got = binding.attention_rows(*args, **kw)
        rows = binding.read_kv_rows(*args[1:4], t["tables"], loc, num_tokens=240)[0]
        src = torch.zeros(2, 8, 128, dtype=torch.bfloat16, device="cuda")
        big.mul_(1.0)
        src.add_(3.0)
        kc, vc = torch.zeros(1, 8, 16, 128, dtype=torch.uint8, device="cuda"), None
        vc, sc = kc.clone(), torch.zeros(1, 8, 2, 16, dtype=torch.uint8, device="cuda")
        binding.write_kv_rows(src, src, torch.tensor([2, 5]).cuda(), kc, vc, sc)
        assert torch.equal(got, good) and torch.equal(rows, kept)
        assert sc[0, :, :, 2].eq(120).all() and sc[0, :, :, 5].eq(120).all()  # 3 <= 448 x 2^-7


def test_streams_and_devices(pa_lib):
    """Calls on streams of their own at once; tensors of another device are refused."""
    from paged_kv_cache_42_gb300 import binding
    bs = [rr.Batch([(500, 1), (33, 20), (90, 1)], 32, 8, 128, 1), rr.Batch([(300, 1), (2, 3)], 8, 2, 64, 2)]
    ts = [b.gpu() for b in bs]

    def calls(i, stream=None):
        b, t = bs[i], ts[i]
        o = binding.attention_rows(t["q"], t["k"], t["v"], t["scales"], t["tables"], t["seq_lens"],
                                   t["qsl"], b.scale, max_query_len=b.max_q, max_seq_len=b.max_len,
                                   stream=stream)
        n = len(b.spans)
        loc = torch.arange(0, 5 * n + 1, 5, dtype=torch.int32, device="cuda")
        return (o, *binding.read_kv_rows(t["k"], t["v"], t["scales"], t["tables"], loc,
                                         num_tokens=5 * n, stream=stream))

    alone = [[x.clone() for x in calls(i)] for i in (0, 1)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in bs]
    for _ in range(5):
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
        got = []
        for i in (0, 1):
            with torch.cuda.stream(streams[i]):
                got.append(calls(i))
        torch.cuda.synchronize()
        for x, y in zip(got, alone):
            assert all(torch.equal(p, q) for p, q in zip(x, y))
    with pytest.raises(ValueError, match="CUDA|current device"):
        t = ts[0]
        binding.read_kv_rows(t["k"].cpu(), t["v"].cpu(), t["scales"], t["tables"],
                             torch.zeros(4, dtype=torch.int32).cuda(), num_tokens=5)
    assert binding.get_device_error(True)[0] == 0
