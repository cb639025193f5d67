"""Row-scaled E4M3 caches on the GPU: the write, the write behind norm and rotation,
attention and reading back, against the definitions in 64 bits."""
from __future__ import annotations

import math

import pytest
import torch

from tests import bounded_ref as ref
from tests import rows_ref as rr

pytestmark = pytest.mark.gpu

BF_MAX = torch.finfo(torch.bfloat16).max


def rows(T, hkv, d, seed):
    """bf16 rows of every kind: ordinary, of one element, at the borders of a scale, zero,
    tiny, huge, with infinities and NaN."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, hkv, d, generator=g).bfloat16()
    flat = x.view(-1, d)
    special = [
        torch.zeros(d), torch.full((d,), -0.0), torch.full((d,), 2.0 ** -133),
        torch.full((d,), BF_MAX), flat[0].float() * 2.0 ** 120, flat[1 % len(flat)].float() * 2.0 ** -110,
        torch.full((d,), 448.0), torch.full((d,), 450.0), torch.full((d,), -448.0 * 2.0 ** 5),
        torch.full((d,), 7.0 * 2.0 ** -20), torch.full((d,), 447.0),
    ]
    for v in (math.inf, -math.inf, math.nan):
        s = flat[2 % len(flat)].float().clone()
        s[d // 3] = v
        special.append(s)
    s = torch.zeros(d)
    s[-1] = -3.0
    special.append(s)
    n = min(len(special), len(flat) // 2)
    at = torch.randperm(len(flat), generator=g)[:n]
    which = torch.randperm(len(special), generator=g)[:n]
    for i, w in zip(at, which):
        flat[i] = special[int(w)].bfloat16()
    return x


def junk(blocks, hkv, d, seed):
    g = torch.Generator().manual_seed(seed)
    return [torch.randint(0, 256, s, generator=g, dtype=torch.uint8) for s in
            ((blocks, hkv, 16, d), (blocks, hkv, 16, d), (blocks, hkv, 2, 16))]


@pytest.mark.parametrize("T,hkv,d,strided", [
    (1, 1, 64, False), (1, 8, 128, True), (3, 2, 64, True), (5, 3, 128, False), (17, 5, 64, True),
    (64, 8, 128, True), (300, 2, 128, False), (1000, 8, 64, True), (33, 1, 128, False)])
def test_write_is_exact(pa_lib, T, hkv, d, strided):
    from paged_kv_cache_42_gb300 import binding
    binding.get_device_error(True)
    k, v = rows(T, hkv, d, T + d), rows(T, hkv, d, T + d + 1)
    blocks = T // 16 + 7
    kc, vc, sc = junk(blocks, hkv, d, 5)
    g = torch.Generator().manual_seed(9)
    slots = torch.randperm(blocks * 16, generator=g)[:T]
    if T > 2:
        slots[T // 2] = -1  # a padding token
    want = [kc.clone(), vc.clone(), sc.clone()]
    for i, x in enumerate((k, v)):
        codes, b = rr.quantise(x)
        for t in range(T):
            s = int(slots[t])
            if s >= 0:
                want[i][s // 16, :, s % 16] = codes[t]
                want[2][s // 16, :, i, s % 16] = b[t]
    kg, vg = k.cuda(), v.cuda()
    if strided:  # parts of a wider projection, 8 elements of something else before them
        wide = torch.full((T, 2 * hkv * d + 24), math.nan, dtype=torch.bfloat16, device="cuda")
        wide[:, 8:8 + hkv * d] = kg.flatten(1)
        wide[:, 16 + hkv * d:16 + 2 * hkv * d] = vg.flatten(1)
        kg = wide[:, 8:8 + hkv * d].unflatten(1, (hkv, d))
        vg = wide[:, 16 + hkv * d:16 + 2 * hkv * d].unflatten(1, (hkv, d))
    got = [t.cuda() for t in (kc, vc, sc)]
    binding.write_kv_rows(kg, vg, slots.cuda(), *got)
    for a, b, name in zip(got, want, ("k", "v", "scales")):
        assert torch.equal(a.cpu(), b), name
    assert binding.get_device_error(True)[0] == 0


def test_write_skips_slots_outside_the_pool(pa_lib):
    from paged_kv_cache_42_gb300 import binding
    binding.get_device_error(True)
    k = torch.randn(4, 2, 64).bfloat16()
    kc, vc, sc = junk(3, 2, 64, 1)
    got = [t.cuda() for t in (kc, vc, sc)]
    binding.write_kv_rows(k.cuda(), k.cuda(), torch.tensor([48, -5, 2 ** 40, 47]).cuda(), *got)
    codes, b = rr.quantise(k)
    for i in (0, 1):
        (kc, vc)[i][2, :, 15] = codes[3]
        sc[2, :, i, 15] = b[3]
    for a, w in zip(got, (kc, vc, sc)):
        assert torch.equal(a.cpu(), w)
    code, at = binding.get_device_error(True)
    assert code == 1 and at in (0, 2)


def table(n, rot):
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    a = torch.arange(n, dtype=torch.float64)[:, None] * inv
    return torch.cat([a.cos(), a.sin()], 1).float()


@pytest.mark.parametrize("T,hq,hkv,d,rot,inter,norm", [
    (1, 1, 1, 64, 64, False, True), (3, 8, 2, 128, 128, True, True), (7, 6, 3, 64, 32, False, False),
    (20, 32, 8, 128, 64, False, True), (9, 4, 4, 128, 0, False, True), (5, 5, 5, 64, 48, True, False),
    (1200, 32, 8, 128, 128, False, True), (2500, 16, 4, 64, 64, True, True), (900, 7, 7, 128, 96, False, True)])
def test_norm_rope_write(pa_lib, T, hq, hkv, d, rot, inter, norm):
    from paged_kv_cache_42_gb300 import binding
    binding.get_device_error(True)
    g = torch.Generator().manual_seed(T + rot)
    x = torch.randn(T, (hq + 2 * hkv) * d, generator=g).bfloat16()
    x *= torch.exp2(torch.randint(-6, 7, (T, 1), generator=g).float()).bfloat16()
    q, k, v = (x[:, a * d:b * d].unflatten(1, (-1, d)) for a, b in
               ((0, hq), (hq, hq + hkv), (hq + hkv, hq + 2 * hkv)))
    qw = (1 + 0.1 * torch.randn(d, generator=g)).bfloat16() if norm else None
    kw = (1 + 0.1 * torch.randn(d, generator=g)).bfloat16() if norm else None
    cs = table(500, rot) if rot else None
    pos = torch.randint(0, 500, (T,), generator=g, dtype=torch.int32) if rot else None
    blocks = T // 16 + 3
    kc, vc, sc = junk(blocks, hkv, d, 3)
    slots = torch.randperm(blocks * 16, generator=g)[:T]
    if T > 2:
        slots[1] = -7
    xg = x.cuda()
    args = [xg[:, a * d:b * d].unflatten(1, (-1, d)) for a, b in
            ((0, hq), (hq, hq + hkv), (hq + hkv, hq + 2 * hkv))]
    cuda = lambda t: None if t is None else t.cuda()  # noqa: E731
    got = [t.cuda() for t in (kc, vc, sc)]
    out = torch.full((T, hq, d), math.nan, dtype=torch.bfloat16, device="cuda")
    binding.norm_rope_write_kv_rows(*args, cuda(pos), cuda(cs), slots.cuda(), *got,
                                    q_weight=cuda(qw), k_weight=cuda(kw), interleaved=inter, out=out)
    gk, gv, gs = (t.cpu() for t in got)
    live = slots >= 0
    q64 = ref.norm_rope(q, qw, 1e-6, cs, pos, inter)
    k64 = ref.norm_rope(k, kw, 1e-6, cs, pos, inter)
    # half a bf16 step, and binary32 arithmetic on elements up to the row's largest
    tol = q64.abs() * 2.0 ** -8 + q64.abs().amax(-1, keepdim=True) * 2.0 ** -18
    assert ((out.cpu().double() - q64).abs() <= tol)[live].all()
    assert torch.isnan(out.cpu()[~live]).all()
    # V: the definition exactly
    codes, b = rr.quantise_fast(v.float())
    at = (slots[live] // 16, slice(None), slots[live] % 16)
    assert torch.equal(gv[at], codes[live]) and torch.equal(gs[:, :, 1][at], b[live])
    # K: binary32 before the rounding; a scale's byte may differ where the largest element
    # lies within that of a border
    top = k64[live].abs().amax(-1)
    e = gs[:, :, 0][at].double() - 127
    near = 2.0 ** -18
    assert (top <= 448 * torch.exp2(e) * (1 + near)).all()
    assert (top >= 224 * torch.exp2(e) * (1 - near)).all()
    y = rr.values(gk[at], gs[:, :, 0][at])
    tol = k64[live].abs() * 2.0 ** -4 + torch.exp2(e)[..., None] * 2.0 ** -10 + top[..., None] * near
    assert ((y - k64[live]).abs() <= tol).all()
    # nothing else was touched
    for t, was in ((gk, kc), (gv, vc)):
        t, was = t.clone(), was.clone()
        t[at] = was[at] = 0
        assert torch.equal(t, was)
    gs, sc = gs.clone(), sc.clone()
    for i in (0, 1):
        gs[:, :, i][at] = sc[:, :, i][at] = 0
    assert torch.equal(gs, sc)
    assert binding.get_device_error(True)[0] == 0


def test_norm_rope_write_of_rows_that_are_not_finite(pa_lib):
    """V rows as they are; K rows through the rotation: NaN bytes, codes of zero."""
    from paged_kv_cache_42_gb300 import binding
    x = torch.randn(4, 3, 64).bfloat16()
    x[1, 1, 5], x[2, 1, 60], x[3, 1, 0] = math.inf, math.nan, -math.inf
    x[0, 1] = 0
    got = [t.cuda() for t in junk(1, 1, 64, 2)]
    cs, pos = table(8, 64).cuda(), torch.tensor([1, 2, 3, 4], dtype=torch.int32).cuda()
    xg = x.cuda()
    binding.norm_rope_write_kv_rows(xg[:, :1], xg[:, 1:2], xg[:, 1:2], pos, cs,
                                    torch.arange(4).cuda(), *got)
    for i in (0, 1):
        assert got[2][0, 0, i, :4].tolist() == [27, 255, 255, 255]
        assert not got[i][0, 0, 1:4].any()


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "rows"])
@pytest.mark.parametrize("hkv,d,lens,first", [
    (1, 64, [1], None), (2, 128, [5, 0, 33, 16], None), (8, 128, [100, 1, 257, 0, 3], [0, 15, 16, 4, 31]),
    (3, 64, [40] * 50, None), (4, 64, [0, 0, 7, 0], [3, 0, 250, 0]), (5, 128, [2000, 1500], [1, 17])])
def test_read(pa_lib, fmt, hkv, d, lens, first):
    from paged_kv_cache_42_gb300 import binding
    binding.get_device_error(True)
    f = first or [0] * len(lens)
    b = rr.Batch([(a + n + 2, 1) for a, n in zip(f, lens)], hkv, hkv, d, 4) if fmt == "rows" else \
        ref.Batch([(a + n + 2, 1) for a, n in zip(f, lens)], hkv, hkv, d, 4, fp8=fmt == "fp8")
    g = b.gpu()
    # two rows before the first request and three behind the last belong to nobody
    loc = torch.tensor([2] + lens).cumsum(0).int()
    T = int(loc[-1]) + 3
    kw = {"first": None if first is None else torch.tensor(first, dtype=torch.int32).cuda()}
    if fmt == "bf16":
        want = [b.k.double(), b.v.double()]
    elif fmt == "fp8":  # the binary32 product, rounded once more to bf16
        want = [(c.view(torch.float8_e4m3fn).float() * torch.tensor(s)).bfloat16().double()
                for c, s in ((b.k, b.k_scale), (b.v, b.v_scale))]
    else:
        want = [b.k64, b.v64]
    for given in (False, True):
        if given:
            kw["k_out"] = torch.full((T, hkv, d), 7.0, dtype=torch.bfloat16, device="cuda")
            kw["v_out"] = torch.full_like(kw["k_out"], 7.0)
        else:
            kw["num_tokens"] = T
        if fmt == "bf16":
            got = binding.read_kv(g["k"], g["v"], g["tables"], loc.cuda(), **kw)
        elif fmt == "fp8":
            got = binding.read_kv_fp8(g["k"], g["v"], g["tables"], loc.cuda(), b.k_scale, b.v_scale,
                                      **kw)
        else:
            got = binding.read_kv_rows(g["k"], g["v"], g["scales"], g["tables"], loc.cuda(), **kw)
        for x, w in zip(got, want):
            x = x.cpu()
            assert x.shape == (T, hkv, d) and x.dtype == torch.bfloat16
            for r, (a, n) in enumerate(zip(f, lens)):
                y = ref.dense(w, b.tables[r], a + n)[a:]
                assert torch.equal(x[int(loc[r]):int(loc[r + 1])].double(), y), r
            if given:
                assert (x[:2] == 7).all() and (x[-3:] == 7).all()
    assert binding.get_device_error(True)[0] == 0


def test_read_of_rows_that_are_not_finite_and_of_codes(pa_lib):
    """Every code under scales from the smallest to the largest; a poisoned row is NaN."""
    from paged_kv_cache_42_gb300 import binding
    codes = torch.arange(256, dtype=torch.uint8)
    codes[127], codes[255] = 0, 0  # the NaN codes, which no write makes
    k = codes.view(2, 1, 1, 128).repeat(1, 1, 16, 1)
    by = torch.tensor([27, 28, 100, 119, 120, 127, 130, 200, 245, 246, 255, 27, 27, 27, 27, 27])
    sc = by.to(torch.uint8).view(1, 1, 1, 16).repeat(2, 1, 2, 1)
    loc = torch.tensor([0, 32], dtype=torch.int32).cuda()
    bt = torch.tensor([[1, 0]], dtype=torch.int32).cuda()
    kk, vv = binding.read_kv_rows(k.cuda(), k.cuda(), sc.cuda(), bt, loc, num_tokens=32)
    want = rr.values(k.flip(0), sc.flip(0)[:, :, 0]).transpose(1, 2).reshape(32, 1, 128)
    bad = torch.isnan(want)
    assert bad.view(2, 16, 128)[:, 10].all() and int(bad.sum()) == 256
    for x in (kk, vv):
        x = x.cpu().double()
        assert torch.equal(torch.isnan(x), bad) and torch.equal(x[~bad], want[~bad])


def test_read_skips_what_is_wrong(pa_lib):
    from paged_kv_cache_42_gb300 import binding
    b = ref.Batch([(20, 1), (40, 1), (20, 1)], 2, 2, 64, 1)
    g = b.gpu()

    def read(loc, first=None, tables=None, T=60):
        binding.get_device_error(True)
        out = [torch.full((T, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
        binding.read_kv(g["k"], g["v"], g["tables"] if tables is None else tables,
                        torch.tensor(loc, dtype=torch.int32).cuda(),
                        first=None if first is None else torch.tensor(first, dtype=torch.int32).cuda(),
                        k_out=out[0], v_out=out[1])
        return out[0].cpu(), binding.get_device_error(True)

    k0, k1 = ref.dense(b.k, b.tables[0], 10), ref.dense(b.k, b.tables[1], 40)
    x, err = read([0, 10, 50, 70])                   # the last rows do not exist
    assert err == (4, 2) and torch.equal(x[:10], k0) and torch.equal(x[10:50], k1) and (x[50:] == 7).all()
    x, err = read([0, 10, 50, 55], [0, 9, 0])        # 49 keys, the table holds 48
    assert err == (3, 1) and torch.equal(x[:10], k0) and (x[10:50] == 7).all()
    x, err = read([0, 10, 50, 55], [-1, 0, 0])
    assert err == (3, 0) and (x[:10] == 7).all() and torch.equal(x[10:50], k1)
    bad = g["tables"].clone()
    bad[1, 1] = len(b.k)
    x, err = read([0, 10, 50, 55], tables=bad)
    assert err == (2, 1) and (x[26:42] == 7).all() and torch.equal(x[10:26], k1[:16])
    assert torch.equal(x[42:50], k1[32:40])


SPANS = {
    "one key": [(0, 1)],
    "short decodes": [(8, 1), (55, 1), (16, 1), (32, 1), (0, 1), (15, 1)],
    "long and short": [(1500, 1), (3, 1), (700, 1), (31, 1)],
    "short spans": [(40, 3), (0, 2), (100, 15), (17, 1)],
    "chunk": [(0, 40)],
    "chunks": [(130, 65), (0, 16), (300, 130)],
    "mixed": [(25, 1), (0, 40), (130, 1), (0, 0), (64, 200), (511, 1), (33, 5)],
}


@pytest.mark.parametrize("name", list(SPANS))
@pytest.mark.parametrize("hq,hkv,d", [(1, 1, 64), (4, 2, 64), (16, 4, 64), (8, 1, 64), (2, 2, 128),
                                      (4, 2, 128), (32, 8, 128), (8, 1, 128), (64, 8, 128), (8, 8, 128),
                                      (16, 8, 128)])
def test_attention(pa_lib, name, hq, hkv, d):
    from paged_kv_cache_42_gb300 import binding
    binding.get_device_error(True)
    b = rr.Batch(SPANS[name], hq, hkv, d, 11, trailing_tokens=2, pad_blocks=1)
    g = b.gpu()
    want, tol = rr.attention(b, b.k64, b.v64)
    out = torch.full(b.q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    binding.attention_rows(g["q"], g["k"], g["v"], g["scales"], g["tables"], g["seq_lens"], g["qsl"],
                           b.scale, max_query_len=b.max_q, max_seq_len=b.max_len, out=out)
    got = out.cpu().double()
    mine = ~torch.isnan(want)
    assert ((got - want).abs() <= tol)[mine].all(), float(((got - want).abs() / tol)[mine].max())
    assert (got[~mine] == 7).all()
    assert binding.get_device_error(True)[0] == 0


@pytest.mark.parametrize("hq,hkv,d", [(4, 2, 64), (32, 8, 128), (64, 8, 128), (8, 1, 128)])
@pytest.mark.parametrize("spread", [0.0, 12.0, 40.0])
def test_attention_over_rows_of_very_different_sizes(pa_lib, hq, hkv, d, spread):
    """Values of 2^-40 to 2^40 beside each other; keys alike, at a scale that keeps the
    scores apart but the softmax from being one key's alone."""
    from paged_kv_cache_42_gb300 import binding
    b = rr.Batch([(700, 1), (50, 1), (20, 60), (3, 3)], hq, hkv, d, 3, spread=0.0)
    g = torch.Generator().manual_seed(1)
    by = torch.round((torch.rand(b.scales[:, :, 1].shape, generator=g) - 0.5) * 2 * spread)
    b.scales[:, :, 1] = torch.where(b.scales[:, :, 1] == 255, 255, b.scales[:, :, 1] + by).to(torch.uint8)
    v64 = rr.values(b.v, b.scales[:, :, 1])
    want, tol = rr.attention(b, b.k64, v64)
    t = b.gpu()
    got = binding.attention_rows(t["q"], t["k"], t["v"], t["scales"], t["tables"], t["seq_lens"],
                                 t["qsl"], b.scale, max_query_len=b.max_q, max_seq_len=b.max_len)
    assert ((got.cpu().double() - want).abs() <= tol).all()


@pytest.mark.parametrize("hq,hkv,d", [(4, 2, 64), (32, 8, 128), (64, 8, 128)])
def test_attention_over_zero_and_poisoned_rows(pa_lib, hq, hkv, d):
    from paged_kv_cache_42_gb300 import binding
    b = rr.Batch([(100, 1), (47, 1), (16, 1), (300, 1)], hq, hkv, d, 5)
    G = hq // hkv
    # request 0: every value zero; 1: some keys and values zero; 2: a NaN value of head 0;
    # 3: a NaN key of the last head
    def rows_of(r, pos):
        return b.tables[r].long()[torch.tensor(pos) // 16], torch.tensor(pos) % 16

    for r, pos, which in ((0, list(range(101)), 1), (1, list(range(0, 48, 2)), 1),
                          (1, list(range(0, 48, 3)), 0)):
        blk, off = rows_of(r, pos)
        (b.k, b.v)[which][blk, :, off] = 0
        b.scales[blk, :, which, off] = 27
    for r, pos, which, h in ((2, [4], 1, 0), (3, [299], 0, hkv - 1)):
        blk, off = rows_of(r, pos)
        (b.k, b.v)[which][blk, h, off] = 0
        b.scales[blk, h, which, off] = 255
    want, tol = rr.attention(b, rr.values(b.k, b.scales[:, :, 0]), rr.values(b.v, b.scales[:, :, 1]))
    t = b.gpu()
    got = binding.attention_rows(t["q"], t["k"], t["v"], t["scales"], t["tables"], t["seq_lens"],
                                 t["qsl"], b.scale, max_query_len=1, max_seq_len=b.max_len).cpu().double()
    bad = torch.isnan(want)
    assert bad[2, :G].all() and bad[3, -G:].all() and int(bad.sum()) == 2 * G * d
    assert torch.equal(torch.isnan(got), bad)
    assert (got[0] == 0).all()
    assert ((got - want).abs() <= tol)[~bad].all()


@pytest.mark.parametrize("hq,hkv,d", [(4, 2, 64), (16, 8, 128), (32, 8, 128), (64, 8, 128)])
@pytest.mark.parametrize("octaves", [13.0, 15.0, 15.6])
def test_a_flat_tail_behind_one_large_weight(pa_lib, hq, hkv, d, octaves):
    """One key of 2^octaves times the weight of each of the others, which together weigh
    about as much: their values must count, although each is small. Outputs are 64-bit
    ones to half a bf16 step and 2^-6 of the weights' sum of |V|."""
    from paged_kv_cache_42_gb300 import binding
    n = int(2.0 ** octaves)
    b = rr.Batch([(n, 1)], hq, hkv, d, 3, spread=0.0)
    g = torch.Generator().manual_seed(2)
    k = torch.zeros(len(b.k), hkv, 16, d)
    v = 1 + 0.25 * torch.randn(len(b.k), hkv, 16, d, generator=g)
    where = b.tables[0, 3].long(), 5  # key 53
    k[where[0], :, where[1], 0] = 16.0
    v[where[0], :, where[1]] = -1.0
    b.k, b.scales[:, :, 0] = rr.quantise_fast(k)
    b.v, b.scales[:, :, 1] = rr.quantise_fast(v)
    b.q.zero_()
    b.q[:, :, 0] = 2.0
    b.scale = octaves * math.log(2) / 32
    k64, v64 = rr.values(b.k, b.scales[:, :, 0]), rr.values(b.v, b.scales[:, :, 1])
    want, _ = rr.attention(b, k64, v64)
    size, _ = rr.attention(b, k64, v64.abs())
    t = b.gpu()
    got = binding.attention_rows(t["q"], t["k"], t["v"], t["scales"], t["tables"], t["seq_lens"],
                                 t["qsl"], b.scale, max_query_len=1, max_seq_len=b.max_len)
    err = (got.cpu().double() - want).abs()
    assert (err <= want.abs() * 2.0 ** -8 + size * 2.0 ** -6).all(), float((err / size).max())
