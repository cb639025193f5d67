"""pa_norm_rope_write_kv against the 64-bit formula.

Tolerances: each result is rounded once (half a step: bf16 2^-8, E4M3 2^-4 of
the value, 2^-10 below E4M3's normal range), after binary32 arithmetic whose
error is below 2^-18 of the pair's size (a sum of 128 squares, a reciprocal
root, three products)."""
from __future__ import annotations

import math

import pytest
import torch

from tests import bounded_ref as ref

pytestmark = pytest.mark.gpu


def table(max_pos, rot):
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    a = torch.arange(max_pos, dtype=torch.float64)[:, None] * inv
    return torch.cat([a.cos(), a.sin()], 1).float()


def make(T, hq, hkv, d, rot, seed, fused=True, max_pos=500, fp8=False):
    g = torch.Generator().manual_seed(seed)
    if fused:  # parts of one projection
        x = torch.randn(T, (hq + 2 * hkv) * d, generator=g).bfloat16().cuda()
        q = x[:, :hq * d].unflatten(1, (hq, d))
        k = x[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d))
        v = x[:, (hq + hkv) * d:].unflatten(1, (hkv, d))
    else:
        q, k, v = (torch.randn(T, h, d, generator=g).bfloat16().cuda() for h in (hq, hkv, hkv))
    blocks = T // 8 + 2
    shape = (blocks, hkv, 16, d)
    if fp8:
        caches = [torch.randint(0, 255, shape, generator=g, dtype=torch.uint8).cuda() for _ in "kv"]
    else:
        caches = [torch.randn(shape, generator=g).bfloat16().cuda() for _ in "kv"]
    return {"q": q, "k": k, "v": v, "kc": caches[0], "vc": caches[1],
            "pos": torch.randint(0, max_pos, (T,), generator=g).int(),
            "cs": table(max_pos, rot) if rot else None,
            "slots": torch.randperm(blocks * 16, generator=g)[:T],
            "qw": (1 + 0.2 * torch.randn(d, generator=g)).bfloat16(),
            "kw": (1 + 0.2 * torch.randn(d, generator=g)).bfloat16()}


def pair_size(y, rot, interleaved):
    """|a| + |b| of every element's pair (itself where it is not turned)."""
    half, z = rot // 2, y.abs()
    out = z.clone()
    i = torch.arange(half)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    out[..., a] = out[..., b] = z[..., a] + z[..., b]
    return out


def check(s, out, before, rot, interleaved, norm, eps=1e-6, scales=None, live=None):
    from paged_kv_cache_42_gb300 import binding
    assert binding.get_device_error(True)[0] == 0
    T = s["q"].shape[0]
    live = torch.ones(T, dtype=torch.bool) if live is None else live
    cs = s["cs"]
    for name, x, w, got in (("q", s["q"], s["qw"], None), ("k", s["k"], s["kw"], s["kc"]),
                            ("v", s["v"], None, s["vc"])):
        x = x.cpu()
        if name == "v":
            want = x.double()
            slack = torch.zeros_like(want)
        else:
            w = w if norm else None
            plain = ref.norm_rope(x, w, eps, None, None, interleaved)
            want = ref.norm_rope(x, w, eps, cs, s["pos"].clamp(min=0), interleaved)
            slack = pair_size(plain, rot, interleaved) * 2.0 ** -18
        if got is None:
            have = out.cpu().double()
            err, tol = (have - want).abs(), want.abs() * 2.0 ** -8 + slack
            assert (err <= tol)[live].all(), (name, (err - tol)[live].max())
            continue
        rows = got.cpu().transpose(1, 2).flatten(0, 1)
        old = before[name].transpose(1, 2).flatten(0, 1)
        slots = s["slots"][live]
        have = ref.values(rows[slots])
        if scales is not None:
            sc = scales[0 if name == "k" else 1]
            want, slack = want / sc, slack / sc
            tol = torch.maximum(want.abs() * 2.0 ** -4, torch.tensor(2.0 ** -10)) + slack * 1.1
            want = want.clamp(-448, 448)
        else:
            tol = want.abs() * 2.0 ** -8 + slack
        assert ((have - want[live]).abs() <= tol[live]).all(), name
        rest = torch.ones(len(rows), dtype=torch.bool)
        rest[slots] = False
        assert torch.equal(rows[rest].view(torch.uint8), old[rest].view(torch.uint8)), name


CASES = [  # T, hq, hkv, d, rot, interleaved, norm, fused
    (1, 4, 2, 64, 64, False, True, True), (4, 4, 2, 64, 64, False, True, True),
    (7, 32, 8, 128, 128, False, True, True), (65, 32, 8, 128, 128, True, True, True),
    (33, 8, 8, 64, 32, False, True, False), (33, 8, 1, 128, 64, True, False, False),
    (17, 1, 1, 128, 16, False, True, True), (19, 5, 3, 128, 96, False, True, True),
    (19, 5, 3, 64, 48, True, True, True), (50, 16, 4, 128, 0, False, True, True),
    (300, 64, 8, 128, 128, False, False, True),
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,hq,hkv,d,rot,inter,norm,fused", CASES)
def test_against_formula(pa_lib, T, hq, hkv, d, rot, inter, norm, fused, fp8):
    from paged_kv_cache_42_gb300 import binding
    s = make(T, hq, hkv, d, rot, 100 * T + hq, fused, fp8=fp8)
    before = {"k": s["kc"].cpu(), "v": s["vc"].cpu()}
    pos, cs = (s["pos"].cuda(), s["cs"].cuda()) if rot else (None, None)
    kw = {"q_weight": s["qw"].cuda() if norm else None,
          "k_weight": s["kw"].cuda() if norm else None, "interleaved": inter}
    args = (s["q"], s["k"], s["v"], pos, cs, s["slots"].cuda(), s["kc"], s["vc"])
    scales = (0.0113, 0.0127) if fp8 else None
    out = binding.norm_rope_write_kv_fp8(*args, *scales, **kw) if fp8 else \
        binding.norm_rope_write_kv(*args, **kw)
    torch.cuda.synchronize()
    if not rot:
        s["pos"] = torch.zeros(T, dtype=torch.int32)
    check(s, out, before, rot, inter, norm, scales=scales)


def test_padding_and_bad_tokens_are_skipped_whole(pa_lib):
    from paged_kv_cache_42_gb300 import binding
    binding.get_device_error(True)
    T = 40
    s = make(T, 8, 2, 128, 128, 5)
    live = torch.ones(T, dtype=torch.bool)
    s["slots"][3], s["pos"][3] = -1, 10 ** 9  # a padding token's position is nothing
    live[3] = False
    before = {"k": s["kc"].cpu(), "v": s["vc"].cpu()}
    out = torch.full((T, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    kw = {"q_weight": s["qw"].cuda(), "k_weight": s["kw"].cuda(), "out": out}

    def call():
        binding.norm_rope_write_kv(s["q"], s["k"], s["v"], s["pos"].cuda(), s["cs"].cuda(),
                                   s["slots"].cuda(), s["kc"], s["vc"], **kw)
        return binding.get_device_error(True)

    assert call()[0] == 0
    s["pos"][3] = 0
    check(s, out, before, 128, False, True, live=live)
    assert (out[3] == 7).all()
    # a position past the table, then a slot past the pool: reported, nothing written
    for what, bad in (("pos", 500), ("pos", -1), ("slots", s["kc"].shape[0] * 16)):
        old = s[what][9].item()
        s[what][9] = bad
        out.fill_(7.0)
        k0 = s["kc"].clone()
        code, detail = call()
        assert (binding.DEVICE_ERRORS[code].startswith("position" if what == "pos" else "slot")
                and detail == 9)
        assert (out[9] == 7).all() and (out[8] != 7).any()
        assert torch.equal(k0.view(torch.int16), s["kc"].view(torch.int16))
        s[what][9] = old


def test_in_place_other_stream_and_zero_rows(pa_lib):
    from paged_kv_cache_42_gb300 import binding
    s = make(20, 8, 2, 64, 64, 6, fused=False)
    s["q"][4] = 0  # a zero head stays zero: eps keeps the root finite
    before = {"k": s["kc"].cpu(), "v": s["vc"].cpu()}
    q0 = s["q"].clone()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    pos, cs, sl, qw, kw = (s[n].cuda() for n in ("pos", "cs", "slots", "qw", "kw"))
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        out = binding.norm_rope_write_kv(s["q"], s["k"], s["v"], pos, cs, sl, s["kc"], s["vc"],
                                         q_weight=qw, k_weight=kw, out=s["q"])
    st.synchronize()
    assert out.data_ptr() == s["q"].data_ptr() and (out[4] == 0).all()
    s["q"] = q0
    check(s, out, before, 64, False, True)


def test_captured_step_replays(pa_lib):
    """The write and attention of one step, captured, replayed on new inputs."""
    from paged_kv_cache_42_gb300 import binding
    b = ref.Batch([(40, 1), (7, 1), (130, 1)], 8, 2, 128, 9)
    g = b.gpu()
    T = 3
    slots = torch.tensor([int(b.tables[r, (L - 1) // 16]) * 16 + (L - 1) % 16
                          for r, L in enumerate(b.seq_lens.tolist())]).cuda()
    pos = (g["seq_lens"] - 1).int()
    cs = table(256, 128).cuda()
    gen = torch.Generator().manual_seed(1)
    qkv = torch.randn(2, T, 12 * 128, generator=gen).bfloat16().cuda()
    x = torch.empty(T, 12 * 128, dtype=torch.bfloat16, device="cuda")
    q, k, v = (x[:, a * 128:e * 128].unflatten(1, (-1, 128)) for a, e in ((0, 8), (8, 10), (10, 12)))
    qo, out = torch.empty(T, 8, 128, dtype=torch.bfloat16, device="cuda"), None
    out = torch.empty_like(qo)
    ws = torch.empty(binding.workspace_size(3, T, 8, 2, 128), dtype=torch.uint8, device="cuda")

    def step():
        binding.norm_rope_write_kv(q, k, v, pos, cs, slots, g["k"], g["v"], out=qo)
        binding.attention(qo, g["k"], g["v"], g["tables"], g["seq_lens"], g["qsl"], b.scale,
                          max_query_len=1, max_seq_len=b.max_len, out=out, workspace=ws)

    want = []
    for i in range(2):
        x.copy_(qkv[i])
        step()
        torch.cuda.synchronize()
        want.append((qo.clone(), out.clone()))
        kc = g["k"].cpu()
        full = ref.window_attention(qo.cpu(), kc, g["v"].cpu(), b.tables, b.seq_lens, b.qsl,
                                    b.scale, 10 ** 6, 0)
        assert (out.cpu().double() - full).abs().max() < 2e-2
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(2):
        x.copy_(qkv[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(qo, want[i][0]) and torch.equal(out, want[i][1])
    assert binding.get_device_error(True)[0] == 0


def test_refused_tensors(pa_lib):
    from paged_kv_cache_42_gb300 import binding
    s = make(6, 4, 2, 64, 64, 7)
    pos, cs, sl = s["pos"].cuda(), s["cs"].cuda(), s["slots"].cuda()
    good = [s["q"], s["k"], s["v"], pos, cs, sl, s["kc"], s["vc"]]
    for i, bad, exc in ((0, s["q"].transpose(1, 2), ValueError), (0, s["q"].float(), TypeError),
                        (1, s["k"][:, :1], ValueError), (3, pos.long(), TypeError),
                        (3, None, ValueError), (4, cs.double(), TypeError),
                        (5, sl[:5], ValueError), (6, s["kc"].float(), TypeError),
                        (0, s["q"].cpu(), ValueError)):
        args = list(good)
        args[i] = bad
        with pytest.raises(exc):
            binding.norm_rope_write_kv(*args)
    with pytest.raises(ValueError):
        binding.norm_rope_write_kv(*good, q_weight=cs[0].bfloat16()[:32])
    with pytest.raises(binding.PagedAttentionError):
        binding.norm_rope_write_kv(*good, eps=math.nan)
    with pytest.raises(binding.PagedAttentionError):  # 24 is not a multiple of 16
        binding.norm_rope_write_kv(*good[:4], cs[:, :24].contiguous(), *good[5:])
