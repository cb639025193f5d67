"""pa_norm_rope_write_kv: the elements past rotary_dim stay what they are, and
the kernel variant of large batches.

An element that is neither normalised nor turned is not computed at all: its
bits stay, whatever stands beside it. The other tolerances are those of
tests/test_gpu_norm_rope.py."""
from __future__ import annotations

import pytest
import torch

from tests import bounded_ref as ref
from tests import test_gpu_norm_rope as tn

pytestmark = pytest.mark.gpu

ODD = torch.tensor([0x7f80, 0xff80, 0x7fc0, 0xffc1, 0x7f81, 0x8000, 0x0001, 0x7f7f]).to(torch.int16)


def write(s, fp8=False, norm=False, inter=False, eps=1e-6):
    from paged_kv_cache_42_gb300 import binding
    pos, cs = (s["pos"].cuda(), s["cs"].cuda()) if s["cs"] is not None else (None, None)
    kw = {"q_weight": s["qw"].cuda() if norm else None,
          "k_weight": s["kw"].cuda() if norm else None, "interleaved": inter, "eps": eps}
    args = (s["q"], s["k"], s["v"], pos, cs, s["slots"].cuda(), s["kc"], s["vc"])
    out = binding.norm_rope_write_kv_fp8(*args, 0.0113, 0.0127, **kw) if fp8 else \
        binding.norm_rope_write_kv(*args, **kw)
    torch.cuda.synchronize()
    return out


@pytest.mark.parametrize("T", [5, 1200])  # both kernel variants
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("d,rot", [(64, 0), (64, 16), (64, 48), (128, 0), (128, 64), (128, 112)])
def test_elements_past_rotary_dim_keep_their_bits(pa_lib, d, rot, inter, T):
    """Infinities, NaN of any payload, minus zero and the smallest and largest
    numbers among them: every one stays, and none reaches another element."""
    s = tn.make(T, 8, 2, d, rot, 7 * T + d + rot)
    g = torch.Generator().manual_seed(rot)
    for n in "qk":
        x = s[n].view(torch.int16)
        odd = ODD[torch.randint(0, len(ODD), x.shape, generator=g)].cuda()
        pick = (torch.rand(x.shape, generator=g) < 0.2).cuda()
        pick[..., :rot] = False
        x.copy_(torch.where(pick, odd, x))
    before = {n: s[n].cpu().clone() for n in "qk"}
    out = write(s, inter=inter)
    rows = s["kc"].cpu().transpose(1, 2).flatten(0, 1)[s["slots"]]
    for n, got in (("q", out.cpu()), ("k", rows)):
        assert torch.equal(got[..., rot:].view(torch.int16), before[n][..., rot:].view(torch.int16))
        if rot:
            want = ref.norm_rope(before[n][..., :rot], None, 0.0, s["cs"], s["pos"], inter)
            slack = tn.pair_size(before[n][..., :rot].double(), rot, inter) * 2.0 ** -18
            err = (got[..., :rot].double() - want).abs()
            assert (err <= want.abs() * 2.0 ** -8 + slack).all()


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("inter", [False, True])
def test_non_finite_past_rotary_dim_e4m3(pa_lib, inter, norm):
    """Over an E4M3 cache they saturate or become its NaN, as in pa_write_kv_fp8;
    under the norm only that head is lost."""
    from paged_kv_cache_42_gb300 import binding
    s = tn.make(9, 4, 2, 128, 64, 3, fp8=True)
    bad = [(1, 0, 70, float("inf")), (4, 1, 127, -float("inf")), (6, 0, 64, float("nan"))]
    clean = {n: s[n].clone() for n in "qkv"}
    for t, h, e, x in bad:
        s["k"][t, h, e] = x
    write(s, fp8=True, norm=norm, inter=inter)
    got = s["kc"].cpu().transpose(1, 2).flatten(0, 1)[s["slots"]]
    plain_k, plain_v = torch.zeros_like(s["kc"]), torch.zeros_like(s["vc"])
    binding.write_kv_fp8(s["k"].contiguous(), s["v"].contiguous(), s["slots"].cuda(), plain_k,
                         plain_v, 0.0113, 0.0127)
    plain = plain_k.cpu().transpose(1, 2).flatten(0, 1)[s["slots"]]
    for n in "qkv":
        s[n].copy_(clean[n])
    write(s, fp8=True, norm=norm, inter=inter)
    want = s["kc"].cpu().transpose(1, 2).flatten(0, 1)[s["slots"]]
    for t, h, e, _ in bad:
        if norm:
            want[t, h] = got[t, h]
        else:
            want[t, h, e] = plain[t, h, e]
    assert torch.equal(got, want)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,hq,hkv,d,rot,inter,norm", [
    (1500, 32, 8, 128, 128, False, True), (1500, 32, 8, 128, 128, True, True),
    (1500, 5, 3, 128, 96, False, True), (1500, 5, 3, 128, 96, True, True),
    (2300, 5, 3, 64, 48, False, True), (2300, 5, 3, 64, 64, True, True),
    (1500, 32, 8, 64, 32, False, True), (5000, 1, 1, 64, 64, False, True),
    (1300, 17, 1, 128, 0, False, True), (1300, 9, 9, 64, 16, True, False)])
def test_many_tokens(pa_lib, T, hq, hkv, d, rot, inter, norm, fp8):
    """Batches that take four groups of heads per warp (more than eight CTAs per
    SM of one): the norm's sums past the last head, ragged last units."""
    s = tn.make(T, hq, hkv, d, rot, T + hq + d, fp8=fp8)
    before = {"k": s["kc"].cpu(), "v": s["vc"].cpu()}
    out = write(s, fp8, norm, inter)
    if not rot:
        s["pos"] = torch.zeros(T, dtype=torch.int32)
    tn.check(s, out, before, rot, inter, norm, scales=(0.0113, 0.0127) if fp8 else None)
