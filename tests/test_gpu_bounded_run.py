"""The bounded-cache operators together, as a serving loop uses them.

Two requests with different prompts: each prompt chunk and decode goes through
norm + rotation + write, attention (windowed, and over everything), and the
accumulated weights; when a cache passes the high-water mark it is cut, its old
blocks go back to the pool, and decoding continues at the rotations of the true
positions. A 64-bit model beside it keeps each (request, head)'s keys and values
in dense lists and is compared at every step."""
from __future__ import annotations

import math

import pytest
import torch

from tests import bounded_ref as ref

pytestmark = pytest.mark.gpu

HQ, HKV, D, BLOCKS, SCALE = 8, 2, 64, 64, 1 / 8.0
KEEP, RECENT, SINKS, HIGH, WIDTH, WINDOW = 40, 16, 4, 56, 128, 24


def table(n):
    inv = 10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)
    a = torch.arange(n, dtype=torch.float64)[:, None] * inv
    return torch.cat([a.cos(), a.sin()], 1).float()


@pytest.mark.parametrize("fp8", [False, True])
def test_serving_loop(pa_lib, fp8):
    from paged_kv_cache_42_gb300 import binding, host
    binding.get_device_error(True)
    gen = torch.Generator().manual_seed(7)
    pool = host.BlockPool(BLOCKS)
    dtype = torch.uint8 if fp8 else torch.bfloat16
    ks, vs = (0.0113, 0.0127) if fp8 else (1.0, 1.0)
    kc = torch.zeros(BLOCKS, HKV, 16, D, dtype=dtype, device="cuda")
    vc = torch.zeros_like(kc)
    cs = table(512).cuda()
    qw, kw = ((1 + 0.1 * torch.randn(D, generator=gen)).bfloat16().cuda() for _ in "qk")
    blocks = [[], []]      # physical blocks of each request
    length, place = [0, 0], [0, 0]   # cached tokens, true position of the next one
    keys = [[[] for _ in range(HKV)] for _ in range(2)]  # the model: 64-bit rows, as stored
    vals = [[[] for _ in range(HKV)] for _ in range(2)]
    w = torch.zeros(2, HKV, WIDTH, device="cuda")
    w64 = [[[] for _ in range(HKV)] for _ in range(2)]

    def tables():
        t = torch.full((2, WIDTH // 16), -1, dtype=torch.int32)
        for r in range(2):
            t[r, :len(blocks[r])] = torch.tensor(blocks[r], dtype=torch.int32)
        return t.cuda()

    def step(new):
        T, qsl, pos, slots = sum(new), [0], [], []
        for r in range(2):
            while len(blocks[r]) * 16 < length[r] + new[r]:
                blocks[r] += [int(b) for b in pool.allocate(1)]
            for j in range(new[r]):
                p = length[r] + j
                slots.append(blocks[r][p // 16] * 16 + p % 16)
                pos.append(place[r] + j)
            length[r] += new[r]
            place[r] += new[r]
            qsl.append(qsl[-1] + new[r])
        x = torch.randn(T, (HQ + 2 * HKV) * D, generator=gen).bfloat16().cuda()
        q, k, v = (x[:, a * D:e * D].unflatten(1, (-1, D))
                   for a, e in ((0, HQ), (HQ, HQ + HKV), (HQ + HKV, HQ + 2 * HKV)))
        pos, slots = torch.tensor(pos, dtype=torch.int32).cuda(), torch.tensor(slots).cuda()
        args = (q, k, v, pos, cs, slots, kc, vc)
        kw_ = dict(q_weight=qw, k_weight=kw)
        qo = binding.norm_rope_write_kv_fp8(*args, ks, vs, **kw_) if fp8 else \
            binding.norm_rope_write_kv(*args, **kw_)
        sl = torch.tensor(length, dtype=torch.int32).cuda()
        ql = torch.tensor(qsl, dtype=torch.int32).cuda()
        t = tables()
        m = dict(max_query_len=max(new), max_seq_len=max(length))
        head = (qo, kc, vc, t, sl, ql, SCALE)
        # one of the two windows holds everything
        outs = [(binding.attention_window_fp8(*head, ks, vs, window=n, sinks=SINKS, **m) if fp8 else
                 binding.attention_window(*head, window=n, sinks=SINKS, **m)) for n in (WINDOW, 512)]
        (binding.attention_weights_fp8(qo, kc, t, sl, ql, SCALE, ks, w, **m) if fp8 else
         binding.attention_weights(qo, kc, t, sl, ql, SCALE, w, **m))
        torch.cuda.synchronize()
        # the model: what the slots now hold, then the step in 64 bits
        kd = ref.values(kc.cpu(), ks).transpose(1, 2).flatten(0, 1)
        vd = ref.values(vc.cpu(), vs).transpose(1, 2).flatten(0, 1)
        want_k = ref.norm_rope(k.cpu(), kw.cpu(), 1e-6, cs.cpu(), pos.cpu(), False)
        step_of = 2.0 ** (-4 if fp8 else -8)
        assert ((kd[slots.cpu()] - want_k).abs() <= want_k.abs() * step_of + ks * 2.0 ** -10 + 1e-4).all()
        for r in range(2):
            for j in range(new[r]):
                for h in range(HKV):
                    keys[r][h].append(kd[slots[qsl[r] + j], h])
                    vals[r][h].append(vd[slots[qsl[r] + j], h])
            if not new[r]:
                continue
            q64 = qo[qsl[r]:qsl[r + 1]].cpu().double()
            see = [ref.visible(length[r] - new[r], new[r], n, SINKS) for n in (WINDOW, None)]
            for h in range(HKV):
                K, V = torch.stack(keys[r][h]), torch.stack(vals[r][h])
                qh = q64[:, h * 4:h * 4 + 4]
                s = torch.einsum("qgd,kd->qgk", qh, K) * SCALE
                for o, vis in zip(outs, see):
                    p = torch.softmax(s.masked_fill(~vis[:, None], -math.inf), -1)
                    want = torch.einsum("qgk,kd->qgd", p, V)
                    size = torch.einsum("qgk,kd->qgd", p, V.abs())
                    got = o[qsl[r]:qsl[r + 1], h * 4:h * 4 + 4].cpu().double()
                    tol = want.abs() * 2.0 ** -8 + size * 2.0 ** -7 + V.abs().max() * 2.0 ** -12
                    assert ((got - want).abs() <= tol).all()
                got = p.sum((0, 1))  # the last one saw everything
                old = w64[r][h] + [0.0] * new[r]
                w64[r][h] = [a + float(b) for a, b in zip(old, got)]
                have = w[r, h, :length[r]].cpu().double()
                want = torch.tensor(w64[r][h], dtype=torch.float64)
                assert ((have - want).abs() <= want * 2.0 ** -16 * 64).all()  # up to 64 steps' sums

    def cut():
        if max(length) <= HIGH:
            return False
        sl = torch.tensor(length, dtype=torch.int32).cuda()
        fresh = [[int(b) for b in pool.allocate((KEEP + 15) // 16)] if n > KEEP else [] for n in length]
        nt = torch.tensor([f or [-1] * 3 for f in fresh], dtype=torch.int32).cuda()
        new_w = torch.full((2, HKV, WIDTH), -1.0, device="cuda")
        before = w.clone()
        lens, kept, new_w = binding.evict_kv(kc, vc, tables(), sl, w, nt, keep=KEEP, recent=RECENT,
                                             sinks=SINKS, max_seq_len=max(length), new_weights=new_w)
        torch.cuda.synchronize()
        want_lens, want = ref.evict(before.cpu(), length, KEEP, RECENT, SINKS)
        assert lens.tolist() == want_lens
        for r in range(2):
            if length[r] <= KEEP:
                continue
            for h in range(HKV):
                ids = want[r, h]
                assert kept[r, h].tolist() == ids
                keys[r][h] = [keys[r][h][i] for i in ids]
                vals[r][h] = [vals[r][h][i] for i in ids]
                w64[r][h] = [w64[r][h][i] for i in ids]
            w[r, :, :KEEP] = new_w[r, :, :KEEP]
            pool.release(blocks[r])
            blocks[r], length[r] = fresh[r], KEEP
        return True

    cuts = 0
    step([20, 37])                       # the prompts, one chunk each
    for i in range(30):
        step([1, 1] if i % 3 else [1, 0] if i % 2 else [0, 2])
        cuts += cut()
    step([18, 1])                        # a second turn: a chunk beside a decode
    cuts += cut()
    step([1, 1])
    assert cuts >= 2
    assert binding.get_device_error(True)[0] == 0
