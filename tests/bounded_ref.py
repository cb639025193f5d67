"""Plain 64-bit implementations of the bounded-cache operators, for the tests:
request by request, on dense K and V gathered through the block table.

Inputs are torch CPU tensors; bf16 and E4M3 caches are read as the values they
hold. Nothing here is shared with the library."""
from __future__ import annotations

import math

import torch


def values(cache: torch.Tensor, scale: float = 1.0) -> torch.Tensor:
    """A cache's values in 64 bits (uint8: E4M3 codes times the scale)."""
    if cache.dtype == torch.uint8:
        return cache.view(torch.float8_e4m3fn).float().double() * scale
    return cache.double()


def dense(cache64: torch.Tensor, table: torch.Tensor, n: int) -> torch.Tensor:
    """[n, Hkv, D] of the first n positions of one request."""
    ids = table[:(n + 15) // 16].long()
    x = cache64[ids].transpose(1, 2)
    return x.reshape(-1, x.shape[2], x.shape[3])[:n]


def norm_rope(x, w, eps, cs, pos, interleaved):
    """[T, H, D] in 64 bits: x / rms * w, pairs turned by cs[pos]."""
    y = x.double()
    if w is not None:
        y = y / (y.pow(2).mean(-1, keepdim=True) + eps).sqrt() * w.double()
    if cs is None:
        return y
    half = cs.shape[1] // 2
    c = cs.double()[pos.long()][:, None, :half]
    s = cs.double()[pos.long()][:, None, half:]
    out = y.clone()
    i = torch.arange(half)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    out[..., a] = y[..., a] * c - y[..., b] * s
    out[..., b] = y[..., b] * c + y[..., a] * s
    return out


def visible(ctx, qlen, window=None, sinks=0):
    """[qlen, ctx + qlen]: which keys the new tokens see."""
    p = torch.arange(ctx, ctx + qlen)[:, None]
    k = torch.arange(ctx + qlen)[None]
    see = k <= p
    if window is not None:
        see = see & ((k > p - window) | (k < sinks))
    return see


def softmax_rows(q, k, scale, see):
    """[qlen, Hq, L] weights; q [qlen, Hq, D], k [L, Hkv, D] in 64 bits."""
    G = q.shape[1] // k.shape[1]
    s = torch.einsum("qhd,khd->qhk", q.double(), k.repeat_interleave(G, 1)) * scale
    s = s.masked_fill(~see[:, None], -math.inf)
    return torch.softmax(s, -1)


def window_attention(q, kc, vc, tables, seq_lens, qsl, scale, window, sinks, k_scale=1.0,
                     v_scale=1.0):
    """[T, Hq, D]; rows of no request are NaN."""
    out = torch.full(q.shape, math.nan, dtype=torch.float64)
    k64, v64 = values(kc, k_scale), values(vc, v_scale)
    for r in range(len(seq_lens)):
        a, b, L = int(qsl[r]), int(qsl[r + 1]), int(seq_lens[r])
        if a == b:
            continue
        see = visible(L - (b - a), b - a, window, sinks)
        any_row = see.any(0)  # keys no row sees may hold anything
        k, v = dense(k64, tables[r], L), dense(v64, tables[r], L)
        k = torch.where(any_row[:, None, None], k, 0.0)
        v = torch.where(any_row[:, None, None], v, 0.0)
        p = softmax_rows(q[a:b], k, scale, see)
        G = q.shape[1] // k.shape[1]
        out[a:b] = torch.einsum("qhk,khd->qhd", p, v.repeat_interleave(G, 1))
    return out


def attention_weights(q, kc, tables, seq_lens, qsl, scale, weights, out, k_scale=1.0):
    """out [R, Hkv, width] in 64 bits with the step's weights added."""
    out = out.double().clone()
    k64 = values(kc, k_scale)
    hkv = kc.shape[1]
    for r in range(len(seq_lens)):
        a, b, L = int(qsl[r]), int(qsl[r + 1]), int(seq_lens[r])
        if a == b:
            continue
        ctx = L - (b - a)
        p = softmax_rows(q[a:b], dense(k64, tables[r], L), scale, visible(ctx, b - a))
        got = p.sum(0).view(hkv, -1, L).sum(1)
        old = weights[r, :, :L].double().clone()
        old[:, ctx:] = 0
        out[r, :, :L] = old + got
    return out


def evict(weights, seq_lens, keep, recent, sinks):
    """(new lengths, {(r, h): kept positions}) by sorting (-weight, position)."""
    lens, kept = [], {}
    for r, L in enumerate(int(x) for x in seq_lens):
        lens.append(min(L, keep))
        if L <= keep:
            continue
        for h in range(weights.shape[1]):
            w = [float(x) for x in weights[r, h, :L]]
            mid = sorted(range(sinks, L - recent),
                         key=lambda i: (-(w[i] if w[i] == w[i] else -math.inf), w[i] != w[i], i))
            mid = sorted(mid[:keep - sinks - recent])
            kept[r, h] = list(range(sinks)) + mid + list(range(L - recent, L))
    return lens, kept


class Batch:
    """A paged batch on CPU: permuted blocks, NaN in every slot that no request
    holds (E4M3: the NaN code)."""

    def __init__(self, spans, hq, hkv, d, seed, fp8=False, pad_blocks=0, extra_blocks=0,
                 q_scale=1.0, trailing_tokens=0):
        g = torch.Generator().manual_seed(seed)
        self.spans, self.hq, self.hkv, self.d, self.fp8 = spans, hq, hkv, d, fp8
        lens = [c + n for c, n in spans]
        nb = [(x + 15) // 16 for x in lens]
        blocks = sum(nb) + extra_blocks + 3
        perm = torch.randperm(blocks, generator=g).int()
        self.mb = max(nb + [1]) + pad_blocks
        self.tables = torch.full((len(spans), self.mb), -1, dtype=torch.int32)
        at = 0
        for r, n in enumerate(nb):
            self.tables[r, :n] = perm[at:at + n]
            at += n
        self.free = perm[at:at + extra_blocks]
        self.seq_lens = torch.tensor(lens, dtype=torch.int32)
        self.qsl = torch.tensor([0] + [n for _, n in spans]).cumsum(0).int()
        T = int(self.qsl[-1]) + trailing_tokens
        self.q = (torch.randn(T, hq, d, generator=g) * q_scale).bfloat16()
        self.k_scale, self.v_scale = (0.0113, 0.0127) if fp8 else (1.0, 1.0)
        shape = (blocks, hkv, 16, d)

        def cache(scale):
            x = torch.randn(shape, generator=g)
            if fp8:
                return (x / scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            return x.bfloat16()

        self.k, self.v = cache(self.k_scale), cache(self.v_scale)
        held = torch.zeros(blocks * 16, dtype=torch.bool)
        for r, L in enumerate(lens):
            p = torch.arange(L)
            held[self.tables[r].long()[p // 16] * 16 + p % 16] = True
        hole = ~held.view(blocks, 1, 16, 1)
        for c in (self.k, self.v):
            c.masked_fill_(hole.expand(shape), 0x7f if fp8 else math.nan)
        self.max_q = max([n for _, n in spans] + [0])
        self.max_len = max(lens + [0])
        self.scale = 1.0 / math.sqrt(d)

    def gpu(self):
        names = ("tables", "seq_lens", "qsl", "q", "k", "v", "free")
        return {n: getattr(self, n).cuda() for n in names}
