"""Plain 64-bit implementations of the row-scaled cache's operators, for the
tests. Inputs are torch CPU tensors; nothing here is shared with the library."""
from __future__ import annotations

import math

import torch

from tests import bounded_ref as ref

E_MIN, E_MAX = -100, 119
POWERS = torch.tensor([2.0 ** (b - 127) for b in range(255)] + [math.nan], dtype=torch.float64)


def scale_bytes(x: torch.Tensor) -> torch.Tensor:
    """The byte of every row of x [..., D] (any float type, taken exactly)."""
    x = x.double()
    top = x.abs().amax(-1)
    out = torch.empty(top.shape, dtype=torch.uint8)
    for i, row in enumerate(x.reshape(-1, x.shape[-1])):
        a = float(row.abs().max()) if torch.isfinite(row).all() else math.inf
        if not math.isfinite(a):
            b = 255
        else:
            e = E_MIN
            while e < E_MAX and a > 448 * 2.0 ** e:
                e += 1
            b = e + 127
        out.view(-1)[i] = b
    return out


def quantise(x: torch.Tensor):
    """(codes uint8 [..., D], bytes uint8 [...]) of rows x."""
    b = scale_bytes(x)
    size = POWERS[b.long()]
    bad = (b == 255)[..., None]
    y = torch.where(bad, 0.0, x.double() / size[..., None])  # exact: a power of two
    codes = y.clamp(-448, 448).float().to(torch.float8_e4m3fn).view(torch.uint8)
    # -0 of a poisoned row: its codes are +0
    return torch.where(bad, 0, codes).to(torch.uint8), b


def values(codes: torch.Tensor, size_bytes: torch.Tensor) -> torch.Tensor:
    """Rows in 64 bits."""
    return codes.view(torch.float8_e4m3fn).float().double() * POWERS[size_bytes.long()][..., None]


class Batch(ref.Batch):
    """A paged batch over a row-scaled cache on CPU: k and v become codes, scales the
    bytes, and every slot that no request holds NaN codes and a NaN byte. Rows differ in
    size by factors of up to 2^spread."""

    def __init__(self, spans, hq, hkv, d, seed, spread=3.0, **kw):
        super().__init__(spans, hq, hkv, d, seed, **kw)
        g = torch.Generator().manual_seed(seed + 1000)
        self.scales = torch.empty(self.k.shape[0], hkv, 2, 16, dtype=torch.uint8)
        for i, name in enumerate(("k", "v")):
            x = getattr(self, name)
            size = torch.exp2((torch.rand(x.shape[:-1], generator=g) - 0.5) * 2 * spread)
            codes, self.scales[:, :, i] = quantise_fast(x.float() * size[..., None])
            hole = torch.isnan(x[..., 0])
            setattr(self, name, torch.where(hole[..., None], 0x7f, codes).to(torch.uint8))
        self.k64 = values(self.k, self.scales[:, :, 0])
        self.v64 = values(self.v, self.scales[:, :, 1])

    def gpu(self):
        g = super().gpu()
        g["scales"] = self.scales.cuda()
        return g


def quantise_fast(x: torch.Tensor):
    """quantise() of finite rows (or NaN ones) without a loop."""
    top = x.double().abs().amax(-1)
    e = torch.ceil(torch.log2(top / 448)).nan_to_num(0, 0, E_MIN).clamp(E_MIN, E_MAX)
    e = torch.where(top > 448 * POWERS[(e + 127).long()], e + 1, e)
    e = torch.where(top <= 448 * POWERS[(e + 126).long()], e - 1, e).clamp(E_MIN, E_MAX)
    b = torch.where(torch.isfinite(top), e + 127, 255).to(torch.uint8)
    y = (x.double() / POWERS[b.long()][..., None]).nan_to_num(0, 0, 0)
    return y.clamp(-448, 448).float().to(torch.float8_e4m3fn).view(torch.uint8), b


def attention(b, k64, v64):
    """(out, tol) [T, Hq, D] of a batch over dense 64-bit caches; rows of no request are
    NaN. tol: what the kernels may be off by. bf16 output: half a step, 2^-8 of the value.
    Weights on the tensor cores: two E4M3 terms (2^-4 x 2^-4) or one bf16 (2^-8) of each,
    and the query's second term, together below 2^-7 of the sum of weight x |V|; the terms'
    smallest step, 2^-10 of a weight's 256 when the largest weight x size is 2^-3 of that
    at least: 2^-15 of the largest weight x row maximum (row maxima are 224 to 448 sizes,
    codes up to 448: 2^-14) for each key."""
    G = b.hq // b.hkv
    out = torch.full(b.q.shape, math.nan, dtype=torch.float64)
    tol = torch.zeros_like(out)
    for r in range(len(b.spans)):
        a, e, L = int(b.qsl[r]), int(b.qsl[r + 1]), int(b.seq_lens[r])
        if a == e:
            continue
        k, v = ref.dense(k64, b.tables[r], L), ref.dense(v64, b.tables[r], L)
        p = ref.softmax_rows(b.q[a:e], k, b.scale, ref.visible(L - (e - a), e - a))
        v = v.repeat_interleave(G, 1)
        out[a:e] = torch.einsum("qhk,khd->qhd", p, v)
        size = torch.einsum("qhk,khd->qhd", p, v.abs())
        top = (p * v.abs().amax(-1).T).amax(-1)[..., None]
        tol[a:e] = out[a:e].abs() * 2.0 ** -8 + size * 2.0 ** -7 + top * L * 2.0 ** -14
    return out, tol
