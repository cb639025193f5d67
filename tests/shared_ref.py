"""Batches whose groups of requests share prefixes, on CPU, in every cache format; the
reference is plain attention, request by request (tests/rows_ref.py)."""
from __future__ import annotations

import math

import torch

from tests import bounded_ref as ref
from tests import rows_ref as rr


class Batch:
    """groups: [(prefix length, [(own context, new tokens), ...]), ...]: a member's context is
    the prefix and `own context` keys behind it; a negative own context takes that many keys
    off the prefix, and the request has blocks of its own only. before, after: requests of
    no group."""

    def __init__(self, groups, hq, hkv, d, seed, fmt="bf16", before=(), after=(), trailing_tokens=0):
        g = torch.Generator().manual_seed(seed)
        self.hq, self.hkv, self.d, self.fmt, self.groups = hq, hkv, d, fmt, groups
        reqs = [(None, 0, c, n) for c, n in before]
        loc = [len(reqs)]
        for i, (p, members) in enumerate(groups):
            reqs += [(i if c >= 0 else None, p, p + c, n) for c, n in members]
            loc.append(len(reqs))
        reqs += [(None, 0, c, n) for c, n in after]
        self.group_loc = torch.tensor(loc, dtype=torch.int32)
        self.prefix = torch.tensor([p for p, _ in groups], dtype=torch.int32)
        self.max_prefix = max([p for p, _ in groups] + [0])
        self.spans = [(c, n) for _, _, c, n in reqs]
        lens = [c + n for c, n in self.spans]
        self.mb = max([(x + 15) // 16 for x in lens] + [1]) + 1
        total = sum((x + 15) // 16 for x in lens) + sum(p // 16 for p, _ in groups) + 3
        perm = torch.randperm(total, generator=g).int()
        self.tables = torch.full((len(reqs), self.mb), -1, dtype=torch.int32)
        at, prefix_blocks = 0, {}
        for r, (grp, p, c, n) in enumerate(reqs):
            k = 0
            if grp is not None:
                if grp not in prefix_blocks:
                    prefix_blocks[grp] = perm[at:at + p // 16]
                    at += p // 16
                k = p // 16
                self.tables[r, :k] = prefix_blocks[grp]
            m = (lens[r] + 15) // 16 - k
            self.tables[r, k:k + m] = perm[at:at + m]
            at += m
        self.seq_lens = torch.tensor(lens, dtype=torch.int32)
        self.qsl = torch.tensor([0] + [n for _, n in self.spans]).cumsum(0).int()
        T = int(self.qsl[-1]) + trailing_tokens
        self.q = torch.randn(T, hq, d, generator=g).bfloat16()
        self.max_q = max([n for _, n in self.spans] + [0])
        self.max_len = max(lens + [0])
        self.scale = 1 / math.sqrt(d)
        self.k_scale, self.v_scale = 0.0113, 0.0127
        held = torch.zeros(total * 16, dtype=torch.bool)
        for r, L in enumerate(lens):
            pos = torch.arange(L)
            held[self.tables[r].long()[pos // 16] * 16 + pos % 16] = True
        hole = ~held.view(total, 1, 16, 1)
        shape = (total, hkv, 16, d)
        self.scales = torch.full((total, hkv, 2, 16), 255, dtype=torch.uint8)
        for i, name in enumerate(("k", "v")):
            x = torch.randn(shape, generator=g)
            if fmt == "rows":
                size = torch.exp2((torch.rand(shape[:3], generator=g) - 0.5) * 4)
                c, by = rr.quantise_fast((x * size[..., None]).bfloat16().float())
                self.scales[:, :, i] = torch.where(hole[..., 0].expand(shape[:3]), 255, by)
                c = c.masked_fill(hole.expand(shape), 0x7f)
                val = rr.values(c, self.scales[:, :, i])
            elif fmt == "fp8":
                s = (self.k_scale, self.v_scale)[i]
                c = (x / s).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
                c = c.masked_fill(hole.expand(shape), 0x7f)
                val = ref.values(c, float(torch.tensor(s)))
            else:
                c = x.bfloat16().masked_fill(hole.expand(shape), math.nan)
                val = c.double()
            setattr(self, name, c)
            setattr(self, name + "64", val)

    def want(self):
        return rr.attention(self, self.k64, self.v64)

    def gpu(self):
        names = ("tables", "seq_lens", "qsl", "q", "k", "v", "scales", "group_loc", "prefix")
        return {n: getattr(self, n).cuda() for n in names}

    def run(self, g, **kw):
        """attention_shared[_fp8, _rows] on a gpu() dictionary."""
        from paged_kv_cache_42_gb300 import binding
        kw = {"max_prefix_len": self.max_prefix, "max_query_len": self.max_q,
              "max_seq_len": self.max_len, **kw}
        meta = (g["tables"], g["seq_lens"], g["qsl"], g["group_loc"], g["prefix"], self.scale)
        if self.fmt == "rows":
            return binding.attention_shared_rows(g["q"], g["k"], g["v"], g["scales"], *meta, **kw)
        if self.fmt == "fp8":
            return binding.attention_shared_fp8(g["q"], g["k"], g["v"], *meta, self.k_scale,
                                                self.v_scale, **kw)
        return binding.attention_shared(g["q"], g["k"], g["v"], *meta, **kw)

    def plain(self, g, **kw):
        """The same by attention[_fp8, _rows]."""
        from paged_kv_cache_42_gb300 import binding
        kw = {"max_query_len": self.max_q, "max_seq_len": self.max_len, **kw}
        meta = (g["tables"], g["seq_lens"], g["qsl"], self.scale)
        if self.fmt == "rows":
            return binding.attention_rows(g["q"], g["k"], g["v"], g["scales"], *meta, **kw)
        if self.fmt == "fp8":
            return binding.attention_fp8(g["q"], g["k"], g["v"], *meta, self.k_scale, self.v_scale, **kw)
        return binding.attention(g["q"], g["k"], g["v"], *meta, **kw)
