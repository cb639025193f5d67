"""Operators around quantised and shared parts of a paged KV cache, measured one call at a time.

Five operators of the library in ``paged_kv_cache_42_gb300``, each in its plain
form (elementary torch operations in 32 bits, rounded once) and as the calls a
serving step makes of ``paged_kv_cache_42_gb300.binding``:

  write      new K and V rows into an E4M3 cache with one power-of-two scale for
             every row, found as it is written (bf16 rows in, codes and scales out)
  normwrite  the same behind the norm of every query and key head and the rotation
  attend     paged attention over such a cache, for decodes and prompt chunks
  read       ranges of cached keys and values as dense bf16 rows
  shared     attention of a batch whose groups of requests share long prefixes,
             over a bf16, an E4M3 (one scale per tensor) or a row-scaled cache

Caches are [num_blocks][kv heads][16][head dim]; a request finds its blocks in
its row of block_tables. A row-scaled cache has ``scales`` beside it, bytes
[num_blocks][kv heads][2][16] (K, then V): b stands for 2^(b - 127), 255 for
NaN. ``own`` chooses the library's calls.
"""
from __future__ import annotations

import math
import random

import torch

own = False

BLOCK = 16
K_SCALE, V_SCALE = 0.0113, 0.0127  # E4M3 caches with one scale per tensor
EPS = 1e-6
E_MIN, E_MAX = -100, 119  # exponents of a row's scale


def listed():
    llama = {"hq": 32, "hkv": 8, "d": 128}
    tiny = {"hq": 4, "hkv": 2, "d": 64}
    wide = {"hq": 64, "hkv": 8, "d": 128}
    return [
        # one token each of four short conversations: the smallest step there is
        {"name": "write tiny decode", "op": "write", **tiny, "tokens": 4},
        # a step of 512 decodes and three prompt chunks: 2048 tokens
        {"name": "write mixed batch", "op": "write", **llama, "tokens": 2048},
        # the newest token of 64 conversations, heads normalised and turned
        {"name": "normwrite decode batch", "op": "normwrite", **llama, "tokens": 64, "norm": True,
         "interleaved": False, "rot": 128, "max_pos": 32768},
        # a whole mixed step of it
        {"name": "normwrite mixed batch", "op": "normwrite", **llama, "tokens": 2048,
         "norm": True, "interleaved": False, "rot": 128, "max_pos": 32768},
        # four short conversations
        {"name": "attend tiny decode", "op": "attend", **tiny, "decodes": 4, "lmin": 9,
         "lmax": 57, "lens_seed": 1, "qlen": 0, "ctx": ""},
        # 64 conversations of 512 to 4096 tokens
        {"name": "attend decode batch", "op": "attend", **llama, "decodes": 64, "lmin": 512,
         "lmax": 4096, "lens_seed": 2, "qlen": 0, "ctx": ""},
        # a mixed step: 512 decodes and three prompt chunks of 512
        {"name": "attend mixed batch", "op": "attend", **llama, "decodes": 512, "lmin": 128,
         "lmax": 2048, "lens_seed": 3, "qlen": 512, "ctx": "0,1024,2048"},
        # the cached part of one short prompt handed to another program
        {"name": "read one prompt", "op": "read", **tiny, "fmt": "bf16", "reqs": 1, "lmin": 100,
         "lmax": 100, "lens_seed": 4, "first": False},
        # 64 conversations moved out of a row-scaled cache, from somewhere inside a block on
        {"name": "read decode batch rows", "op": "read", **llama, "fmt": "rows", "reqs": 64,
         "lmin": 512, "lmax": 4096, "lens_seed": 2, "first": True},
        # two pairs of short conversations behind two short system prompts
        {"name": "shared tiny", "op": "shared", **tiny, "fmt": "bf16", "groups": 2, "mmin": 2,
         "mmax": 2, "pmin": 32, "pmax": 64, "smin": 3, "smax": 40, "alone": 0, "qlen": 1,
         "lens_seed": 6},
        # 128 conversations behind eight system prompts, and eight without one
        {"name": "shared system prompts", "op": "shared", **llama, "fmt": "bf16", "groups": 8,
         "mmin": 8, "mmax": 24, "pmin": 512, "pmax": 2048, "smin": 16, "smax": 512, "alone": 8,
         "qlen": 1, "lens_seed": 7},
        # questions about three long documents, a row-scaled cache
        {"name": "shared documents rows", "op": "shared", **wide, "fmt": "rows", "groups": 3,
         "mmin": 12, "mmax": 20, "pmin": 16384, "pmax": 32768, "smin": 64, "smax": 1024,
         "alone": 0, "qlen": 1, "lens_seed": 8},
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    hkv = rng.choice([1, 2, 4, 8, 8])
    c = {"hq": hkv * rng.choice([1, 2, 4, 8]), "hkv": hkv, "d": rng.choice([64, 128, 128])}
    op = rng.choice(["write", "normwrite", "attend", "attend", "read", "shared", "shared"])
    if op == "write":
        return {"op": op, **c, "tokens": _log(rng, 1, 2048)}
    if op == "normwrite":
        return {"op": op, **c, "tokens": _log(rng, 1, 2048), "norm": rng.random() < 0.75,
                "interleaved": rng.random() < 0.3, "rot": rng.choice([c["d"], c["d"] // 2]),
                "max_pos": _log(rng, 2048, 32768)}
    c["lens_seed"] = rng.randrange(1 << 30)
    if op == "attend":
        lmax = _log(rng, 8, 32768)
        c.update(decodes=_log(rng, 1, max(1, min(256, 262144 // lmax))), lmin=_log(rng, 1, lmax),
                 lmax=lmax, qlen=0, ctx="")
        if rng.random() < 0.4:  # prompt chunks, or short spans, beside the decodes
            c["qlen"] = _log(rng, 2, 512)
            c["ctx"] = ",".join(str(_log(rng, 1, 2048) - 1) for _ in range(rng.randint(1, 3)))
        return {"op": op, **c}
    fmt = rng.choice(["bf16", "fp8", "rows", "rows"])
    if op == "read":
        lmax = _log(rng, 1, 8192)
        return {"op": op, **c, "fmt": fmt, "reqs": _log(rng, 1, max(1, min(256, 131072 // lmax))),
                "lmin": _log(rng, 1, lmax), "lmax": lmax, "first": rng.random() < 0.5}
    pmax = 16 * _log(rng, 1, 1024)
    smax = _log(rng, 1, 1024)
    groups = rng.randint(1, 8)
    mmax = _log(rng, 1, max(1, min(64, 131072 // (groups * (pmax + smax)))))
    return {"op": op, **c, "fmt": fmt, "groups": groups, "mmin": _log(rng, 1, mmax), "mmax": mmax,
            "pmin": 16 * _log(rng, 1, pmax // 16), "pmax": pmax, "smin": _log(rng, 1, smax),
            "smax": smax, "alone": rng.choice([0, 0, 1, 5]), "qlen": rng.choice([1, 1, 1, 2, 4])}


def _spans(case):
    """(context, new tokens) of every request: the decodes, then the chunks."""
    r = random.Random(case["lens_seed"])
    spans = [(r.randint(case["lmin"], case["lmax"]) - 1, 1) for _ in range(case["decodes"])]
    if case["qlen"]:
        spans += [(int(x), case["qlen"]) for x in case["ctx"].split(",")]
    return spans


def _groups(case):
    """Members and prefix length of every group; suffix length of every request, its new
    tokens included (the requests of the groups in turn, then those without a prefix)."""
    r = random.Random(case["lens_seed"])
    members = [r.randint(case["mmin"], case["mmax"]) for _ in range(case["groups"])]
    prefix = [16 * r.randint(case["pmin"] // 16, case["pmax"] // 16) for _ in members]
    n = case["qlen"]
    suffix = [max(n, r.randint(case["smin"], case["smax"]))
              for _ in range(sum(members) + case["alone"])]
    return members, prefix, suffix


def _reads(case):
    """(first key, number of keys, cached keys) of every request."""
    r = random.Random(case["lens_seed"])
    out = []
    for _ in range(case["reqs"]):
        n = r.randint(case["lmin"], case["lmax"])
        first = r.randint(0, 40) if case["first"] else 0
        out.append((first, n, first + n + r.randint(0, 20)))
    return out


def _rows_like(g, blocks, case):
    """Rows as a model leaves them: some of many times the others' size."""
    x = torch.randn(blocks, case["hkv"], BLOCK, case["d"], generator=g, device="cuda")
    size = torch.randn(blocks, case["hkv"], BLOCK, 1, generator=g, device="cuda")
    return x * (0.5 * size).exp()


def _code(x):
    """Rows in 32 bits as E4M3 codes and their scales' bytes."""
    top = x.abs().amax(-1, keepdim=True)
    m, e = torch.frexp(top)
    e = torch.where(top > 0, e - 9 + (m > 0.875), E_MIN).clamp(E_MIN, E_MAX)
    fine = torch.isfinite(top)
    e = torch.where(fine, e, 0)
    # 2^-e in two steps: one factor may pass the largest number
    x = torch.where(fine, x * torch.exp2(-(e // 2).float()) * torch.exp2(-(e - e // 2).float()), 0)
    codes = x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes, torch.where(fine, e + 127, 255).to(torch.uint8).squeeze(-1)


def _size(b):
    """Scale bytes as the numbers they stand for, in 32 bits."""
    return torch.where(b == 255, math.nan, torch.exp2(b.float() - 127))


def _caches(g, blocks, case, s):
    """Filled caches of the case's format into the state."""
    fmt = case.get("fmt", "rows")
    if fmt == "rows":
        s["k_cache"], a = _code(_rows_like(g, blocks, case))
        s["v_cache"], b = _code(_rows_like(g, blocks, case))
        s["scales"] = torch.stack([a, b], 2).contiguous()
        return
    k, v = (torch.randn(blocks, case["hkv"], BLOCK, case["d"], generator=g, device="cuda")
            for _ in range(2))
    if fmt == "bf16":
        s["k_cache"], s["v_cache"] = k.bfloat16(), v.bfloat16()
    else:
        s["k_cache"] = (k / K_SCALE).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        s["v_cache"] = (v / V_SCALE).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def _tables(g, shared, own_blocks):
    """Block tables [R, width] and the number of blocks: request r holds the blocks of
    the run shared[r] (a run's number and length, or None), then own_blocks[r] of its own."""
    runs = {}
    rows, at = [], 0
    for run, n in zip(shared, own_blocks):
        row = []
        if run is not None:
            if run not in runs:
                runs[run] = list(range(at, at + run[1]))
                at += run[1]
            row += runs[run]
        rows.append(row + list(range(at, at + n)))
        at += n
    width = max(len(r) for r in rows)
    ids = torch.tensor([r + [-1] * (width - len(r)) for r in rows], device="cuda")
    perm = torch.randperm(at + 16, generator=g, device="cuda")
    return torch.where(ids >= 0, perm[ids.clamp(min=0)], -1).int(), at + 16


def _loc(counts):
    return torch.tensor([0] + list(counts), device="cuda").cumsum(0).int()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    s = {"case": case, "scale": 1.0 / math.sqrt(d)}
    if case["op"] in ("write", "normwrite"):
        T = case["tokens"]
        # q, k and v side by side, as one projection leaves them
        qkv = torch.randn(T, (hq + 2 * hkv) * d, generator=g, device="cuda", dtype=torch.bfloat16)
        qkv *= torch.randn(T, 1, generator=g, device="cuda").mul(0.5).exp().bfloat16()
        s["q"] = qkv[:, :hq * d].unflatten(1, (hq, d))
        s["k"] = qkv[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d))
        s["v"] = qkv[:, (hq + hkv) * d:].unflatten(1, (hkv, d))
        blocks = T + 16
        s["slots"] = torch.randperm(blocks * BLOCK, generator=g, device="cuda")[:T]
        _caches(g, blocks, case, s)
        if case["op"] == "normwrite":
            rot = case["rot"]
            s["positions"] = torch.randint(0, case["max_pos"], (T,), generator=g, device="cuda",
                                           dtype=torch.int32)
            inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
            a = torch.arange(case["max_pos"], dtype=torch.float64, device="cuda")[:, None] * inv
            s["cos_sin"] = torch.cat([a.cos(), a.sin()], 1).float()
            s["q_weight"] = s["k_weight"] = None
            if case["norm"]:
                s["q_weight"] = (1 + 0.1 * torch.randn(d, generator=g, device="cuda")).bfloat16()
                s["k_weight"] = (1 + 0.1 * torch.randn(d, generator=g, device="cuda")).bfloat16()
            s["out"] = torch.zeros(T, hq, d, device="cuda", dtype=torch.bfloat16)
        return s
    if case["op"] == "read":
        reads = _reads(case)
        s["bt"], blocks = _tables(g, [None] * len(reads), [-(-L // BLOCK) for _, _, L in reads])
        _caches(g, blocks, case, s)
        s["first"] = torch.tensor([a for a, _, _ in reads], device="cuda", dtype=torch.int32)
        s["loc"] = _loc(n for _, n, _ in reads)
        s["tokens"] = sum(n for _, n, _ in reads)
        s["k_out"], s["v_out"] = (torch.zeros(s["tokens"], hkv, d, device="cuda",
                                              dtype=torch.bfloat16) for _ in range(2))
        return s
    if case["op"] == "attend":
        spans = _spans(case)
        shared = [None] * len(spans)
        lens, new = [c + n for c, n in spans], [n for _, n in spans]
        own_blocks = [-(-L // BLOCK) for L in lens]
        s["max_decode"] = max(lens[:case["decodes"]])
    else:
        members, prefix, suffix = _groups(case)
        of = [i for i, m in enumerate(members) for _ in range(m)] + [None] * case["alone"]
        shared = [None if i is None else (i, prefix[i] // BLOCK) for i in of]
        lens = [n + (0 if i is None else prefix[i]) for i, n in zip(of, suffix)]
        new = [case["qlen"]] * len(lens)
        own_blocks = [-(-n // BLOCK) for n in suffix]
        s["group_loc"] = _loc(members)
        s["prefix"] = torch.tensor(prefix, device="cuda", dtype=torch.int32)
        s["max_prefix"] = max(prefix)
    s["bt"], blocks = _tables(g, shared, own_blocks)
    _caches(g, blocks, case, s)
    s["seq_lens"] = torch.tensor(lens, device="cuda", dtype=torch.int32)
    s["qsl"] = _loc(new)
    s["max_q"], s["max_len"] = max(new), max(lens)
    s["q"] = torch.randn(sum(new), hq, d, generator=g, device="cuda", dtype=torch.bfloat16)
    s["out"] = torch.zeros_like(s["q"])
    return s


def run(s):
    case = s["case"]
    return {"write": _write, "normwrite": _normwrite, "attend": _attend, "read": _read,
            "shared": _shared}[case["op"]](s, case)


def _held(s):
    """A row-scaled cache as the values that its bytes stand for."""
    return {"k_cache": s["k_cache"].view(torch.float8_e4m3fn),
            "v_cache": s["v_cache"].view(torch.float8_e4m3fn),
            "scales": s["scales"].view(torch.float8_e8m0fnu)}


def _scatter(s, k, v):
    """K and V rows in 32 bits into their slots."""
    blk, off = s["slots"] // BLOCK, s["slots"] % BLOCK
    s["k_cache"][blk, :, off], a = _code(k)
    s["v_cache"][blk, :, off], b = _code(v)
    s["scales"][blk, :, 0, off] = a
    s["scales"][blk, :, 1, off] = b


def _write(s, case):
    if own:
        from paged_kv_cache_42_gb300 import binding
        binding.write_kv_rows(s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"], s["scales"])
    else:
        _scatter(s, s["k"].float(), s["v"].float())
    return _held(s)


def _norm_rotate(x, w, s, case):
    """One head after the other: x / rms(x) * w, then the pairs turned by the position's angles."""
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
    rot = case["rot"]
    cs = s["cos_sin"][s["positions"].long()][:, None]
    c, n = cs[..., :rot // 2], cs[..., rot // 2:]
    if case["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * c - b * n, b * c + a * n], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat([a * c - b * n, b * c + a * n], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _normwrite(s, case):
    if own:
        from paged_kv_cache_42_gb300 import binding
        q = binding.norm_rope_write_kv_rows(
            s["q"], s["k"], s["v"], s["positions"], s["cos_sin"], s["slots"], s["k_cache"],
            s["v_cache"], s["scales"], q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS,
            interleaved=case["interleaved"], out=s["out"])
        return {"q": q, **_held(s)}
    q = _norm_rotate(s["q"], s["q_weight"], s, case).bfloat16()
    _scatter(s, _norm_rotate(s["k"], s["k_weight"], s, case), s["v"].float())
    return {"q": q, **_held(s)}


def _rows(s, case, which, blocks, offs):
    """Cache rows [..., kv heads, d] of the given blocks and offsets in 32 bits."""
    fmt = case.get("fmt", "rows")
    x = s["k_cache" if which == 0 else "v_cache"][blocks, :, offs]
    if fmt == "bf16":
        return x.float()
    x = x.view(torch.float8_e4m3fn).float()
    if fmt == "fp8":
        return x * (V_SCALE if which else K_SCALE)
    return x * _size(s["scales"][blocks, :, which, offs])[..., None]


def _batch(s, case, r0, r1, n, max_len):
    """Attention of requests r0 .. r1 - 1, n new tokens each: [R, n, heads, d] in 32 bits."""
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    R, L = r1 - r0, s["seq_lens"][r0:r1].long()
    t0 = s["qsl"][r0:r1].long()
    p = torch.arange(max_len, device="cuda")
    blocks = s["bt"][r0:r1].long().clamp(min=0)[:, p // BLOCK]
    offs = (p % BLOCK).expand(R, -1)
    j = torch.arange(n, device="cuda")
    q = s["q"][t0[:, None] + j].float().view(R, n, hkv, hq // hkv, d).permute(0, 2, 1, 3, 4)
    seen = p <= (L[:, None] - n + j)[..., None]  # [R, n, keys]
    k = _rows(s, case, 0, blocks, offs).permute(0, 2, 3, 1)
    a = torch.matmul(q.flatten(2, 3), k).mul_(s["scale"])
    del k
    a = a.view(R, hkv, n, hq // hkv, max_len).masked_fill_(~seen[:, None, :, None], -math.inf)
    a = torch.exp(a - a.amax(-1, keepdim=True))
    a = (a / a.sum(-1, keepdim=True)).flatten(2, 3)
    v = _rows(s, case, 1, blocks, offs).transpose(1, 2)
    o = torch.matmul(a, v).view(R, hkv, n, hq // hkv, d)
    return o.permute(0, 2, 1, 3, 4).reshape(R * n, hq, d)


def _attend(s, case):
    if own:
        from paged_kv_cache_42_gb300 import binding
        if "ws" not in s:  # kept by the caller from step to step
            T, hq, d = s["q"].shape
            s["ws"] = torch.empty(binding.workspace_size(s["seq_lens"].shape[0], T, hq,
                                                         case["hkv"], d),
                                  dtype=torch.uint8, device="cuda")
        return binding.attention_rows(s["q"], s["k_cache"], s["v_cache"], s["scales"], s["bt"],
                                      s["seq_lens"], s["qsl"], s["scale"],
                                      max_query_len=s["max_q"], max_seq_len=s["max_len"],
                                      out=s["out"], workspace=s["ws"])
    R, n = s["seq_lens"].shape[0], case["decodes"]
    o = _batch(s, case, 0, n, 1, s["max_decode"])
    if n < R:
        o = torch.cat([o, _batch(s, case, n, R, case["qlen"], s["max_len"])])
    return o.bfloat16()


def _read(s, case):
    if own:
        from paged_kv_cache_42_gb300 import binding
        kw = {"first": s["first"], "k_out": s["k_out"], "v_out": s["v_out"]}
        if case["fmt"] == "bf16":
            return binding.read_kv(s["k_cache"], s["v_cache"], s["bt"], s["loc"], **kw)
        if case["fmt"] == "fp8":
            return binding.read_kv_fp8(s["k_cache"], s["v_cache"], s["bt"], s["loc"], K_SCALE,
                                       V_SCALE, **kw)
        return binding.read_kv_rows(s["k_cache"], s["v_cache"], s["scales"], s["bt"], s["loc"],
                                    **kw)
    t = torch.arange(s["tokens"], device="cuda")
    r = torch.searchsorted(s["loc"][1:].long(), t, right=True)
    pos = s["first"].long()[r] + t - s["loc"].long()[r]
    blocks = s["bt"].long()[r, pos // BLOCK]
    return tuple(_rows(s, case, w, blocks, pos % BLOCK).bfloat16() for w in (0, 1))


def _shared(s, case):
    if own:
        from paged_kv_cache_42_gb300 import binding
        if "ws" not in s:  # kept by the caller from step to step
            T, hq, d = s["q"].shape
            s["ws"] = torch.empty(binding.shared_workspace_size(
                s["seq_lens"].shape[0], T, hq, case["hkv"], d, case["groups"], s["max_prefix"]),
                dtype=torch.uint8, device="cuda")
        args = (s["bt"], s["seq_lens"], s["qsl"], s["group_loc"], s["prefix"], s["scale"])
        kw = {"max_prefix_len": s["max_prefix"], "max_query_len": s["max_q"],
              "max_seq_len": s["max_len"], "out": s["out"], "workspace": s["ws"]}
        if case["fmt"] == "bf16":
            return binding.attention_shared(s["q"], s["k_cache"], s["v_cache"], *args, **kw)
        if case["fmt"] == "fp8":
            return binding.attention_shared_fp8(s["q"], s["k_cache"], s["v_cache"], *args,
                                                K_SCALE, V_SCALE, **kw)
        return binding.attention_shared_rows(s["q"], s["k_cache"], s["v_cache"], s["scales"],
                                             *args, **kw)
    return _batch(s, case, 0, s["seq_lens"].shape[0], case["qlen"], s["max_len"]).bfloat16()


def work(case):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    fmt = case.get("fmt", "rows")
    row = {"bf16": 2 * d, "fp8": d, "rows": d + 1}[fmt]  # bytes of a cached row of one head
    if case["op"] == "write":
        T = case["tokens"]
        return {"bytes": T * (2 * hkv * (2 * d + row) + 8), "flops": T * 2 * hkv * d * 3}
    if case["op"] == "normwrite":
        T = case["tokens"]
        return {"bytes": T * (4 * hq * d + 2 * hkv * (2 * d + row) + 12 + case["rot"] * 4)
                + (4 * d if case["norm"] else 0),
                "flops": T * ((hq + hkv) * d * (8 if case["norm"] else 3) + 2 * hkv * d * 3)}
    if case["op"] == "read":
        n = sum(n for _, n, _ in _reads(case))
        return {"bytes": n * 2 * hkv * (row + 2 * d) + n // BLOCK * 4, "flops": n * 2 * hkv * d}
    if case["op"] == "attend":
        by = fl = 0
        for c, n in _spans(case):
            L = c + n
            by += L * hkv * 2 * row + 4 * n * hq * d + L // BLOCK * 4
            fl += sum(range(c + 1, L + 1)) * hq * 4 * d
        return {"bytes": by, "flops": fl}
    members, prefix, suffix = _groups(case)
    n = case["qlen"]
    keys = sum(prefix) + sum(suffix)  # each read once
    before = [p for p, m in zip(prefix, members) for _ in range(m)] + [0] * case["alone"]
    fl = sum((p + x) * n - n * (n - 1) // 2 for p, x in zip(before, suffix)) * hq * 4 * d
    return {"bytes": keys * hkv * 2 * row + len(suffix) * n * 4 * hq * d + keys // BLOCK * 4,
            "flops": fl}


def exact(case, seed):
    """The definitions, request by request, in 64 bits."""
    s = prepare(case, seed)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    fmt = case.get("fmt", "rows")

    # 2^-127 .. 2^127, then NaN: a power function need not be exact
    powers = torch.tensor([2.0 ** (b - 127) for b in range(255)] + [math.nan],
                          dtype=torch.float64, device="cuda")

    def power(b):
        return powers[b.long()]

    if case["op"] in ("write", "normwrite"):
        def head(x, w):
            x = x.double().clone()
            if w is not None:
                x = x / (x.pow(2).sum(-1, keepdim=True) / d + EPS).sqrt() * w.double()
            y, half = x.clone(), case["rot"] // 2
            ang = s["cos_sin"].double()[s["positions"].long()]
            for m in range(half):
                a, b = (2 * m, 2 * m + 1) if case["interleaved"] else (m, m + half)
                co, si = ang[:, None, m], ang[:, None, half + m]
                y[..., a] = x[..., a] * co - x[..., b] * si
                y[..., b] = x[..., a] * si + x[..., b] * co
            return y

        out = {}
        k = s["k"].double()
        if case["op"] == "normwrite":
            out["q"], k = head(s["q"], s["q_weight"]), head(k, s["k_weight"])
        size = power(s["scales"])
        for i, (name, x) in enumerate((("k_cache", k), ("v_cache", s["v"].double()))):
            top = x.abs().amax(-1)
            # the smallest power of two by which the largest element is at most 448
            e = torch.ceil(torch.log2(top / 448)).clamp(E_MIN, E_MAX)
            e = torch.where(top > 448 * power(e + 127), e + 1, e)
            e = torch.where(top <= 448 * power(e + 126), e - 1, e).clamp(E_MIN, E_MAX)
            size_of = power(e + 127)
            c = s[name].view(torch.float8_e4m3fn).float().double().transpose(1, 2).reshape(-1, hkv, d)
            c[s["slots"]] = (x / size_of[..., None]).clamp(-448, 448)
            out[name] = c.view(-1, BLOCK, hkv, d).transpose(1, 2).contiguous()
            z = size[:, :, i].transpose(1, 2).reshape(-1, hkv)
            z[s["slots"]] = size_of
            size[:, :, i] = z.view(-1, BLOCK, hkv).transpose(1, 2)
        out["scales"] = size
        return out

    def dense(which, ids):
        """Keys or values of a run of blocks: [tokens, kv heads, d]."""
        x = s["k_cache" if which == 0 else "v_cache"][ids]
        if fmt == "bf16":
            x = x.double()
        else:
            x = x.view(torch.float8_e4m3fn).float().double()
            x = x * (power(s["scales"][ids][:, :, which])[..., None] if fmt == "rows"
                     else (K_SCALE, V_SCALE)[which])
        return x.transpose(1, 2).reshape(-1, hkv, d)

    if case["op"] == "read":
        got = ([], [])
        for r, (a, n, L) in enumerate(_reads(case)):
            ids = s["bt"][r, :-(-L // BLOCK)].long()
            for w in (0, 1):
                got[w].append(dense(w, ids)[a:a + n])
        return tuple(torch.cat(x) for x in got)
    g = hq // hkv
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lens, qsl = s["seq_lens"].tolist(), s["qsl"].tolist()
    for r, L in enumerate(lens):
        t0, t1 = qsl[r], qsl[r + 1]
        ids = s["bt"][r, :-(-L // BLOCK)].long()
        k, v = dense(0, ids)[:L], dense(1, ids)[:L]
        me = torch.arange(L - (t1 - t0), L, device="cuda")[:, None]
        hide = torch.arange(L, device="cuda") > me
        for h in range(hkv):
            q = s["q"][t0:t1, h * g:(h + 1) * g].double()
            x = torch.einsum("ngd,ld->ngl", q, k[:, h]) * s["scale"]
            x = x.masked_fill(hide[:, None], -math.inf).softmax(-1)
            out[t0:t1, h * g:(h + 1) * g] = torch.einsum("ngl,ld->ngd", x, v[:, h])
    return out
