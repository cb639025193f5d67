"""Operators around a paged KV cache whose size is bounded, measured one call at a time.

Four operators of the library in ``paged_kv_cache_42_gb300``, each in its plain
form (elementary torch operations in 32 bits, rounded once) and as the calls a
serving step makes of ``paged_kv_cache_42_gb300.binding``:

  write    the norm of every query and key head, the position rotation, and the
           scatter of K and V into their cache slots (bf16 or E4M3)
  window   paged attention over the first `sinks` tokens and the last `window`
           ones, for decodes and prompt chunks
  weights  what every cached key has received of attention, added up
  evict    a cache cut to `keep` tokens for each KV head: the first ones, the
           newest ones and the heaviest of the rest, moved into new blocks

Caches are [num_blocks][kv heads][16][head dim]; a request finds its blocks in
its row of block_tables. ``own`` chooses the library's calls.
"""
from __future__ import annotations

import math
import random

import torch

own = False

BLOCK = 16
K_SCALE, V_SCALE = 0.0113, 0.0127  # E4M3 caches: one scale per tensor
EPS = 1e-6


def listed():
    llama = {"hq": 32, "hkv": 8, "d": 128}
    tiny = {"hq": 4, "hkv": 2, "d": 64}
    wide = {"hq": 64, "hkv": 8, "d": 128}
    return [
        # one token each of four short conversations: the smallest step there is
        {"name": "write tiny decode", "op": "write", **tiny, "tokens": 4, "fp8": False,
         "norm": True, "interleaved": False, "rot": 64, "max_pos": 4096},
        # the newest token of 64 conversations into an E4M3 cache
        {"name": "write decode batch e4m3", "op": "write", **llama, "tokens": 64, "fp8": True,
         "norm": True, "interleaved": False, "rot": 128, "max_pos": 32768},
        # a step of 512 decodes and three prompt chunks: 2048 tokens
        {"name": "write mixed batch", "op": "write", **llama, "tokens": 2048, "fp8": False,
         "norm": True, "interleaved": False, "rot": 128, "max_pos": 32768},
        # four short conversations, a window of one block
        {"name": "window tiny decode", "op": "window", **tiny, "decodes": 4, "lmin": 9,
         "lmax": 57, "lens_seed": 1, "qlen": 0, "ctx": "", "window": 16, "sinks": 4,
         "fp8": False},
        # 64 conversations that each see their last 1024 tokens and the first four
        {"name": "window decode batch", "op": "window", **llama, "decodes": 64, "lmin": 512,
         "lmax": 4096, "lens_seed": 2, "qlen": 0, "ctx": "", "window": 1024, "sinks": 4,
         "fp8": False},
        # a mixed step: 512 decodes and three prompt chunks of 512
        {"name": "window mixed batch", "op": "window", **llama, "decodes": 512, "lmin": 128,
         "lmax": 2048, "lens_seed": 3, "qlen": 512, "ctx": "0,1024,2048", "window": 1024,
         "sinks": 4, "fp8": False},
        # eight long documents, a window that ends inside a block, an E4M3 cache
        {"name": "window long context e4m3", "op": "window", **wide, "decodes": 8, "lmin": 32768,
         "lmax": 32768, "lens_seed": 5, "qlen": 0, "ctx": "", "window": 4001, "sinks": 16,
         "fp8": True},
        # what one decode step of 64 conversations adds to the keys' weights
        {"name": "weights decode batch", "op": "weights", **llama, "decodes": 64, "lmin": 512,
         "lmax": 4096, "lens_seed": 2, "qlen": 0, "ctx": "", "fp8": False},
        # the same over eight long documents and an E4M3 cache
        {"name": "weights long context e4m3", "op": "weights", **wide, "decodes": 8,
         "lmin": 32768, "lmax": 32768, "lens_seed": 5, "qlen": 0, "ctx": "", "fp8": True},
        # three prompt chunks: every query of the prompt has its say
        {"name": "weights prompt chunks", "op": "weights", **llama, "decodes": 0, "lmin": 0,
         "lmax": 0, "lens_seed": 3, "qlen": 512, "ctx": "0,1024,2048", "fp8": False},
        # 64 caches cut to 1000 tokens; the short ones among them stay whole
        {"name": "evict decode batch", "op": "evict", **llama, "decodes": 64, "lmin": 512,
         "lmax": 4096, "lens_seed": 2, "keep": 1000, "recent": 500, "sinks": 4, "fp8": False},
        # eight long documents cut to an eighth, an E4M3 cache
        {"name": "evict long context e4m3", "op": "evict", **wide, "decodes": 8, "lmin": 32768,
         "lmax": 32768, "lens_seed": 5, "keep": 4096, "recent": 2048, "sinks": 16, "fp8": True},
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    hkv = rng.choice([1, 2, 4, 8])
    c = {"hq": hkv * rng.choice([1, 2, 4, 8]), "hkv": hkv, "d": rng.choice([64, 128, 128]),
         "fp8": rng.random() < 0.5}
    op = rng.choice(["write", "window", "weights", "evict"])
    if op == "write":
        return {"op": op, **c, "tokens": _log(rng, 1, 2048), "norm": rng.random() < 0.75,
                "interleaved": rng.random() < 0.3, "rot": rng.choice([c["d"], c["d"] // 2]),
                "max_pos": _log(rng, 2048, 32768)}
    lmax = _log(rng, 8, 8192)
    c.update(decodes=_log(rng, 1, max(1, min(256, 262144 // lmax))), lmin=_log(rng, 1, lmax),
             lmax=lmax, lens_seed=rng.randrange(1 << 30))
    if op == "evict":
        keep = _log(rng, 2, max(2, min(4096, lmax)))
        sinks = rng.randint(0, min(16, keep // 2))
        return {"op": op, **c, "keep": keep, "recent": rng.randint(0, keep - sinks),
                "sinks": sinks}
    c.update(qlen=0, ctx="")
    if rng.random() < 0.5:  # prompt chunks, or short spans, beside or without the decodes
        if op == "weights":
            c["decodes"] = 0
        c["qlen"] = _log(rng, 2, 512)
        c["ctx"] = ",".join(str(_log(rng, 1, 2048) - 1) for _ in range(rng.randint(1, 3)))
    if op == "window":
        c.update(window=_log(rng, 1, 1024 if c["qlen"] else 4096), sinks=rng.choice([0, 1, 4, 16, 33]))
    return {"op": op, **c}


def _spans(case):
    """(context, new tokens) of every request: the decodes, then the chunks."""
    r = random.Random(case["lens_seed"])
    spans = [(r.randint(case["lmin"], case["lmax"]) - 1, 1) for _ in range(case["decodes"])]
    if case.get("qlen"):
        spans += [(int(x), case["qlen"]) for x in case["ctx"].split(",")]
    return spans


def _cache(g, blocks, case):
    x = torch.randn(blocks, case["hkv"], BLOCK, case["d"], generator=g, device="cuda",
                    dtype=torch.float32 if case["fp8"] else torch.bfloat16)
    return x


def _caches(g, blocks, case):
    k, v = _cache(g, blocks, case), _cache(g, blocks, case)
    if case["fp8"]:
        k = (k / K_SCALE).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        v = (v / V_SCALE).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return k, v


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    s = {"case": case, "scale": 1.0 / math.sqrt(d)}
    if case["op"] == "write":
        T, rot = case["tokens"], case["rot"]
        # q, k and v side by side, as one projection leaves them
        qkv = torch.randn(T, (hq + 2 * hkv) * d, generator=g, device="cuda", dtype=torch.bfloat16)
        s["q"] = qkv[:, :hq * d].unflatten(1, (hq, d))
        s["k"] = qkv[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d))
        s["v"] = qkv[:, (hq + hkv) * d:].unflatten(1, (hkv, d))
        s["positions"] = torch.randint(0, case["max_pos"], (T,), generator=g, device="cuda",
                                       dtype=torch.int32)
        inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
        a = torch.arange(case["max_pos"], dtype=torch.float64, device="cuda")[:, None] * inv
        s["cos_sin"] = torch.cat([a.cos(), a.sin()], 1).float()
        blocks = T + 16
        s["slots"] = torch.randperm(blocks * BLOCK, generator=g, device="cuda")[:T]
        s["k_cache"], s["v_cache"] = _caches(g, blocks, case)
        s["q_weight"] = s["k_weight"] = None
        if case["norm"]:
            s["q_weight"] = (1 + 0.1 * torch.randn(d, generator=g, device="cuda")).bfloat16()
            s["k_weight"] = (1 + 0.1 * torch.randn(d, generator=g, device="cuda")).bfloat16()
        s["out"] = torch.zeros(T, hq, d, device="cuda", dtype=torch.bfloat16)
        return s
    spans = _spans(case)
    R, T = len(spans), sum(n for _, n in spans)
    lens = [c + n for c, n in spans]
    nb = [(n + BLOCK - 1) // BLOCK for n in lens]
    mb, extra = max(nb), 0
    if case["op"] == "evict":
        nnew = (case["keep"] + BLOCK - 1) // BLOCK
        extra = R * nnew
    blocks = sum(nb) + extra + 16
    perm = torch.randperm(blocks, generator=g, device="cuda").int()
    off = torch.tensor([0] + nb, device="cuda").cumsum(0)
    i = torch.arange(mb, device="cuda")
    n = torch.tensor(nb, device="cuda")[:, None]
    s["bt"] = torch.where(i < n, perm[(off[:-1, None] + i).clamp(max=blocks - 1)], -1).int()
    s["seq_lens"] = torch.tensor(lens, device="cuda", dtype=torch.int32)
    s["qsl"] = torch.tensor([0] + [n for _, n in spans], device="cuda").cumsum(0).int()
    s["max_q"], s["max_len"] = max(n for _, n in spans), max(lens)
    s["k_cache"], s["v_cache"] = _caches(g, blocks, case)
    if case["op"] == "evict":
        a = sum(nb)
        s["new_bt"] = perm[a:a + extra].view(R, nnew).contiguous()
        # heavy-tailed, and coarse enough that some are equal
        w = torch.randn(R, hkv, mb * BLOCK, generator=g, device="cuda").mul(1.5).exp()
        s["w"] = (w * 256).round() / 256
        s["new_lens"] = torch.zeros(R, device="cuda", dtype=torch.int32)
        s["kept"] = torch.zeros(R, hkv, case["keep"], device="cuda", dtype=torch.int32)
        s["new_w"] = torch.zeros(R, hkv, case["keep"], device="cuda")
        return s
    s["q"] = torch.randn(T, hq, d, generator=g, device="cuda", dtype=torch.bfloat16)
    if case["op"] == "weights":
        s["q"] = s["q"] * 2  # attention with some keys well ahead of the others
        s["w"] = torch.rand(R, hkv, mb * BLOCK, generator=g, device="cuda") * 4
        s["w_out"] = torch.zeros_like(s["w"])
    else:
        s["out"] = torch.zeros_like(s["q"])
    return s


def run(s):
    case = s["case"]
    return {"write": _write, "window": _window, "weights": _weights, "evict": _evict}[case["op"]](s, case)


def _values(cache):
    """A cache as the values it holds: E4M3 codes by their own type."""
    return cache.view(torch.float8_e4m3fn) if cache.dtype == torch.uint8 else cache


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


def _write(s, case):
    if own:
        from paged_kv_cache_42_gb300 import binding
        args = (s["q"], s["k"], s["v"], s["positions"], s["cos_sin"], s["slots"], s["k_cache"],
                s["v_cache"])
        kw = {"q_weight": s["q_weight"], "k_weight": s["k_weight"], "eps": EPS,
              "interleaved": case["interleaved"], "out": s["out"]}
        if case["fp8"]:
            binding.norm_rope_write_kv_fp8(*args, K_SCALE, V_SCALE, **kw)
        else:
            binding.norm_rope_write_kv(*args, **kw)
        return {"q": s["out"], "k_cache": _values(s["k_cache"]), "v_cache": _values(s["v_cache"])}
    q = _norm_rotate(s["q"], s["q_weight"], s, case)
    k = _norm_rotate(s["k"], s["k_weight"], s, case)
    v = s["v"].float()
    at = s["slots"] // BLOCK, slice(None), s["slots"] % BLOCK
    if case["fp8"]:
        s["k_cache"][at] = (k / K_SCALE).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        s["v_cache"][at] = (v / V_SCALE).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        s["k_cache"][at] = k.bfloat16()
        s["v_cache"][at] = v.bfloat16()
    return {"q": q.bfloat16(), "k_cache": _values(s["k_cache"]), "v_cache": _values(s["v_cache"])}


def _rows(cache, blocks, offs, scale):
    """Cache rows [..., kv heads, d] in 32 bits of the given blocks and offsets."""
    x = cache[blocks, :, offs]
    return x.view(torch.float8_e4m3fn).float() * scale if x.dtype == torch.uint8 else x.float()


def _window(s, case):
    if own:
        from paged_kv_cache_42_gb300 import binding
        if "ws" not in s:  # kept by the caller from step to step
            T, hq, d = s["q"].shape
            s["ws"] = torch.empty(binding.workspace_size(s["seq_lens"].shape[0], T, hq,
                                                         case["hkv"], d),
                                  dtype=torch.uint8, device="cuda")
        args = (s["q"], s["k_cache"], s["v_cache"], s["bt"], s["seq_lens"], s["qsl"], s["scale"])
        kw = {"window": case["window"], "sinks": case["sinks"], "max_query_len": s["max_q"],
              "max_seq_len": s["max_len"], "out": s["out"], "workspace": s["ws"]}
        if case["fp8"]:
            return binding.attention_window_fp8(*args, K_SCALE, V_SCALE, **kw)
        return binding.attention_window(*args, **kw)
    T, hq, d = s["q"].shape
    hkv, W, S = case["hkv"], case["window"], min(case["sinks"], s["max_len"])
    t = torch.arange(T, device="cuda")
    req = torch.searchsorted(s["qsl"][1:].long(), t, right=True)
    # keys that token t may see at all: up to and with its own
    n = (s["seq_lens"][req] - s["qsl"][req + 1]).long() + t + 1
    lo = (n - W).clamp(min=0)[:, None]
    i = torch.arange(S, device="cuda")[None]
    j = torch.arange(min(W, s["max_len"]), device="cuda")[None] + lo
    pos = torch.cat([i.expand(T, -1), j], 1)
    seen = torch.cat([i < lo, j < n[:, None]], 1)
    pos = torch.where(seen, pos, 0)
    blocks = s["bt"].long()[req[:, None], pos // BLOCK]
    k = _rows(s["k_cache"], blocks, pos % BLOCK, K_SCALE).transpose(1, 2)
    q = s["q"].float().view(T, hkv, hq // hkv, d)
    a = torch.matmul(q, k.transpose(2, 3)) * s["scale"]
    del k
    a = a.masked_fill(~seen[:, None, None], -math.inf)
    a = torch.exp(a - a.amax(-1, keepdim=True))
    v = _rows(s["v_cache"], blocks, pos % BLOCK, V_SCALE).transpose(1, 2)
    o = torch.matmul(a, v) / a.sum(-1, keepdim=True)
    return o.reshape(T, hq, d).bfloat16()


def _weights(s, case):
    if own:
        from paged_kv_cache_42_gb300 import binding
        if "ws" not in s:  # kept by the caller from step to step
            T, hq, d = s["q"].shape
            s["ws"] = torch.empty(binding.weights_workspace_size(s["seq_lens"].shape[0], T, hq,
                                                                 case["hkv"], d, s["max_q"],
                                                                 s["max_len"]),
                                  dtype=torch.uint8, device="cuda")
        kw = {"max_query_len": s["max_q"], "max_seq_len": s["max_len"], "out": s["w_out"],
              "workspace": s["ws"]}
        args = (s["q"], s["k_cache"], s["bt"], s["seq_lens"], s["qsl"], s["scale"])
        if case["fp8"]:
            return binding.attention_weights_fp8(*args, K_SCALE, s["w"], **kw)
        return binding.attention_weights(*args, s["w"], **kw)
    T, hq, d = s["q"].shape
    R, hkv, width = s["w"].shape
    L, qsl = s["seq_lens"].long(), s["qsl"].long()
    ctx = L - (qsl[1:] - qsl[:-1])
    p = torch.arange(width, device="cuda")
    blocks = s["bt"].long().clamp(min=0)[:, p // BLOCK]
    k = _rows(s["k_cache"], blocks, (p % BLOCK).expand(R, -1), K_SCALE).permute(0, 2, 1, 3)
    j = torch.arange(s["max_q"], device="cuda")
    rows = (qsl[:-1, None] + j).clamp(max=T - 1)
    q = s["q"][rows].float().view(R, len(j), hkv, hq // hkv, d).permute(0, 2, 1, 3, 4)
    a = torch.matmul(q.flatten(2, 3), k.transpose(2, 3)).mul_(s["scale"])
    a = a.view(R, hkv, len(j), hq // hkv, width)
    last = torch.minimum(ctx[:, None] + j, L[:, None] - 1)  # the last key that a query sees
    a = a.masked_fill((p > last[..., None])[:, None, :, None], -math.inf)
    a = torch.exp(a - a.amax(-1, keepdim=True))
    a = a / a.sum(-1, keepdim=True)
    real = (j < (L - ctx)[:, None])[:, None, :, None, None]
    got = torch.where(real, a, 0.0).sum((2, 3))
    old = torch.where(p < ctx[:, None, None], s["w"], 0.0)
    return torch.where(p < L[:, None, None], old + got, s["w_out"])


def _evict(s, case):
    keep, recent, sinks = case["keep"], case["recent"], case["sinks"]
    if own:
        from paged_kv_cache_42_gb300 import binding
        binding.evict_kv(s["k_cache"], s["v_cache"], s["bt"], s["seq_lens"], s["w"], s["new_bt"],
                         keep=keep, recent=recent, sinks=sinks, max_seq_len=s["max_len"],
                         new_seq_lens=s["new_lens"], kept=s["kept"], new_weights=s["new_w"])
        return {"lens": s["new_lens"], "kept": s["kept"], "weights": s["new_w"],
                "k_cache": _values(s["k_cache"]), "v_cache": _values(s["v_cache"])}
    R, hkv, width = s["w"].shape
    L = s["seq_lens"].long()[:, None, None]
    p = torch.arange(width, device="cuda")
    score = torch.where((p < sinks) | (p >= L - recent), math.inf, s["w"])
    score = torch.where(p < L, score, -math.inf)
    kept = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :keep]
    kept = torch.sort(torch.nn.functional.pad(kept, (0, keep - kept.shape[-1]))).values
    cut = (L > keep)
    some = cut.expand(R, hkv, keep)
    i = torch.arange(keep, device="cuda")
    src = torch.gather(s["bt"].long()[:, None].expand(R, hkv, -1), 2, kept // BLOCK)[some]
    dst = s["new_bt"].long()[:, i // BLOCK][:, None].expand(R, hkv, keep)[some]
    head = torch.arange(hkv, device="cuda")[None, :, None].expand(R, hkv, keep)[some]
    so, do = (kept % BLOCK)[some], (i % BLOCK).expand(R, hkv, keep)[some]
    s["k_cache"][dst, head, do] = s["k_cache"][src, head, so]
    s["v_cache"][dst, head, do] = s["v_cache"][src, head, so]
    return {"lens": s["seq_lens"].clamp(max=keep), "kept": torch.where(cut, kept, s["kept"]).int(),
            "weights": torch.where(cut, torch.gather(s["w"], 2, kept), s["new_w"]),
            "k_cache": _values(s["k_cache"]), "v_cache": _values(s["v_cache"])}


def work(case):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    e = 1 if case["fp8"] else 2
    if case["op"] == "write":
        T = case["tokens"]
        return {"bytes": T * ((hq + 2 * hkv) * d * 2 + hq * d * 2 + 2 * hkv * d * e + 12
                              + case["rot"] * 4) + (4 * d if case["norm"] else 0),
                "flops": T * (hq + hkv) * d * (8 if case["norm"] else 3)}
    spans = _spans(case)
    by = fl = 0
    for c, n in spans:
        L = c + n
        if case["op"] == "window":
            lo = max(0, c + 1 - case["window"])
            keys = L - lo + min(case["sinks"], lo)
            by += keys * hkv * d * 2 * e + 2 * n * hq * d * 2 + keys // BLOCK * 4
            seen = sum(min(p, case["window"]) + min(case["sinks"], max(0, p - case["window"]))
                       for p in range(c + 1, L + 1))
            fl += seen * hq * 4 * d
        elif case["op"] == "weights":
            by += L * hkv * d * e + (c + L) * hkv * 4 + n * hq * d * 2 + L // BLOCK * 4
            fl += sum(range(c + 1, L + 1)) * hq * 2 * d
        elif L > case["keep"]:
            m = case["keep"]
            by += L * hkv * 4 + m * hkv * (8 + 4 * d * e) + (L + m) // BLOCK * 4
            fl += L * hkv
    return {"bytes": by, "flops": fl}


def exact(case, seed):
    """The definitions, request by request, in 64 bits."""
    s = prepare(case, seed)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if case["op"] == "write":
        half, T = case["rot"] // 2, case["tokens"]
        ang = s["cos_sin"].double()[s["positions"].long()]

        def head(x, w):
            x = x.double().clone()
            if w is not None:
                x = x / (x.pow(2).sum(-1, keepdim=True) / d + EPS).sqrt() * w.double()
            y = x.clone()
            for m in range(half):
                a, b = (2 * m, 2 * m + 1) if case["interleaved"] else (m, m + half)
                co, si = ang[:, None, m], ang[:, None, half + m]
                y[..., a] = x[..., a] * co - x[..., b] * si
                y[..., b] = x[..., a] * si + x[..., b] * co
            return y

        out = {"q": head(s["q"], s["q_weight"])}
        for name, x, sc in (("k_cache", head(s["k"], s["k_weight"]), K_SCALE),
                            ("v_cache", s["v"].double(), V_SCALE)):
            c = _values(s[name]).to(torch.float32).double()
            c = c.transpose(1, 2).reshape(-1, hkv, d)
            c[s["slots"]] = (x / sc).clamp(-448, 448) if case["fp8"] else x
            out[name] = c.view(-1, BLOCK, hkv, d).transpose(1, 2).contiguous()
        return out
    if case["op"] == "evict":
        keep, lens = case["keep"], s["seq_lens"].tolist()
        kc, vc = s["k_cache"].clone(), s["v_cache"].clone()
        kept, new_w, wide = s["kept"].clone(), s["new_w"].double(), s["w"].double().cpu().numpy()
        for r, L in enumerate(lens):
            if L <= keep:
                continue
            a, b = case["sinks"], L - case["recent"]
            for h in range(hkv):
                # (-weight, position) in rising order: heaviest first, ties to the lowest position
                mid = wide[r, h, a:b]
                ids = torch.from_numpy((-mid).argsort(kind="stable")[:keep - a - case["recent"]] + a)
                ids = torch.cat([torch.arange(a), ids.sort().values, torch.arange(b, L)]).cuda()
                to = torch.arange(keep, device="cuda")
                kept[r, h] = ids
                new_w[r, h] = s["w"][r, h, ids].double()
                f, t = s["bt"][r, ids // BLOCK].long(), s["new_bt"][r, to // BLOCK].long()
                kc[t, h, to % BLOCK] = s["k_cache"][f, h, ids % BLOCK]
                vc[t, h, to % BLOCK] = s["v_cache"][f, h, ids % BLOCK]
        return {"lens": torch.tensor([min(x, keep) for x in lens]), "kept": kept, "weights": new_w,
                "k_cache": _values(kc), "v_cache": _values(vc)}
    T, g = s["q"].shape[0], hq // hkv
    out = torch.zeros(T, hq, d, dtype=torch.float64, device="cuda")
    total = s["w_out"].double() if case["op"] == "weights" else None
    t0 = 0
    for r, (c, n) in enumerate(_spans(case)):
        L = c + n
        ids = s["bt"][r, :(L + BLOCK - 1) // BLOCK].long()

        def dense(cache, sc):
            x = _values(cache[ids]).to(torch.float32).double() * (sc if case["fp8"] else 1.0)
            return x.transpose(1, 2).reshape(-1, hkv, d)[:L]

        k = dense(s["k_cache"], K_SCALE)
        key = torch.arange(L, device="cuda")
        me = torch.arange(c, L, device="cuda")[:, None]
        see = key <= me
        if case["op"] == "window":
            see = see & ((key > me - case["window"]) | (key < case["sinks"]))
            v = dense(s["v_cache"], V_SCALE)
        for h in range(hkv):
            q = s["q"][t0:t0 + n, h * g:(h + 1) * g].double()
            x = torch.einsum("ngd,ld->ngl", q, k[:, h]) * s["scale"]
            x = x.masked_fill(~see[:, None], -math.inf).softmax(-1)
            if case["op"] == "window":
                out[t0:t0 + n, h * g:(h + 1) * g] = torch.einsum("ngl,ld->ngd", x, v[:, h])
            else:
                old = torch.where(key < c, s["w"][r, h, :L].double(), 0.0)
                total[r, h, :L] = old + x.sum((0, 1))
        t0 += n
    return out if total is None else total
