"""Refusals of the calls around row-scaled caches, checked on the host before any CUDA
call (no GPU needed), and the layout of their argument structs."""
from __future__ import annotations

import math

import pytest
import torch

from paged_kv_cache_42_gb300 import binding

FAKE = 0x10000  # aligned, never dereferenced
OK, ARG, UNSUP, WS = 0, -1, -2, -3


def write(**kw):
    a = dict(k=FAKE, v=FAKE, slot=FAKE, kc=FAKE, vc=FAKE, sc=FAKE, ks=128, vs=128, T=4, hkv=2, d=64,
             bs=16, nb=8)
    a.update(kw)
    return binding.lib().pa_write_kv_rows(binding._pack_wr(
        a["k"] or 0, a["v"] or 0, a["slot"] or 0, a["kc"] or 0, a["vc"] or 0, a["sc"] or 0, 0,
        a["ks"], a["vs"], a["T"], a["hkv"], a["d"], a["bs"], a["nb"]))


def test_write(pa_lib):
    for name in ("k", "v", "slot", "kc", "vc", "sc"):
        assert write(**{name: None}) == ARG, name
        if name != "slot":
            assert write(**{name: FAKE + 8}) == ARG, name
    assert write(slot=FAKE + 4) == ARG
    assert write(T=-1) == ARG and write(hkv=0) == ARG and write(nb=-1) == ARG and write(d=0) == ARG
    assert write(d=96) == UNSUP and write(d=32) == UNSUP and write(bs=32) == UNSUP
    assert write(hkv=65537, ks=65537 * 64, vs=65537 * 64) == UNSUP
    assert write(ks=127) == ARG and write(ks=132) == ARG and write(vs=120) == ARG
    assert write(T=0, k=None, slot=None, sc=None) == OK
    assert pa_lib.pa_write_kv_rows(None) == ARG


def nrope(**kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, pos=FAKE, cs=FAKE, qw=FAKE, kw=FAKE, slot=FAKE,
             out=FAKE + 4096, kc=FAKE, vc=FAKE, sc=FAKE, qs=256, ks=128, vs=128, eps=1e-6, rot=64,
             inter=0, mp=100, T=4, hq=4, hkv=2, d=64, bs=16, nb=8)
    a.update(kw)
    p = [a[n] or 0 for n in ("q", "k", "v", "pos", "cs", "qw", "kw", "slot", "out", "kc", "vc", "sc")]
    return binding.lib().pa_norm_rope_write_kv_rows(binding._pack_nrr(
        *p, 0, a["qs"], a["ks"], a["vs"], a["eps"], a["rot"], a["inter"], a["mp"], a["T"], a["hq"],
        a["hkv"], a["d"], a["bs"], a["nb"]))


def test_norm_rope_write(pa_lib):
    for name in ("q", "k", "v", "slot", "out", "kc", "vc", "sc", "pos", "cs"):
        assert nrope(**{name: None}) == ARG, name
    for name in ("q", "k", "v", "out", "kc", "vc", "sc", "qw", "kw", "cs"):
        assert nrope(**{name: FAKE + 8}) == ARG, name
    assert nrope(d=96) == UNSUP and nrope(bs=8) == UNSUP and nrope(rot=24) == UNSUP
    assert nrope(eps=math.nan) == ARG and nrope(qs=255) == ARG and nrope(T=-1) == ARG
    assert nrope(T=0, sc=None, q=None) == OK
    assert pa_lib.pa_norm_rope_write_kv_rows(None) == ARG


def attend(**kw):
    a = dict(q=FAKE, kc=FAKE, vc=FAKE, sc=FAKE, bt=FAKE, sl=FAKE, qsl=FAKE, out=FAKE, ws=FAKE,
             wsb=None, scale=0.125, R=4, T=4, hq=4, hkv=2, d=64, bs=16, nb=32, mb=4, mq=1, ms=56)
    a.update(kw)
    L = binding.lib()
    if a["wsb"] is None:
        a["wsb"] = L.pa_attention_workspace_size(a["R"], a["T"], a["hq"], a["hkv"], a["d"])
    p = [a[n] or 0 for n in ("q", "kc", "vc", "sc", "bt", "sl", "qsl", "out", "ws")]
    return L.pa_attention_rows(binding._pack_ar(
        *p, 0, a["wsb"], a["scale"], a["R"], a["T"], a["hq"], a["hkv"], a["d"], a["bs"], a["nb"],
        a["mb"], a["mq"], a["ms"]))


def test_attention(pa_lib):
    for name in ("q", "kc", "vc", "sc", "bt", "sl", "qsl", "out"):
        assert attend(**{name: None}) == ARG, name
    for name in ("q", "kc", "vc", "sc", "out"):
        assert attend(**{name: FAKE + 8}) == ARG, name
    assert attend(R=-1, wsb=0) == ARG and attend(hq=6, hkv=4, wsb=0) == ARG
    assert attend(d=96) == UNSUP and attend(bs=32) == UNSUP and attend(hq=32) == UNSUP
    assert attend(scale=math.nan) == ARG and attend(nb=0) == ARG
    assert attend(ws=None) == WS and attend(wsb=16) == WS and attend(ws=FAKE + 16) == WS
    assert attend(R=0, wsb=0) == OK and attend(T=0, wsb=0) == OK
    assert pa_lib.pa_attention_rows(None) == ARG


def read(**kw):
    a = dict(kc=FAKE, vc=FAKE, sc=FAKE, bt=FAKE, loc=FAKE, first=FAKE, ko=FAKE, vo=FAKE, ks=0.5,
             vs=0.5, fmt=2, R=4, T=4, hkv=2, d=64, bs=16, nb=8, mb=4)
    a.update(kw)
    p = [a[n] or 0 for n in ("kc", "vc", "sc", "bt", "loc", "first", "ko", "vo")]
    return binding.lib().pa_read_kv(binding._pack_read(
        *p, 0, a["ks"], a["vs"], a["fmt"], a["R"], a["T"], a["hkv"], a["d"], a["bs"], a["nb"], a["mb"]))


def test_read(pa_lib):
    for name in ("kc", "vc", "sc", "bt", "loc", "ko", "vo"):
        assert read(**{name: None}) == ARG, name
    for name in ("kc", "vc", "sc"):
        assert read(**{name: FAKE + 8}) == ARG, name
    assert read(ko=FAKE + 16) == ARG and read(vo=FAKE + 16) == ARG  # 32-byte stores
    assert read(bt=FAKE + 2) == ARG and read(loc=FAKE + 1) == ARG and read(first=FAKE + 2) == ARG
    assert read(fmt=3) == ARG and read(fmt=-1) == ARG and read(R=-1) == ARG and read(T=-1) == ARG
    assert read(nb=0) == ARG and read(mb=-1) == ARG and read(hkv=0) == ARG
    assert read(d=80) == UNSUP and read(bs=8) == UNSUP and read(hkv=8193) == UNSUP
    for s in (0.0, -1.0, math.inf, math.nan):
        assert read(fmt=1, ks=s) == ARG and read(fmt=1, vs=s) == ARG
    assert read(R=0, kc=None, nb=0) == OK and read(T=0, ko=None) == OK
    assert pa_lib.pa_read_kv(None) == ARG


def shared(**kw):
    a = dict(q=FAKE, kc=FAKE, vc=FAKE, sc=FAKE, bt=FAKE, sl=FAKE, qsl=FAKE, gl=FAKE, pl=FAKE,
             out=FAKE, ws=FAKE, wsb=None, scale=0.125, ks=0.5, vs=0.5, fmt=2, R=4, T=4, hq=4, hkv=2,
             d=64, bs=16, nb=32, mb=4, mq=1, ms=56, G=2, mp=32)
    a.update(kw)
    L = binding.lib()
    if a["wsb"] is None:
        a["wsb"] = L.pa_attention_shared_workspace_size(a["R"], a["T"], a["hq"], a["hkv"], a["d"],
                                                        a["G"], a["mp"])
    p = [a[n] or 0 for n in ("q", "kc", "vc", "sc", "bt", "sl", "qsl", "gl", "pl", "out", "ws")]
    return L.pa_attention_shared(binding._pack_sh(
        *p, 0, a["wsb"], a["scale"], a["ks"], a["vs"], a["fmt"], a["R"], a["T"], a["hq"], a["hkv"],
        a["d"], a["bs"], a["nb"], a["mb"], a["mq"], a["ms"], a["G"], a["mp"]))


def test_shared(pa_lib):
    for name in ("q", "kc", "vc", "sc", "bt", "sl", "qsl", "out", "gl", "pl"):
        assert shared(**{name: None}) == ARG, name
    for name in ("q", "kc", "vc", "sc", "out"):
        assert shared(**{name: FAKE + 8}) == ARG, name
    assert shared(gl=FAKE + 2) == ARG and shared(pl=FAKE + 1) == ARG
    assert shared(R=-1, wsb=0) == ARG and shared(G=-1, wsb=0) == ARG and shared(mp=-1, wsb=0) == ARG
    assert shared(fmt=3) == ARG and shared(fmt=-1) == ARG and shared(scale=math.nan) == ARG
    assert shared(nb=0) == ARG
    assert shared(fmt=1, ks=0.0) == ARG and shared(fmt=1, vs=math.inf) == ARG
    assert shared(d=96) == UNSUP and shared(bs=32) == UNSUP and shared(hq=32, wsb=0) == UNSUP
    assert shared(G=1025, wsb=0) == UNSUP
    assert shared(R=2 ** 20, mb=2 ** 11, wsb=2 ** 62) == UNSUP  # table offsets past 32 bits
    assert shared(ws=None) == WS and shared(wsb=16) == WS and shared(ws=FAKE + 16) == WS
    assert shared(R=0, wsb=0) == OK and shared(T=0, wsb=0) == OK
    assert pa_lib.pa_attention_shared(None) == ARG
    size = pa_lib.pa_attention_shared_workspace_size
    plain = pa_lib.pa_attention_workspace_size(4, 4, 4, 2, 64)
    assert size(4, 4, 4, 2, 64, 2, 32) > plain and size(4, 4, 4, 2, 64, 0, 0) > plain
    assert size(4, 4, 4, 2, 64, 1025, 32) == 0 and size(4, 4, 4, 2, 64, 2, -1) == 0
    assert size(4, 4, 6, 2, 64, 2, 32) == 0


def test_struct_sizes(pa_lib):
    binding.lib()  # checks pa_args_size against every layout
    assert pa_lib.pa_args_size(15) == 0 and pa_lib.pa_args_size(16) > 0


def test_binding_refuses_cpu_tensors_and_shapes(pa_lib, monkeypatch):
    """What the binding itself checks, with the device stubbed out."""
    monkeypatch.setattr(binding, "_where", lambda stream: (0, 0))
    kc = torch.zeros(4, 2, 16, 64, dtype=torch.uint8)
    sc = torch.zeros(4, 2, 2, 16, dtype=torch.uint8)
    k = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    slots = torch.zeros(3, dtype=torch.int64)
    with pytest.raises(ValueError, match="CUDA"):
        binding.write_kv_rows(k, k, slots, kc, kc, sc)
    with pytest.raises(ValueError, match="shape"):
        binding.write_kv_rows(k[:, :1], k, slots, kc, kc, sc)
    with pytest.raises(ValueError, match="caches"):
        binding.write_kv_rows(k, k, slots, kc, kc[:3], sc)
    with pytest.raises(TypeError):
        binding.write_kv_rows(k.float(), k, slots, kc, kc, sc)
    bt = torch.zeros(2, 3, dtype=torch.int32)
    with pytest.raises(ValueError, match="read_start_loc"):
        binding.read_kv(kc, kc, bt, torch.zeros(2, dtype=torch.int32), num_tokens=4)
    with pytest.raises(ValueError, match="num_tokens"):
        binding.read_kv(kc, kc, bt, torch.zeros(3, dtype=torch.int32))


def test_shared_min_kb_option(pa_lib):
    assert pa_lib.pa_set_option(10, -1) == ARG
    assert pa_lib.pa_set_option(10, 0) == OK and pa_lib.pa_set_option(10, 24576) == OK
