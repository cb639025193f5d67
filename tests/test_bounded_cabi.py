"""Refusals of the bounded-cache calls, checked on the host before any CUDA call
(no GPU needed), and the layout of their argument structs."""
from __future__ import annotations

import ctypes
import math

import pytest

from paged_kv_cache_42_gb300 import binding

FAKE = 0x10000  # aligned, never dereferenced
OK, ARG, UNSUP, WS = 0, -1, -2, -3


def nr(lib, fp8=False, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, qs=256, ks=128, vs=128, pos=FAKE, cs=FAKE, qw=FAKE, kw=FAKE,
             eps=1e-6, rot=64, inter=0, mp=100, slot=FAKE, out=FAKE + 4096, kc=FAKE, vc=FAKE,
             k_scale=0.5, v_scale=0.5, T=4, hq=4, hkv=2, d=64, bs=16, nb=8)
    a.update(kw)
    head = [a[n] for n in ("q", "k", "v", "qs", "ks", "vs", "pos", "cs", "qw", "kw", "eps", "rot",
                           "inter", "mp", "slot", "out", "kc", "vc")]
    tail = [a[n] for n in ("T", "hq", "hkv", "d", "bs", "nb")]
    if fp8:
        return lib.pa_norm_rope_write_kv_fp8(*head, a["k_scale"], a["v_scale"], *tail, None)
    return lib.pa_norm_rope_write_kv(*head, *tail, None)


@pytest.mark.parametrize("fp8", [False, True])
def test_norm_rope_write(pa_lib, fp8):
    def f(**kw):
        return nr(pa_lib, fp8, **kw)
    for name in ("q", "k", "v", "slot", "out", "kc", "vc"):
        assert f(**{name: None}) == ARG, name
        if name != "slot":
            assert f(**{name: FAKE + 8}) == ARG, name
    assert f(slot=FAKE + 4) == ARG and f(pos=FAKE + 2) == ARG
    assert f(pos=None) == ARG and f(cs=None) == ARG and f(cs=FAKE + 8) == ARG
    assert f(qw=FAKE + 2) == ARG and f(kw=FAKE + 2) == ARG
    assert f(T=-1) == ARG and f(hq=0) == ARG and f(hkv=-1) == ARG and f(nb=-1) == ARG
    assert f(d=96) == UNSUP and f(d=32, rot=32) == UNSUP and f(bs=32) == UNSUP
    assert f(hq=65537, qs=65537 * 64) == UNSUP
    assert f(hkv=65537, ks=65537 * 64, vs=65537 * 64) == UNSUP
    assert f(rot=24) == UNSUP and f(rot=80) == ARG and f(rot=-16) == ARG and f(mp=-1) == ARG
    assert f(eps=-1e-6) == ARG and f(eps=math.nan) == ARG and f(eps=math.inf) == ARG
    assert f(qs=255) == ARG and f(qs=260) == ARG and f(ks=120) == ARG and f(vs=132) == ARG
    assert f(out=FAKE, qs=512) == ARG            # in place needs q's own rows
    assert f(T=0, q=None, slot=None) == OK       # an empty batch: nothing to do
    if fp8:
        for s in (0.0, -1.0, math.inf, math.nan):
            assert f(k_scale=s) == ARG and f(v_scale=s) == ARG


def window(lib, fp8=False, **kw):
    a = dict(q=FAKE, kc=FAKE, vc=FAKE, bt=FAKE, sl=FAKE, qsl=FAKE, scale=0.125, ks=0.5, vs=0.5,
             out=FAKE, R=4, T=4, hq=4, hkv=2, d=64, bs=16, nb=32, mb=4, mq=1, ms=56, w=16, s=4,
             ws=FAKE, wsb=None)
    a.update(kw)
    if a["wsb"] is None:
        a["wsb"] = lib.pa_attention_workspace_size(a["R"], a["T"], a["hq"], a["hkv"], a["d"])
    head = [a[n] for n in ("q", "kc", "vc", "bt", "sl", "qsl", "scale")]
    tail = [a[n] for n in ("out", "R", "T", "hq", "hkv", "d", "bs", "nb", "mb", "mq", "ms", "w",
                           "s", "ws", "wsb")]
    if fp8:
        return lib.pa_attention_window_fp8(*head, a["ks"], a["vs"], *tail, None)
    return lib.pa_attention_window(*head, *tail, None)


@pytest.mark.parametrize("fp8", [False, True])
def test_window(pa_lib, fp8):
    def f(**kw):
        return window(pa_lib, fp8, **kw)
    assert f(w=0) == ARG and f(w=-5) == ARG and f(s=-1) == ARG
    for name in ("q", "kc", "vc", "bt", "sl", "qsl", "out"):
        assert f(**{name: None}) == ARG, name
    assert f(R=-1, wsb=0) == ARG and f(hq=6, hkv=4, wsb=0) == ARG
    assert f(d=96) == UNSUP and f(bs=32) == UNSUP and f(hq=32, hkv=2) == UNSUP
    assert f(scale=math.nan) == ARG
    assert f(ws=None) == WS and f(wsb=16) == WS and f(ws=FAKE + 16) == WS
    assert f(R=0, wsb=0) == OK and f(T=0, wsb=0) == OK
    assert f(R=0, w=0, wsb=0) == ARG
    assert f(nb=0) == ARG and f(nb=0, R=0, wsb=0) == OK
    # the flattened work follows the window, not the sequence: too long without one
    assert f(T=4096, hkv=2, ms=2 ** 22, mb=2 ** 18, wsb=16, w=2 ** 22 - 1) == UNSUP
    assert f(T=4096, hkv=2, ms=2 ** 22, mb=2 ** 18, wsb=16) == WS
    if fp8:
        assert f(ks=0.0) == ARG and f(vs=math.inf) == ARG


def weights(lib, fp8=False, **kw):
    a = dict(q=FAKE, kc=FAKE, bt=FAKE, sl=FAKE, qsl=FAKE, scale=0.125, ks=0.5, w=FAKE, out=FAKE,
             width=64, R=4, T=4, hq=4, hkv=2, d=64, bs=16, nb=32, mb=4, mq=1, ms=56, ws=FAKE,
             wsb=None)
    a.update(kw)
    if a["wsb"] is None:
        a["wsb"] = lib.pa_attention_weights_workspace_size(a["R"], a["T"], a["hq"], a["hkv"],
                                                           a["d"], a["mq"], a["ms"])
    head = [a[n] for n in ("q", "kc", "bt", "sl", "qsl", "scale")]
    tail = [a[n] for n in ("w", "out", "width", "R", "T", "hq", "hkv", "d", "bs", "nb", "mb", "mq",
                           "ms", "ws", "wsb")]
    if fp8:
        return lib.pa_attention_weights_fp8(*head, a["ks"], *tail, None)
    return lib.pa_attention_weights(*head, *tail, None)


@pytest.mark.parametrize("fp8", [False, True])
def test_weights(pa_lib, fp8):
    def f(**kw):
        return weights(pa_lib, fp8, **kw)
    for name in ("q", "kc", "bt", "sl", "qsl", "w", "out"):
        assert f(**{name: None}) == ARG, name
    assert f(w=FAKE + 2) == ARG and f(out=FAKE + 2) == ARG and f(width=-1) == ARG
    assert f(R=-1, wsb=0) == ARG and f(hq=6, hkv=4, wsb=0) == ARG and f(scale=math.nan) == ARG
    assert f(d=96) == UNSUP and f(bs=32) == UNSUP and f(hq=32, hkv=2, wsb=0) == UNSUP
    assert f(ws=None) == WS and f(wsb=16) == WS and f(ws=FAKE + 16) == WS
    assert f(R=0, wsb=0) == OK and f(T=0, wsb=0) == OK
    assert f(nb=0) == ARG and f(ms=-1, wsb=0) == ARG
    assert f(mq=0, ws=None) == OK and f(ms=0, ws=None) == OK  # no request can have a new token
    assert f(ms=(1 << 30) + 1, R=1, T=1, hkv=1, wsb=0) == UNSUP
    # 2 R x 2^22 key tiles: 8.4e8 for 100 requests, past 2^31 (grids) for 600
    assert f(ms=1 << 29, R=100, wsb=0) == WS and f(ms=1 << 29, R=600, wsb=0) == UNSUP
    if fp8:
        assert f(ks=0.0) == ARG


def test_weights_workspace_size(pa_lib):
    f = pa_lib.pa_attention_weights_workspace_size
    assert f(-1, 4, 4, 2, 64, 1, 56) == 0 and f(4, 4, 6, 4, 64, 1, 56) == 0
    assert f(4, 4, 48, 4, 64, 1, 56) == 0
    a, b = f(4, 4, 4, 2, 64, 1, 56), f(4, 4, 4, 2, 64, 1, 5600)
    c = f(4, 400, 4, 2, 64, 100, 5600)
    assert 0 < a < b < c and a % 256 == 0 and c % 256 == 0


def evict(lib, **kw):
    a = dict(kc=FAKE, vc=FAKE, bt=FAKE, sl=FAKE, w=FAKE, nbt=FAKE, nsl=FAKE + 64, kept=FAKE,
             nw=FAKE + 64, R=4, hkv=2, d=64, eb=2, bs=16, nb=32, mb=8, mnb=2, ww=128, nww=32,
             ms=100, keep=20, recent=4, sinks=2)
    a.update(kw)
    return lib.pa_evict_kv(*[a[n] for n in ("kc", "vc", "bt", "sl", "w", "nbt", "nsl", "kept", "nw",
                                            "R", "hkv", "d", "eb", "bs", "nb", "mb", "mnb", "ww",
                                            "nww", "ms", "keep", "recent", "sinks")], None)


def test_evict(pa_lib):
    def f(**kw):
        return evict(pa_lib, **kw)
    for name in ("kc", "vc", "bt", "sl", "w", "nbt", "nsl", "kept"):
        assert f(**{name: None}) == ARG, name
    assert f(kc=FAKE + 8) == ARG and f(vc=FAKE + 8) == ARG and f(kept=FAKE + 2) == ARG
    assert f(nsl=FAKE) == ARG                    # seq_lens itself
    assert f(nw=FAKE) == ARG                     # weights themselves
    assert f(keep=0) == ARG and f(recent=-1) == ARG and f(sinks=-1) == ARG
    assert f(recent=19) == ARG and f(recent=2 ** 31 - 1, sinks=2 ** 31 - 1) == ARG
    assert f(keep=33, nww=64) == ARG             # three blocks, two given
    assert f(nww=19) == ARG and f(R=-1) == ARG and f(hkv=0) == ARG
    assert f(d=96) == UNSUP and f(bs=32) == UNSUP and f(eb=4) == UNSUP
    assert f(R=2 ** 30, keep=2 ** 20, mnb=2 ** 17, nww=2 ** 21) == UNSUP
    assert f(R=0, kc=None) == OK


def test_struct_forms(pa_lib):
    """The packed layouts match, and the struct forms refuse what the calls do."""
    binding.lib()  # checks pa_args_size against every layout
    assert pa_lib.pa_args_size(4) == 0
    for name in binding._ARGS:
        assert getattr(pa_lib, name)(None) == ARG
    assert pa_lib.pa_evict_kv_args(binding._pack_evict(
        FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE + 64, FAKE, FAKE + 64, 0, 128, 32, 4, 2, 64, 2, 16,
        32, 8, 2, 100, 0, 4, 2)) == ARG          # keep 0
    assert pa_lib.pa_evict_kv_args(binding._pack_evict(
        FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE + 64, FAKE, FAKE + 64, 0, 128, 32, 0, 2, 64, 2, 16,
        32, 8, 2, 100, 20, 4, 2)) == OK          # no request
    assert pa_lib.pa_attention_window_args(binding._pack_win(
        FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 0, 0, 0.1, 1.0, 1.0, 0, 4, 4, 4, 2, 64, 16,
        32, 4, 1, 56, 0, 4)) == ARG              # window 0
    assert pa_lib.pa_attention_window_args(binding._pack_win(
        FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 0, 0, 0.1, 1.0, 1.0, 0, 4, 4, 4, 2, 64, 16,
        32, 4, 1, 56, 16, 4)) == WS              # no workspace bytes
    assert pa_lib.pa_attention_weights_args(binding._pack_wts(
        FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 0, 0, 64, 0.1, 0.0, 1, 4, 4, 4, 2, 64, 16,
        32, 4, 1, 56)) == ARG                    # a scale of 0 for an E4M3 cache
    assert pa_lib.pa_norm_rope_write_kv_args(binding._pack_nr(
        FAKE, FAKE, FAKE, FAKE, FAKE, 0, 0, FAKE, FAKE, FAKE, FAKE, 0, 256, 128, 128, 1e-6, 1.0,
        1.0, 24, 0, 10, 0, 4, 4, 2, 64, 16, 8)) == UNSUP  # rotary_dim 24


def test_binding_refuses_cpu_tensors():
    import torch
    if torch.cuda.is_available():
        pytest.skip("checks the way without a GPU")
    z = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    with pytest.raises((RuntimeError, AssertionError, ValueError)):
        binding.norm_rope_write_kv(z, z[:, :2], z[:, :2], None, None, torch.zeros(2).long(),
                                   z.view(1, 2, 4, 64), z.view(1, 2, 4, 64))


def test_ctypes_signatures_cover_the_header(pa_lib):
    for name in ("pa_norm_rope_write_kv", "pa_norm_rope_write_kv_fp8", "pa_attention_window",
                 "pa_attention_window_fp8", "pa_attention_weights", "pa_attention_weights_fp8",
                 "pa_evict_kv"):
        assert getattr(pa_lib, name).argtypes[-1] is ctypes.c_void_p  # the stream
