"""Python binding of libpagedattn (ctypes): argument marshalling only.

Every step of the path runs in the library's CUDA kernels; this module checks
tensor dtypes/devices, passes raw device pointers and the current CUDA stream
through the C ABI declared in ``include/pa_api.h``, and turns a non-zero status
into an exception. There is no fallback: if the compiled library is missing
the import-time loader raises.

Function names follow the C ABI: ``pa_write_kv`` -> :func:`write_kv`,
``pa_attention`` -> :func:`attention`, and so on.

The attention calls also take a pinned CPU tensor as ``out``. It is passed by
its mapped device address (``pa_mapped_pointer``), and the kernels store the
result straight into host memory. That overlaps the device-to-host transfer
with the computation::

    host_out = torch.empty(q.shape, dtype=torch.bfloat16).pin_memory()
    attention(q, k_cache, v_cache, block_tables, seq_lens, qsl, scale,
              max_query_len=1, max_seq_len=L, out=host_out)
    torch.cuda.current_stream().synchronize()  # host_out now holds the result
"""
from __future__ import annotations

import ctypes
import os
import struct

import torch

from . import build as _build

_LIB = None

_c_p = ctypes.c_void_p
_c_i = ctypes.c_int
_INT_MAX = 2 ** 31 - 1  # counts beyond it mean the same as it
_BF16, _U8, _I32, _I64 = torch.bfloat16, torch.uint8, torch.int32, torch.int64

STATUS = {0: "PA_OK", -1: "PA_ERR_INVALID_ARG", -2: "PA_ERR_UNSUPPORTED",
          -3: "PA_ERR_WORKSPACE", -4: "PA_ERR_CUDA", -5: "PA_ERR_BOUNDS", -6: "PA_ERR_TIMEOUT"}
DEVICE_ERRORS = {0: "none", 1: "slot outside the pool", 2: "block id outside the pool",
                 3: "inconsistent lengths", 4: "query_start_loc out of range",
                 5: "bounded wait timed out", 6: "table does not start with the common prefix",
                 7: "position outside the rotation table"}
KERNEL_IDS = {"write_kv": 0, "plan": 1, "decode": 2, "prefill": 3, "prefix": 4, "merge": 5,
              "weights": 6, "evict": 7, "read": 8}


class PagedAttentionError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {STATUS.get(status, status)}")
        self.status = status


def library_path() -> str:
    return _build.LIB_PATH


def lib() -> ctypes.CDLL:
    """The loaded library; raises if it has not been built."""
    global _LIB
    if _LIB is None:
        path = library_path()
        if not os.path.exists(path):
            raise RuntimeError(
                f"{path} is missing: build it with `python -m paged_kv_cache_42_gb300.build` "
                "(there is no CPU fallback)")
        L = ctypes.CDLL(path)
        L.pa_init.argtypes = []
        L.pa_init.restype = _c_i
        L.pa_write_kv.argtypes = [_c_p, _c_p, _c_p, _c_p, _c_p, _c_i, _c_i, _c_i, _c_i, _c_i, _c_p]
        L.pa_write_kv.restype = _c_i
        L.pa_attention_workspace_size.argtypes = [_c_i, _c_i, _c_i, _c_i, _c_i]
        L.pa_attention_workspace_size.restype = ctypes.c_size_t
        L.pa_attention.argtypes = [_c_p, _c_p, _c_p, _c_p, _c_p, _c_p, ctypes.c_float, _c_p,
                                   _c_i, _c_i, _c_i, _c_i, _c_i, _c_i, _c_i, _c_i, _c_i, _c_i,
                                   _c_p, ctypes.c_size_t, _c_p]
        L.pa_attention.restype = _c_i
        L.pa_attention_cascade_workspace_size.argtypes = [_c_i, _c_i, _c_i, _c_i, _c_i]
        L.pa_attention_cascade_workspace_size.restype = ctypes.c_size_t
        L.pa_attention_cascade.argtypes = [_c_p, _c_p, _c_p, _c_p, _c_p, _c_p, ctypes.c_float,
                                           _c_p, _c_i, _c_i, _c_i, _c_i, _c_i, _c_i, _c_i, _c_i,
                                           _c_i, _c_i, _c_i, _c_p, ctypes.c_size_t, _c_p]
        L.pa_attention_cascade.restype = _c_i
        L.pa_write_kv_fp8.argtypes = [_c_p, _c_p, _c_p, _c_p, _c_p, ctypes.c_float,
                                      ctypes.c_float, _c_i, _c_i, _c_i, _c_i, _c_i, _c_p]
        L.pa_write_kv_fp8.restype = _c_i
        L.pa_attention_fp8.argtypes = [_c_p, _c_p, _c_p, _c_p, _c_p, _c_p, ctypes.c_float,
                                       ctypes.c_float, ctypes.c_float, _c_p, _c_i, _c_i, _c_i,
                                       _c_i, _c_i, _c_i, _c_i, _c_i, _c_i, _c_i, _c_p,
                                       ctypes.c_size_t, _c_p]
        L.pa_attention_fp8.restype = _c_i
        _ll, _f = ctypes.c_longlong, ctypes.c_float
        nr = [_c_p, _c_p, _c_p, _ll, _ll, _ll, _c_p, _c_p, _c_p, _c_p, _f, _c_i, _c_i, _c_i, _c_p,
              _c_p, _c_p, _c_p]
        L.pa_norm_rope_write_kv.argtypes = nr + [_c_i] * 6 + [_c_p]
        L.pa_norm_rope_write_kv_fp8.argtypes = nr + [_f, _f] + [_c_i] * 6 + [_c_p]
        L.pa_attention_window.argtypes = ([_c_p] * 6 + [_f, _c_p] + [_c_i] * 12 +
                                          [_c_p, ctypes.c_size_t, _c_p])
        L.pa_attention_window_fp8.argtypes = ([_c_p] * 6 + [_f, _f, _f, _c_p] + [_c_i] * 12 +
                                              [_c_p, ctypes.c_size_t, _c_p])
        # the struct forms: one packed argument (see _ARGS)
        for i, (name, layout) in enumerate(_ARGS.items()):
            fn = getattr(L, name)
            fn.argtypes = [ctypes.c_char_p]
            fn.restype = _c_i
            if L.pa_args_size(i) != -(-layout.size // 8) * 8:
                raise RuntimeError(f"{name}: the library's argument struct has another layout")
        for i, (name, layout) in enumerate(_ARGS2.items()):
            fn = getattr(L, name)
            fn.argtypes = [ctypes.c_char_p]
            fn.restype = _c_i
            if L.pa_args_size(16 + i) != -(-layout.size // 8) * 8:
                raise RuntimeError(f"{name}: the library's argument struct has another layout")
        L.pa_attention_shared_workspace_size.argtypes = [_c_i] * 7
        L.pa_attention_shared_workspace_size.restype = ctypes.c_size_t
        L.pa_attention_weights_workspace_size.argtypes = [_c_i] * 7
        L.pa_attention_weights_workspace_size.restype = ctypes.c_size_t
        L.pa_attention_weights.argtypes = ([_c_p] * 5 + [_f, _c_p, _c_p, _ll] + [_c_i] * 10 +
                                           [_c_p, ctypes.c_size_t, _c_p])
        L.pa_attention_weights.restype = _c_i
        L.pa_attention_weights_fp8.argtypes = ([_c_p] * 5 + [_f, _f, _c_p, _c_p, _ll] +
                                               [_c_i] * 10 + [_c_p, ctypes.c_size_t, _c_p])
        L.pa_attention_weights_fp8.restype = _c_i
        L.pa_evict_kv.argtypes = [_c_p] * 9 + [_c_i] * 8 + [_ll, _ll] + [_c_i] * 4 + [_c_p]
        L.pa_evict_kv.restype = _c_i
        L.pa_status_string.argtypes = [_c_i]
        L.pa_status_string.restype = ctypes.c_char_p
        L.pa_get_device_error.argtypes = [ctypes.POINTER(_c_i), ctypes.POINTER(ctypes.c_longlong),
                                          _c_i]
        L.pa_get_device_error.restype = _c_i
        L.pa_set_kernel_timer.argtypes = [_c_i, _c_p, _c_p]
        L.pa_set_kernel_timer.restype = _c_i
        L.pa_mapped_pointer.argtypes = [_c_p, ctypes.POINTER(ctypes.c_void_p)]
        L.pa_mapped_pointer.restype = _c_i
        L.pa_launch_count.argtypes = []
        L.pa_launch_count.restype = ctypes.c_longlong
        L.pa_version.argtypes = []
        L.pa_version.restype = _c_i
        _LIB = L
    return _LIB


# The argument structs of include/pa_api.h, packed with one call instead of a
# ctypes conversion per argument (25 of them take longer than a small kernel).
_ARGS = {"pa_norm_rope_write_kv_args": struct.Struct("@12P3q3f10i"),
         "pa_attention_window_args": struct.Struct("@9PN3f13i"),
         "pa_attention_weights_args": struct.Struct("@9PNq2f11i"),
         "pa_evict_kv_args": struct.Struct("@10P2q12i")}
_pack_nr, _pack_win, _pack_wts, _pack_evict = (s.pack for s in _ARGS.values())
# The calls that take a struct only.
_ARGS2 = {"pa_write_kv_rows": struct.Struct("@7P2q5i"),
          "pa_norm_rope_write_kv_rows": struct.Struct("@13P3qf9i"),
          "pa_attention_rows": struct.Struct("@10PNf10i"),
          "pa_read_kv": struct.Struct("@9P2f8i"),
          "pa_attention_shared": struct.Struct("@12PN3f13i")}
_pack_wr, _pack_nrr, _pack_ar, _pack_read, _pack_sh = (s.pack for s in _ARGS2.values())


def _check(status: int, what: str) -> None:
    if status != 0:
        raise PagedAttentionError(status, what)


def _stream_ptr(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream)


def _dev(t: torch.Tensor, dtype, name: str) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _out(t: torch.Tensor) -> int:
    """Address of an output tensor: a CUDA tensor, or a pinned CPU tensor
    reached through its mapped device address (pa_mapped_pointer)."""
    if isinstance(t, torch.Tensor) and not t.is_cuda:
        if t.dtype != torch.bfloat16 or not t.is_contiguous():
            raise TypeError("out must be a contiguous bf16 tensor")
        if not t.is_pinned():
            raise ValueError("a host out tensor must be pinned")
        return mapped_pointer(t)
    return _dev(t, torch.bfloat16, "out")


def mapped_pointer(t: torch.Tensor) -> int:
    """pa_mapped_pointer: the device address of a pinned host tensor."""
    dp = ctypes.c_void_p()
    _check(lib().pa_mapped_pointer(t.data_ptr(), ctypes.byref(dp)), "pa_mapped_pointer")
    return int(dp.value)


def status_string(status: int) -> str:
    return lib().pa_status_string(status).decode()


def init() -> None:
    _check(lib().pa_init(), "pa_init")


def write_kv(k: torch.Tensor, v: torch.Tensor, slot_mapping: torch.Tensor,
             k_cache: torch.Tensor, v_cache: torch.Tensor, stream=None) -> None:
    """pa_write_kv: scatter k/v [T, Hkv, D] into caches [num_blocks, Hkv, 16, D]."""
    T, hkv, d = k.shape
    nb, hkv2, bs, d2 = k_cache.shape
    if v.shape != k.shape or v_cache.shape != k_cache.shape or hkv2 != hkv or d2 != d:
        raise ValueError("shape mismatch between k/v and the caches")
    if slot_mapping.shape != (T,):
        raise ValueError("slot_mapping must be [num_tokens]")
    st = lib().pa_write_kv(_dev(k, torch.bfloat16, "k"), _dev(v, torch.bfloat16, "v"),
                           _dev(slot_mapping, torch.int64, "slot_mapping"),
                           _dev(k_cache, torch.bfloat16, "k_cache"),
                           _dev(v_cache, torch.bfloat16, "v_cache"), T, hkv, d, bs, nb,
                           _stream_ptr(stream))
    _check(st, "pa_write_kv")


def _refuse(t, dtype, dev: int, name: str):
    """Say what is wrong with a tensor that _ptr did not take."""
    _dev(t, dtype, name)
    raise ValueError(f"{name} is on {t.device}; the current device is cuda:{dev}, where the "
                     "kernels run")


def _ptr(t: torch.Tensor, dtype, dev: int, name: str) -> int:
    """Address of a contiguous tensor of the current device (a launch goes
    there, whatever device a tensor lives on). The checks of a call cost more
    host time than a small kernel takes, so this is the short way of _dev."""
    try:
        if t.dtype is dtype and t.get_device() == dev and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    return _refuse(t, dtype, dev, name)


def _where(stream) -> tuple[int, int]:
    """(current device, raw stream)."""
    if not torch.cuda.is_initialized():
        torch.cuda.init()
    dev = torch._C._cuda_getDevice()
    if stream is None:
        return dev, torch._C._cuda_getCurrentRawStream(dev)
    return dev, int(stream.cuda_stream)


def _empty(shape, dtype, device, stream) -> torch.Tensor:
    """Memory for a call on `stream`, from that stream's own: the allocator may
    hand memory of another one to later work there while this call still runs."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _heads(t: torch.Tensor, shape: tuple, dev: int, name: str) -> tuple[int, int]:
    """(address, token stride in elements) of [tokens, heads, head_dim] whose
    tokens may lie apart (a part of a wider projection)."""
    try:
        if t.dtype is _BF16 and t.shape == shape and t.get_device() == dev:
            s0, s1, s2 = t.stride()
            if s2 == 1 and (s1 == shape[2] or shape[1] == 1):
                return t.data_ptr(), (s0 if shape[0] > 1 else shape[1] * shape[2])
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name} must be torch.bfloat16, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"shape mismatch: {name} is {tuple(t.shape)}, not {shape}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be a CUDA tensor on the current device cuda:{dev}")
    raise ValueError(f"the heads of a token of {name} must be contiguous")


def _scales(t: torch.Tensor, cache_shape, dev: int) -> int:
    """Address of a row-scaled cache's scale bytes."""
    at = _ptr(t, _U8, dev, "scales")
    if t.shape != (cache_shape[0], cache_shape[1], 2, 16):
        raise ValueError("scales must be [num_blocks, Hkv, 2, 16]")
    return at


def _norm_rope(q, k, v, positions, cos_sin, slot_mapping, k_cache, v_cache, q_weight, k_weight,
               eps, interleaved, out, fp8, k_scale, v_scale, stream, scales=None):
    T, hq, d = qshape = q.shape
    cshape = k_cache.shape
    nb, hkv, bs, d2 = cshape
    if v_cache.shape != cshape or d2 != d:
        raise ValueError("shape mismatch between q and the caches")
    dev, raw_stream = _where(stream)
    rot = max_pos = pos_p = cs_p = qw_p = kw_p = 0
    if cos_sin is not None:
        if positions is None:
            raise ValueError("positions and cos_sin come together")
        max_pos, rot = cos_sin.shape
        pos_p = _ptr(positions, torch.int32, dev, "positions")
        cs_p = _ptr(cos_sin, torch.float32, dev, "cos_sin")
        if positions.numel() != T:
            raise ValueError("positions must be [num_tokens]")
    elif positions is not None:
        raise ValueError("positions and cos_sin come together")
    if q_weight is not None:
        qw_p = _ptr(q_weight, torch.bfloat16, dev, "q_weight")
        if q_weight.numel() != d:
            raise ValueError("a norm weight must be [head_dim]")
    if k_weight is not None:
        kw_p = _ptr(k_weight, torch.bfloat16, dev, "k_weight")
        if k_weight.numel() != d:
            raise ValueError("a norm weight must be [head_dim]")
    if out is None:
        out = _empty(qshape, torch.bfloat16, q.device, stream)
    elif out.shape != qshape:
        raise ValueError("out must have q's shape")
    qp, qs = _heads(q, qshape, dev, "q")
    kshape = (T, hkv, d)
    kp, ks = _heads(k, kshape, dev, "k")
    vp, vs = _heads(v, kshape, dev, "v")
    sp = _ptr(slot_mapping, torch.int64, dev, "slot_mapping")
    if slot_mapping.numel() != T:
        raise ValueError("slot_mapping must be [num_tokens]")
    cache_dtype = torch.uint8 if fp8 else torch.bfloat16
    if fp8 == 2:
        st = lib().pa_norm_rope_write_kv_rows(_pack_nrr(
            qp, kp, vp, pos_p, cs_p, qw_p, kw_p, sp, _ptr(out, torch.bfloat16, dev, "out"),
            _ptr(k_cache, cache_dtype, dev, "k_cache"), _ptr(v_cache, cache_dtype, dev, "v_cache"),
            _scales(scales, cshape, dev), raw_stream, qs, ks, vs, eps, rot,
            1 if interleaved else 0, max_pos, T, hq, hkv, d, bs, nb))
        if st:
            _check(st, "pa_norm_rope_write_kv_rows")
        return out
    st = lib().pa_norm_rope_write_kv_args(_pack_nr(
        qp, kp, vp, pos_p, cs_p, qw_p, kw_p, sp, _ptr(out, torch.bfloat16, dev, "out"),
        _ptr(k_cache, cache_dtype, dev, "k_cache"), _ptr(v_cache, cache_dtype, dev, "v_cache"),
        raw_stream, qs, ks, vs, eps, k_scale, v_scale, rot, 1 if interleaved else 0, max_pos, fp8,
        T, hq, hkv, d, bs, nb))
    if st:
        _check(st, "pa_norm_rope_write_kv_fp8" if fp8 else "pa_norm_rope_write_kv")
    return out


def norm_rope_write_kv(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                       positions: torch.Tensor | None, cos_sin: torch.Tensor | None,
                       slot_mapping: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                       *, q_weight: torch.Tensor | None = None,
                       k_weight: torch.Tensor | None = None, eps: float = 1e-6,
                       interleaved: bool = False, out: torch.Tensor | None = None,
                       stream=None) -> torch.Tensor:
    """pa_norm_rope_write_kv: norm and rotate the heads of q [T, Hq, D] and k
    [T, Hkv, D], scatter k and v into the caches, return the queries [T, Hq, D].

    q, k and v may be views into one projection's output (tokens apart, a
    token's heads contiguous). ``cos_sin`` is fp32 [max_position, rotary_dim],
    cosines then sines; ``positions`` is int32 [T]; both None: no rotation.
    """
    return _norm_rope(q, k, v, positions, cos_sin, slot_mapping, k_cache, v_cache, q_weight,
                      k_weight, eps, interleaved, out, 0, 1.0, 1.0, stream)


def norm_rope_write_kv_fp8(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                           positions: torch.Tensor | None, cos_sin: torch.Tensor | None,
                           slot_mapping: torch.Tensor, k_cache: torch.Tensor,
                           v_cache: torch.Tensor, k_scale: float, v_scale: float, *,
                           q_weight: torch.Tensor | None = None,
                           k_weight: torch.Tensor | None = None, eps: float = 1e-6,
                           interleaved: bool = False, out: torch.Tensor | None = None,
                           stream=None) -> torch.Tensor:
    """pa_norm_rope_write_kv_fp8: the same into E4M3 caches (uint8)."""
    return _norm_rope(q, k, v, positions, cos_sin, slot_mapping, k_cache, v_cache, q_weight,
                      k_weight, eps, interleaved, out, 1, k_scale, v_scale, stream)


def workspace_size(num_reqs: int, num_tokens: int, num_q_heads: int, num_kv_heads: int,
                   head_dim: int) -> int:
    return int(lib().pa_attention_workspace_size(num_reqs, num_tokens, num_q_heads,
                                                 num_kv_heads, head_dim))


def attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
              block_tables: torch.Tensor, seq_lens: torch.Tensor,
              query_start_loc: torch.Tensor, scale: float, *, max_query_len: int,
              max_seq_len: int, out: torch.Tensor | None = None,
              workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """pa_attention for a mixed batch; returns ``out`` [T, Hq, D] bf16.

    ``workspace`` (uint8, >= workspace_size(...) bytes) is allocated here with
    torch if not given; pass a persistent one on hot loops.
    """
    T, hq, d = q.shape
    nb, hkv, bs, d2 = k_cache.shape
    R = int(seq_lens.shape[0])
    if d2 != d or v_cache.shape != k_cache.shape:
        raise ValueError("shape mismatch between q and the caches")
    if query_start_loc.shape != (R + 1,) or block_tables.dim() != 2 or block_tables.shape[0] != R:
        raise ValueError("metadata shapes must be qsl [R+1], block_tables [R, max_blocks]")
    if out is None:
        out = torch.empty_like(q)
    need = workspace_size(R, T, hq, hkv, d)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    st = lib().pa_attention(
        _dev(q, torch.bfloat16, "q"), _dev(k_cache, torch.bfloat16, "k_cache"),
        _dev(v_cache, torch.bfloat16, "v_cache"), _dev(block_tables, torch.int32, "block_tables"),
        _dev(seq_lens, torch.int32, "seq_lens"),
        _dev(query_start_loc, torch.int32, "query_start_loc"), float(scale),
        _out(out), R, T, hq, hkv, d, bs, nb, int(block_tables.shape[1]),
        int(max_query_len), int(max_seq_len), _dev(workspace, torch.uint8, "workspace"),
        int(workspace.numel()), _stream_ptr(stream))
    _check(st, "pa_attention")
    return out


def write_kv_fp8(k: torch.Tensor, v: torch.Tensor, slot_mapping: torch.Tensor,
                 k_cache: torch.Tensor, v_cache: torch.Tensor, k_scale: float, v_scale: float,
                 stream=None) -> None:
    """pa_write_kv_fp8: quantise k/v [T, Hkv, D] bf16 into E4M3 caches
    [num_blocks, Hkv, 16, D] (uint8) with per-tensor scales."""
    T, hkv, d = k.shape
    nb, hkv2, bs, d2 = k_cache.shape
    if v.shape != k.shape or v_cache.shape != k_cache.shape or hkv2 != hkv or d2 != d:
        raise ValueError("shape mismatch between k/v and the caches")
    if slot_mapping.shape != (T,):
        raise ValueError("slot_mapping must be [num_tokens]")
    st = lib().pa_write_kv_fp8(_dev(k, torch.bfloat16, "k"), _dev(v, torch.bfloat16, "v"),
                               _dev(slot_mapping, torch.int64, "slot_mapping"),
                               _dev(k_cache, torch.uint8, "k_cache"),
                               _dev(v_cache, torch.uint8, "v_cache"), float(k_scale),
                               float(v_scale), T, hkv, d, bs, nb, _stream_ptr(stream))
    _check(st, "pa_write_kv_fp8")


def attention_fp8(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                  block_tables: torch.Tensor, seq_lens: torch.Tensor,
                  query_start_loc: torch.Tensor, scale: float, k_scale: float, v_scale: float,
                  *, max_query_len: int, max_seq_len: int, out: torch.Tensor | None = None,
                  workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """pa_attention_fp8 over E4M3 caches (uint8 [num_blocks, Hkv, 16, D])."""
    T, hq, d = q.shape
    nb, hkv, bs, d2 = k_cache.shape
    R = int(seq_lens.shape[0])
    if d2 != d or v_cache.shape != k_cache.shape:
        raise ValueError("shape mismatch between q and the caches")
    if query_start_loc.shape != (R + 1,) or block_tables.dim() != 2 or block_tables.shape[0] != R:
        raise ValueError("metadata shapes must be qsl [R+1], block_tables [R, max_blocks]")
    if out is None:
        out = torch.empty_like(q)
    need = workspace_size(R, T, hq, hkv, d)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    st = lib().pa_attention_fp8(
        _dev(q, torch.bfloat16, "q"), _dev(k_cache, torch.uint8, "k_cache"),
        _dev(v_cache, torch.uint8, "v_cache"), _dev(block_tables, torch.int32, "block_tables"),
        _dev(seq_lens, torch.int32, "seq_lens"),
        _dev(query_start_loc, torch.int32, "query_start_loc"), float(scale), float(k_scale),
        float(v_scale), _out(out), R, T, hq, hkv, d, bs, nb,
        int(block_tables.shape[1]), int(max_query_len), int(max_seq_len),
        _dev(workspace, torch.uint8, "workspace"), int(workspace.numel()), _stream_ptr(stream))
    _check(st, "pa_attention_fp8")
    return out


def cascade_workspace_size(num_reqs: int, num_tokens: int, num_q_heads: int, num_kv_heads: int,
                           head_dim: int) -> int:
    return int(lib().pa_attention_cascade_workspace_size(num_reqs, num_tokens, num_q_heads,
                                                         num_kv_heads, head_dim))


def attention_cascade(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                      block_tables: torch.Tensor, seq_lens: torch.Tensor,
                      query_start_loc: torch.Tensor, scale: float, *, common_prefix_len: int,
                      max_query_len: int, max_seq_len: int, out: torch.Tensor | None = None,
                      workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """pa_attention_cascade: every request shares the first ``common_prefix_len``
    keys (the same blocks); the prefix is attended once for the whole batch."""
    T, hq, d = q.shape
    nb, hkv, bs, d2 = k_cache.shape
    R = int(seq_lens.shape[0])
    if d2 != d or v_cache.shape != k_cache.shape:
        raise ValueError("shape mismatch between q and the caches")
    if query_start_loc.shape != (R + 1,) or block_tables.dim() != 2 or block_tables.shape[0] != R:
        raise ValueError("metadata shapes must be qsl [R+1], block_tables [R, max_blocks]")
    if out is None:
        out = torch.empty_like(q)
    need = cascade_workspace_size(R, T, hq, hkv, d)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    st = lib().pa_attention_cascade(
        _dev(q, torch.bfloat16, "q"), _dev(k_cache, torch.bfloat16, "k_cache"),
        _dev(v_cache, torch.bfloat16, "v_cache"), _dev(block_tables, torch.int32, "block_tables"),
        _dev(seq_lens, torch.int32, "seq_lens"),
        _dev(query_start_loc, torch.int32, "query_start_loc"), float(scale),
        _out(out), R, T, hq, hkv, d, bs, nb, int(block_tables.shape[1]),
        int(max_query_len), int(max_seq_len), int(common_prefix_len),
        _dev(workspace, torch.uint8, "workspace"), int(workspace.numel()), _stream_ptr(stream))
    _check(st, "pa_attention_cascade")
    return out


def _window(q, k_cache, v_cache, block_tables, seq_lens, query_start_loc, scale, window, sinks,
            max_query_len, max_seq_len, out, workspace, fp8, k_scale, v_scale, stream):
    T, hq, d = qshape = q.shape
    cshape = k_cache.shape
    nb, hkv, bs, d2 = cshape
    R = seq_lens.shape[0]
    if d2 != d or v_cache.shape != cshape:
        raise ValueError("shape mismatch between q and the caches")
    mr, mb = block_tables.shape
    if query_start_loc.numel() != R + 1 or mr != R:
        raise ValueError("metadata shapes must be qsl [R+1], block_tables [R, max_blocks]")
    if out is None:
        out = _empty(qshape, torch.bfloat16, q.device, stream)
    elif out.shape != qshape:
        raise ValueError("out must have q's shape")
    if workspace is None:
        need = workspace_size(R, T, hq, hkv, d)
        workspace = _empty(max(need, 256), torch.uint8, q.device, stream)
    dev, raw_stream = _where(stream)
    out_p = _ptr(out, torch.bfloat16, dev, "out") if out.is_cuda else _out(out)
    cache_dtype = torch.uint8 if fp8 else torch.bfloat16
    st = lib().pa_attention_window_args(_pack_win(
        _ptr(q, torch.bfloat16, dev, "q"), _ptr(k_cache, cache_dtype, dev, "k_cache"),
        _ptr(v_cache, cache_dtype, dev, "v_cache"),
        _ptr(block_tables, torch.int32, dev, "block_tables"),
        _ptr(seq_lens, torch.int32, dev, "seq_lens"),
        _ptr(query_start_loc, torch.int32, dev, "query_start_loc"), out_p,
        _ptr(workspace, torch.uint8, dev, "workspace"), raw_stream, workspace.numel(), scale,
        k_scale, v_scale, fp8, R, T, hq, hkv, d, bs, nb, mb, max_query_len, max_seq_len,
        min(window, _INT_MAX), min(sinks, _INT_MAX)))
    if st:
        _check(st, "pa_attention_window_fp8" if fp8 else "pa_attention_window")
    return out


def attention_window(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                     block_tables: torch.Tensor, seq_lens: torch.Tensor,
                     query_start_loc: torch.Tensor, scale: float, *, window: int, sinks: int = 0,
                     max_query_len: int, max_seq_len: int, out: torch.Tensor | None = None,
                     workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """pa_attention_window: :func:`attention` where a token attends to the last
    ``window`` keys (its own included) and the first ``sinks``. The workspace is
    ``workspace_size(...)`` bytes, as for :func:`attention`."""
    return _window(q, k_cache, v_cache, block_tables, seq_lens, query_start_loc, scale, window,
                   sinks, max_query_len, max_seq_len, out, workspace, 0, 1.0, 1.0, stream)


def attention_window_fp8(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                         block_tables: torch.Tensor, seq_lens: torch.Tensor,
                         query_start_loc: torch.Tensor, scale: float, k_scale: float,
                         v_scale: float, *, window: int, sinks: int = 0, max_query_len: int,
                         max_seq_len: int, out: torch.Tensor | None = None,
                         workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """pa_attention_window_fp8: the same over E4M3 caches (uint8)."""
    return _window(q, k_cache, v_cache, block_tables, seq_lens, query_start_loc, scale, window,
                   sinks, max_query_len, max_seq_len, out, workspace, 1, k_scale, v_scale, stream)


def weights_workspace_size(num_reqs: int, num_tokens: int, num_q_heads: int, num_kv_heads: int,
                           head_dim: int, max_query_len: int, max_seq_len: int) -> int:
    return int(lib().pa_attention_weights_workspace_size(num_reqs, num_tokens, num_q_heads,
                                                         num_kv_heads, head_dim, max_query_len,
                                                         max_seq_len))


def _weights(q, k_cache, block_tables, seq_lens, query_start_loc, scale, weights, max_query_len,
             max_seq_len, out, workspace, fp8, k_scale, stream):
    T, hq, d = q.shape
    nb, hkv, bs, d2 = k_cache.shape
    R = seq_lens.shape[0]
    if d2 != d:
        raise ValueError("shape mismatch between q and the cache")
    mr, mb = block_tables.shape
    if query_start_loc.numel() != R + 1 or mr != R:
        raise ValueError("metadata shapes must be qsl [R+1], block_tables [R, max_blocks]")
    wshape = weights.shape
    if len(wshape) != 3 or wshape[0] != R or wshape[1] != hkv:
        raise ValueError("weights must be [num_reqs, num_kv_heads, width]")
    if out is None:
        out = weights
    elif out.shape != wshape:
        raise ValueError("out must have weights' shape")
    if workspace is None:
        need = weights_workspace_size(R, T, hq, hkv, d, max_query_len, max_seq_len)
        workspace = _empty(max(need, 256), torch.uint8, q.device, stream)
    dev, raw_stream = _where(stream)
    st = lib().pa_attention_weights_args(_pack_wts(
        _ptr(q, torch.bfloat16, dev, "q"),
        _ptr(k_cache, torch.uint8 if fp8 else torch.bfloat16, dev, "k_cache"),
        _ptr(block_tables, torch.int32, dev, "block_tables"),
        _ptr(seq_lens, torch.int32, dev, "seq_lens"),
        _ptr(query_start_loc, torch.int32, dev, "query_start_loc"),
        _ptr(weights, torch.float32, dev, "weights"), _ptr(out, torch.float32, dev, "out"),
        _ptr(workspace, torch.uint8, dev, "workspace"), raw_stream, workspace.numel(), wshape[2],
        scale, k_scale, fp8, R, T, hq, hkv, d, bs, nb, mb, max_query_len, max_seq_len))
    if st:
        _check(st, "pa_attention_weights_fp8" if fp8 else "pa_attention_weights")
    return out


def attention_weights(q: torch.Tensor, k_cache: torch.Tensor, block_tables: torch.Tensor,
                      seq_lens: torch.Tensor, query_start_loc: torch.Tensor, scale: float,
                      weights: torch.Tensor, *, max_query_len: int, max_seq_len: int,
                      out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                      stream=None) -> torch.Tensor:
    """pa_attention_weights: add this step's attention weight of every key,
    summed over the new tokens and the query heads of its KV head, to
    ``weights`` fp32 [R, Hkv, width >= seq_len]; in place unless ``out`` is given."""
    return _weights(q, k_cache, block_tables, seq_lens, query_start_loc, scale, weights,
                    max_query_len, max_seq_len, out, workspace, 0, 1.0, stream)


def attention_weights_fp8(q: torch.Tensor, k_cache: torch.Tensor, block_tables: torch.Tensor,
                          seq_lens: torch.Tensor, query_start_loc: torch.Tensor, scale: float,
                          k_scale: float, weights: torch.Tensor, *, max_query_len: int,
                          max_seq_len: int, out: torch.Tensor | None = None,
                          workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """pa_attention_weights_fp8: the same over an E4M3 key cache (uint8)."""
    return _weights(q, k_cache, block_tables, seq_lens, query_start_loc, scale, weights,
                    max_query_len, max_seq_len, out, workspace, 1, k_scale, stream)


def evict_kv(k_cache: torch.Tensor, v_cache: torch.Tensor, block_tables: torch.Tensor,
             seq_lens: torch.Tensor, weights: torch.Tensor, new_block_tables: torch.Tensor, *,
             keep: int, recent: int, sinks: int = 0, max_seq_len: int,
             new_seq_lens: torch.Tensor | None = None, kept: torch.Tensor | None = None,
             new_weights: torch.Tensor | None = None, stream=None):
    """pa_evict_kv: cut every request longer than ``keep`` to ``keep`` tokens per
    KV head (its first ``sinks``, last ``recent`` and heaviest others), copying
    the rows kept into the blocks of ``new_block_tables`` [R, >= ceil(keep / 16)].

    ``weights`` is fp32 [R, Hkv, width] (:func:`attention_weights`). Returns
    ``(new_seq_lens [R] int32, kept [R, Hkv, keep] int32, new_weights
    [R, Hkv, >= keep] fp32)``; given buffers are filled, missing ones allocated.
    Requests of at most ``keep`` tokens stay in their old blocks: their rows of
    ``kept`` and ``new_weights`` are not written.
    """
    nb, hkv, bs, d = k_cache.shape
    R = int(seq_lens.shape[0])
    if v_cache.shape != k_cache.shape or v_cache.dtype != k_cache.dtype:
        raise ValueError("the caches must be alike")
    if k_cache.dtype not in (torch.bfloat16, torch.uint8):
        raise TypeError("a cache must be torch.bfloat16 or torch.uint8 (E4M3 codes)")
    if weights.dim() != 3 or weights.shape[:2] != (R, hkv):
        raise ValueError("weights must be [num_reqs, num_kv_heads, width]")
    for t in (block_tables, new_block_tables):
        if t.dim() != 2 or t.shape[0] != R:
            raise ValueError("block tables must be [num_reqs, blocks]")
    if new_seq_lens is None:
        new_seq_lens = _empty(R, torch.int32, k_cache.device, stream)
    if kept is None:
        kept = _empty((R, hkv, max(keep, 0)), torch.int32, k_cache.device, stream)
    if new_weights is None:
        new_weights = _empty((R, hkv, max(keep, 0)), torch.float32, k_cache.device, stream)
    if new_seq_lens.shape != (R,) or kept.shape != (R, hkv, keep) or \
            new_weights.dim() != 3 or new_weights.shape[:2] != (R, hkv):
        raise ValueError("new_seq_lens must be [R], kept [R, Hkv, keep], new_weights [R, Hkv, width]")
    dev, raw_stream = _where(stream)
    st = lib().pa_evict_kv_args(_pack_evict(
        _ptr(k_cache, k_cache.dtype, dev, "k_cache"), _ptr(v_cache, k_cache.dtype, dev, "v_cache"),
        _ptr(block_tables, torch.int32, dev, "block_tables"),
        _ptr(seq_lens, torch.int32, dev, "seq_lens"), _ptr(weights, torch.float32, dev, "weights"),
        _ptr(new_block_tables, torch.int32, dev, "new_block_tables"),
        _ptr(new_seq_lens, torch.int32, dev, "new_seq_lens"), _ptr(kept, torch.int32, dev, "kept"),
        _ptr(new_weights, torch.float32, dev, "new_weights"), raw_stream, weights.shape[2],
        new_weights.shape[2], R, hkv, d, k_cache.element_size(), bs, nb, block_tables.shape[1],
        new_block_tables.shape[1], max_seq_len, keep, min(recent, _INT_MAX), min(sinks, _INT_MAX)))
    if st:
        _check(st, "pa_evict_kv")
    return new_seq_lens, kept, new_weights


def _like_cache(k_cache, v_cache, d: int | None = None):
    """The common shape of two caches [num_blocks, Hkv, 16, D]."""
    shape = k_cache.shape
    if len(shape) != 4 or v_cache.shape != shape or (d is not None and shape[3] != d):
        raise ValueError("shape mismatch between the caches" + ("" if d is None else " and q"))
    return shape


def write_kv_rows(k: torch.Tensor, v: torch.Tensor, slot_mapping: torch.Tensor,
                  k_cache: torch.Tensor, v_cache: torch.Tensor, scales: torch.Tensor, *,
                  stream=None) -> None:
    """pa_write_kv_rows: scatter k/v [T, Hkv, D] bf16 into a row-scaled cache: E4M3
    codes (uint8 [num_blocks, Hkv, 16, D]) and a power of two for every row, which
    the call finds (uint8 ``scales`` [num_blocks, Hkv, 2, 16]: K's, then V's; b
    stands for 2^(b - 127)). k and v may be views into one projection's output.
    """
    nb, hkv, bs, d = cshape = _like_cache(k_cache, v_cache)
    T = k.shape[0]
    dev, raw_stream = _where(stream)
    shape = (T, hkv, d)
    kp, ks = _heads(k, shape, dev, "k")
    vp, vs = _heads(v, shape, dev, "v")
    sp = _ptr(slot_mapping, _I64, dev, "slot_mapping")
    if slot_mapping.numel() != T:
        raise ValueError("slot_mapping must be [num_tokens]")
    st = lib().pa_write_kv_rows(_pack_wr(
        kp, vp, sp, _ptr(k_cache, _U8, dev, "k_cache"), _ptr(v_cache, _U8, dev, "v_cache"),
        _scales(scales, cshape, dev), raw_stream, ks, vs, T, hkv, d, bs, nb))
    if st:
        _check(st, "pa_write_kv_rows")


def norm_rope_write_kv_rows(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                            positions: torch.Tensor | None, cos_sin: torch.Tensor | None,
                            slot_mapping: torch.Tensor, k_cache: torch.Tensor,
                            v_cache: torch.Tensor, scales: torch.Tensor, *,
                            q_weight: torch.Tensor | None = None,
                            k_weight: torch.Tensor | None = None, eps: float = 1e-6,
                            interleaved: bool = False, out: torch.Tensor | None = None,
                            stream=None) -> torch.Tensor:
    """pa_norm_rope_write_kv_rows: :func:`norm_rope_write_kv` into a row-scaled cache
    (see :func:`write_kv_rows`)."""
    return _norm_rope(q, k, v, positions, cos_sin, slot_mapping, k_cache, v_cache, q_weight,
                      k_weight, eps, interleaved, out, 2, 1.0, 1.0, stream, scales)


def attention_rows(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                   scales: torch.Tensor, block_tables: torch.Tensor, seq_lens: torch.Tensor,
                   query_start_loc: torch.Tensor, scale: float, *, max_query_len: int,
                   max_seq_len: int, out: torch.Tensor | None = None,
                   workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """pa_attention_rows: :func:`attention` over a row-scaled cache (see
    :func:`write_kv_rows`). The workspace is ``workspace_size(...)`` bytes."""
    T, hq, d = qshape = q.shape
    cshape = _like_cache(k_cache, v_cache, d)
    nb, hkv, bs, _ = cshape
    R = seq_lens.shape[0]
    mr, mb = block_tables.shape
    if query_start_loc.numel() != R + 1 or mr != R:
        raise ValueError("metadata shapes must be qsl [R+1], block_tables [R, max_blocks]")
    if out is None:
        out = _empty(qshape, torch.bfloat16, q.device, stream)
    elif out.shape != qshape:
        raise ValueError("out must have q's shape")
    if workspace is None:
        need = workspace_size(R, T, hq, hkv, d)
        workspace = _empty(max(need, 256), torch.uint8, q.device, stream)
    dev, raw_stream = _where(stream)
    out_p = _ptr(out, torch.bfloat16, dev, "out") if out.is_cuda else _out(out)
    st = lib().pa_attention_rows(_pack_ar(
        _ptr(q, torch.bfloat16, dev, "q"), _ptr(k_cache, torch.uint8, dev, "k_cache"),
        _ptr(v_cache, torch.uint8, dev, "v_cache"), _scales(scales, cshape, dev),
        _ptr(block_tables, torch.int32, dev, "block_tables"),
        _ptr(seq_lens, torch.int32, dev, "seq_lens"),
        _ptr(query_start_loc, torch.int32, dev, "query_start_loc"), out_p,
        _ptr(workspace, torch.uint8, dev, "workspace"), raw_stream, workspace.numel(), scale, R, T,
        hq, hkv, d, bs, nb, mb, max_query_len, max_seq_len))
    if st:
        _check(st, "pa_attention_rows")
    return out


def _read(k_cache, v_cache, scales, block_tables, read_start_loc, first, num_tokens, k_out, v_out,
          fmt, k_scale, v_scale, stream):
    cshape = _like_cache(k_cache, v_cache)
    nb, hkv, bs, d = cshape
    R, mb = block_tables.shape
    if read_start_loc.numel() != R + 1:
        raise ValueError("read_start_loc must be [num_reqs + 1]")
    if num_tokens is None:
        if k_out is None and v_out is None:
            raise ValueError("give num_tokens, or k_out and v_out")
        num_tokens = (v_out if k_out is None else k_out).shape[0]
    shape = (num_tokens, hkv, d)
    if k_out is None:
        k_out = _empty(shape, torch.bfloat16, k_cache.device, stream)
    if v_out is None:
        v_out = _empty(shape, torch.bfloat16, k_cache.device, stream)
    if k_out.shape != shape or v_out.shape != shape:
        raise ValueError("k_out and v_out must be [num_tokens, Hkv, D]")
    dev, raw_stream = _where(stream)
    first_p = 0
    if first is not None:
        first_p = _ptr(first, torch.int32, dev, "first")
        if first.numel() != R:
            raise ValueError("first must be [num_reqs]")
    cache_dtype = torch.uint8 if fmt else torch.bfloat16
    st = lib().pa_read_kv(_pack_read(
        _ptr(k_cache, cache_dtype, dev, "k_cache"), _ptr(v_cache, cache_dtype, dev, "v_cache"),
        _scales(scales, cshape, dev) if fmt == 2 else 0,
        _ptr(block_tables, torch.int32, dev, "block_tables"),
        _ptr(read_start_loc, torch.int32, dev, "read_start_loc"), first_p,
        _ptr(k_out, torch.bfloat16, dev, "k_out"), _ptr(v_out, torch.bfloat16, dev, "v_out"),
        raw_stream, k_scale, v_scale, fmt, R, num_tokens, hkv, d, bs, nb, mb))
    if st:
        _check(st, "pa_read_kv")
    return k_out, v_out


def read_kv(k_cache: torch.Tensor, v_cache: torch.Tensor, block_tables: torch.Tensor,
            read_start_loc: torch.Tensor, *, first: torch.Tensor | None = None,
            num_tokens: int | None = None, k_out: torch.Tensor | None = None,
            v_out: torch.Tensor | None = None, stream=None):
    """pa_read_kv over a bf16 cache: dense copies [num_tokens, Hkv, D] of cached keys
    and values. Rows ``read_start_loc[r]`` .. ``read_start_loc[r + 1] - 1`` (int32
    [R + 1]) get request r's keys from ``first[r]`` (int32 [R]; None: 0) on. Returns
    ``(k_out, v_out)``; given buffers are filled, missing ones allocated.
    """
    return _read(k_cache, v_cache, None, block_tables, read_start_loc, first, num_tokens, k_out,
                 v_out, 0, 1.0, 1.0, stream)


def read_kv_fp8(k_cache: torch.Tensor, v_cache: torch.Tensor, block_tables: torch.Tensor,
                read_start_loc: torch.Tensor, k_scale: float, v_scale: float, *,
                first: torch.Tensor | None = None, num_tokens: int | None = None,
                k_out: torch.Tensor | None = None, v_out: torch.Tensor | None = None, stream=None):
    """pa_read_kv over an E4M3 cache (uint8) with one scale per tensor."""
    return _read(k_cache, v_cache, None, block_tables, read_start_loc, first, num_tokens, k_out,
                 v_out, 1, k_scale, v_scale, stream)


def read_kv_rows(k_cache: torch.Tensor, v_cache: torch.Tensor, scales: torch.Tensor,
                 block_tables: torch.Tensor, read_start_loc: torch.Tensor, *,
                 first: torch.Tensor | None = None, num_tokens: int | None = None,
                 k_out: torch.Tensor | None = None, v_out: torch.Tensor | None = None, stream=None):
    """pa_read_kv over a row-scaled cache (see :func:`write_kv_rows`)."""
    return _read(k_cache, v_cache, scales, block_tables, read_start_loc, first, num_tokens, k_out,
                 v_out, 2, 1.0, 1.0, stream)


def shared_workspace_size(num_reqs: int, num_tokens: int, num_q_heads: int, num_kv_heads: int,
                          head_dim: int, num_groups: int, max_prefix_len: int) -> int:
    return int(lib().pa_attention_shared_workspace_size(num_reqs, num_tokens, num_q_heads,
                                                        num_kv_heads, head_dim, num_groups,
                                                        max_prefix_len))


def _shared(q, k_cache, v_cache, scales, block_tables, seq_lens, query_start_loc, group_start_loc,
            prefix_lens, scale, max_prefix_len, max_query_len, max_seq_len, out, workspace, fmt,
            k_scale, v_scale, stream):
    T, hq, d = qshape = q.shape
    cshape = _like_cache(k_cache, v_cache, d)
    nb, hkv, bs, _ = cshape
    R = seq_lens.shape[0]
    mr, mb = block_tables.shape
    if query_start_loc.numel() != R + 1 or mr != R:
        raise ValueError("metadata shapes must be qsl [R+1], block_tables [R, max_blocks]")
    G = prefix_lens.numel()
    if group_start_loc.numel() != G + 1:
        raise ValueError("group_start_loc must be [num_groups + 1], prefix_lens [num_groups]")
    if out is None:
        out = _empty(qshape, torch.bfloat16, q.device, stream)
    elif out.shape != qshape:
        raise ValueError("out must have q's shape")
    if workspace is None:
        need = shared_workspace_size(R, T, hq, hkv, d, G, max_prefix_len)
        workspace = _empty(max(need, 256), torch.uint8, q.device, stream)
    dev, raw_stream = _where(stream)
    out_p = _ptr(out, torch.bfloat16, dev, "out") if out.is_cuda else _out(out)
    cache_dtype = torch.uint8 if fmt else torch.bfloat16
    st = lib().pa_attention_shared(_pack_sh(
        _ptr(q, torch.bfloat16, dev, "q"), _ptr(k_cache, cache_dtype, dev, "k_cache"),
        _ptr(v_cache, cache_dtype, dev, "v_cache"),
        _scales(scales, cshape, dev) if fmt == 2 else 0,
        _ptr(block_tables, torch.int32, dev, "block_tables"),
        _ptr(seq_lens, torch.int32, dev, "seq_lens"),
        _ptr(query_start_loc, torch.int32, dev, "query_start_loc"),
        _ptr(group_start_loc, torch.int32, dev, "group_start_loc"),
        _ptr(prefix_lens, torch.int32, dev, "prefix_lens"), out_p,
        _ptr(workspace, torch.uint8, dev, "workspace"), raw_stream, workspace.numel(), scale, k_scale,
        v_scale, fmt, R, T, hq, hkv, d, bs, nb, mb, max_query_len, max_seq_len, G, max_prefix_len))
    if st:
        _check(st, "pa_attention_shared")
    return out


def attention_shared(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                     block_tables: torch.Tensor, seq_lens: torch.Tensor,
                     query_start_loc: torch.Tensor, group_start_loc: torch.Tensor,
                     prefix_lens: torch.Tensor, scale: float, *, max_prefix_len: int,
                     max_query_len: int, max_seq_len: int, out: torch.Tensor | None = None,
                     workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """pa_attention_shared: :func:`attention` where requests ``group_start_loc[g]`` ..
    ``group_start_loc[g + 1] - 1`` (int32 [groups + 1]) share their first
    ``prefix_lens[g]`` keys (int32 [groups], multiples of 16, 0: none), the same blocks
    at the start of their tables; a prefix is attended to once for its group. The
    workspace is ``shared_workspace_size(...)`` bytes."""
    return _shared(q, k_cache, v_cache, None, block_tables, seq_lens, query_start_loc,
                   group_start_loc, prefix_lens, scale, max_prefix_len, max_query_len, max_seq_len,
                   out, workspace, 0, 1.0, 1.0, stream)


def attention_shared_fp8(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                         block_tables: torch.Tensor, seq_lens: torch.Tensor,
                         query_start_loc: torch.Tensor, group_start_loc: torch.Tensor,
                         prefix_lens: torch.Tensor, scale: float, k_scale: float, v_scale: float,
                         *, max_prefix_len: int, max_query_len: int, max_seq_len: int,
                         out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                         stream=None) -> torch.Tensor:
    """pa_attention_shared over E4M3 caches (uint8) with one scale per tensor."""
    return _shared(q, k_cache, v_cache, None, block_tables, seq_lens, query_start_loc,
                   group_start_loc, prefix_lens, scale, max_prefix_len, max_query_len, max_seq_len,
                   out, workspace, 1, k_scale, v_scale, stream)


def attention_shared_rows(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                          scales: torch.Tensor, block_tables: torch.Tensor, seq_lens: torch.Tensor,
                          query_start_loc: torch.Tensor, group_start_loc: torch.Tensor,
                          prefix_lens: torch.Tensor, scale: float, *, max_prefix_len: int,
                          max_query_len: int, max_seq_len: int, out: torch.Tensor | None = None,
                          workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """pa_attention_shared over a row-scaled cache (see :func:`write_kv_rows`)."""
    return _shared(q, k_cache, v_cache, scales, block_tables, seq_lens, query_start_loc,
                   group_start_loc, prefix_lens, scale, max_prefix_len, max_query_len, max_seq_len,
                   out, workspace, 2, 1.0, 1.0, stream)


def get_device_error(clear: bool = True) -> tuple[int, int]:
    """(code, detail) of the device error word (synchronises)."""
    code = _c_i(0)
    detail = ctypes.c_longlong(0)
    _check(lib().pa_get_device_error(ctypes.byref(code), ctypes.byref(detail), int(clear)),
           "pa_get_device_error")
    return int(code.value), int(detail.value)


def set_kernel_timer(kernel: str, start: torch.cuda.Event | None,
                     stop: torch.cuda.Event | None) -> None:
    """Record CUDA events around every later launch of one library kernel."""
    sp = None if start is None else ctypes.c_void_p(start.cuda_event)
    ep = None if stop is None else ctypes.c_void_p(stop.cuda_event)
    _check(lib().pa_set_kernel_timer(KERNEL_IDS[kernel], sp, ep), "pa_set_kernel_timer")


OPTIONS = {"decode_self_plan": 1, "decode_tc": 2, "decode_max_workers": 3, "mixed_overlap": 4,
           "decode_token_major": 5, "cascade_overlap": 6, "decode_tm_ctas_per_sm": 7,
           "mixed_prefill_ctas": 8, "write_overlap": 9, "shared_min_kb": 10}


def set_option(name: str, value: int) -> None:
    """pa_set_option: process-wide library options (see include/pa_api.h)."""
    L = lib()
    L.pa_set_option.argtypes = [_c_i, _c_i]
    L.pa_set_option.restype = _c_i
    _check(L.pa_set_option(OPTIONS[name], int(value)), "pa_set_option")


def launch_count() -> int:
    return int(lib().pa_launch_count())


def noalloc_scratch_bytes() -> int:
    """Size of the fixed scratch array behind :func:`attention_noalloc`."""
    L = lib()
    L.pa_noalloc_scratch_bytes.argtypes = []
    L.pa_noalloc_scratch_bytes.restype = ctypes.c_size_t
    return int(L.pa_noalloc_scratch_bytes())


def attention_noalloc(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                      block_tables: torch.Tensor, seq_lens: torch.Tensor,
                      query_start_loc: torch.Tensor, scale: float, *, max_query_len: int,
                      max_seq_len: int, out: torch.Tensor, stream=None) -> torch.Tensor:
    """pa_attention_noalloc: attention with the library's fixed scratch array
    as workspace, for callers that cannot allocate device memory.

    Nothing is allocated by the call (``out`` must be given). Batches larger
    than the scratch array raise PA_ERR_WORKSPACE; calls that overlap on the
    GPU share the scratch and must be serialised by the caller.
    """
    L = lib()
    L.pa_attention_noalloc.argtypes = [_c_p, _c_p, _c_p, _c_p, _c_p, _c_p, ctypes.c_float, _c_p,
                                       _c_i, _c_i, _c_i, _c_i, _c_i, _c_i, _c_i, _c_i, _c_i,
                                       _c_i, _c_p]
    L.pa_attention_noalloc.restype = _c_i
    T, hq, d = q.shape
    nb, hkv, bs, d2 = k_cache.shape
    R = int(seq_lens.shape[0])
    if d2 != d or v_cache.shape != k_cache.shape:
        raise ValueError("shape mismatch between q and the caches")
    if query_start_loc.shape != (R + 1,) or block_tables.dim() != 2 or block_tables.shape[0] != R:
        raise ValueError("metadata shapes must be qsl [R+1], block_tables [R, max_blocks]")
    if out.shape != q.shape:
        raise ValueError("out must have q's shape")
    st = L.pa_attention_noalloc(
        _dev(q, torch.bfloat16, "q"), _dev(k_cache, torch.bfloat16, "k_cache"),
        _dev(v_cache, torch.bfloat16, "v_cache"), _dev(block_tables, torch.int32, "block_tables"),
        _dev(seq_lens, torch.int32, "seq_lens"),
        _dev(query_start_loc, torch.int32, "query_start_loc"), float(scale),
        _out(out), R, T, hq, hkv, d, bs, nb, int(block_tables.shape[1]),
        int(max_query_len), int(max_seq_len), _stream_ptr(stream))
    _check(st, "pa_attention_noalloc")
    return out
