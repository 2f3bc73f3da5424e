"""Exact attention for B200 (sm_100a): Python binding of the C ABI in ``include/fa.h``.

Every step of the computation runs in the CUDA kernels of ``libfa_b200.so``; this
module only checks tensors, allocates outputs with torch, and passes raw pointers and
the current CUDA stream.  There is no fallback: if the library is missing or a
call is rejected, an exception is raised.

    o, lse = fwd(q, k, v, causal=False)             # q [B,Hq,N,d], k/v [B,Hkv,N,d]
    dq, dk, dv = bwd(q, k, v, o, lse, do, causal=False)
    paged_kv_append(k_new, v_new, k_cache, v_cache, block_table, positions)
    o, lse = paged_decode(q, k_cache, v_cache, block_table, ctx_lens)
    o, lse = paged_prefill(q, k_cache, v_cache, block_table, ctx_lens, q_lens, causal=True)

The passes around attention (per-head norm and rotation of q and k; decode over a shared prefix;
decode that adds up attention weights, and the eviction by them):

    q2, k2 = qk_norm_rope(q, k, q_weight, k_weight, positions, inv_freq)
    dq, dk, dwq, dwk = qk_norm_rope_bwd(dq2, dk2, q, k, q_weight, k_weight, positions, inv_freq)
    q2 = qk_norm_rope_append(q, k, v, q_weight, k_weight, positions, inv_freq, k_cache, v_cache,
                             block_table, ctx_lens, q_lens)
    o, lse = paged_decode_shared(q, k_cache, v_cache, prefix_table, prefix_len, block_table, ctx_lens)
    o, lse = paged_decode_scored(q, k_cache, v_cache, block_table, ctx_lens, weights)
    ctx, weights, slot_pos = paged_evict(k_cache, v_cache, block_table, ctx_lens, seq_lens, weights,
                                         slot_pos, keep, recent)

bf16 inputs run on the tensor cores (d in {64, 96, 128, 256} forward, {64, 96, 128}
backward); fp32 inputs (d = 64) on the CUDA cores.  Paged caches are
[num_blocks, Hkv, 16, d].
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
import struct

import torch

__all__ = [
    "FAError",
    "lib",
    "fwd",
    "bwd",
    "bwd_workspace_size",
    "paged_decode",
    "paged_decode_workspace_size",
    "paged_kv_append",
    "paged_prefill",
    "rope_frequencies",
    "qk_norm_rope",
    "qk_norm_rope_bwd",
    "qk_norm_rope_append",
    "paged_decode_shared",
    "paged_decode_shared_workspace_size",
    "paged_decode_scored",
    "paged_decode_scored_workspace_size",
    "paged_evict",
    "paged_evict_workspace_size",
    "device_status",
    "set_decode_split",
    "set_wait_limit_ns",
    "selftest_wait_timeout",
    "EXPORTED",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfa_b200.so")

FA_OK, FA_ERR_INVALID_ARG, FA_ERR_UNSUPPORTED, FA_ERR_CUDA, FA_ERR_WORKSPACE, FA_ERR_DEVICE_TIMEOUT = range(6)
FA_DTYPE_F32, FA_DTYPE_BF16 = 0, 1
_DT = {torch.float32: FA_DTYPE_F32, torch.bfloat16: FA_DTYPE_BF16}

_vp, _i, _f, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
_i64 = ctypes.c_int64

# name -> (restype, argtypes); the same names as the C entry points
EXPORTED = {
    "fa_status_string": (ctypes.c_char_p, [_i]),
    "fa_version": (_i, []),
    "fa_fwd": (_i, [_vp] * 5 + [_i] * 6 + [_f, _i, _i, _vp]),
    "fa_bwd_workspace_size": (_sz, [_i] * 4),
    "fa_bwd": (_i, [_vp] * 9 + [_i] + [_i] * 6 + [_f, _i, _i, _vp, _sz, _vp]),
    "fa_paged_decode_workspace_size": (_sz, [_i] * 5),
    "fa_paged_decode": (_i, [_vp] * 7 + [_i] * 7 + [_f, _i, _vp, _sz, _vp]),
    "fa_paged_decode_noalloc": (_i, [_vp] * 7 + [_i] * 7 + [_f, _i, _vp]),
    "fa_paged_kv_append": (_i, [_vp] * 6 + [_i] * 6 + [_i, _vp]),
    "fa_paged_prefill": (_i, [_vp] * 6 + [_vp, _vp] + [_i] * 8 + [_f, _i, _i, _vp]),
    # (arguments in one struct, passed as its bytes, and the stream)
    "fa_qk_norm_rope": (_i, [_vp, _vp]),
    "fa_qk_norm_rope_append": (_i, [_vp, _vp]),
    "fa_qk_norm_rope_bwd_workspace_size": (_sz, [_i]),
    "fa_qk_norm_rope_bwd": (_i, [_vp, _vp]),
    "fa_paged_decode_shared_workspace_size": (_sz, [_i] * 7),
    "fa_paged_decode_shared": (_i, [_vp, _vp]),
    "fa_paged_decode_scored_workspace_size": (_sz, [_i] * 6),
    "fa_paged_decode_scored": (_i, [_vp, _vp]),
    "fa_paged_evict_workspace_size": (_sz, [_i] * 4),
    "fa_paged_evict": (_i, [_vp, _vp]),
    "fa_device_status": (_i, [_i]),
    "fa_set_wait_limit_ns": (None, [ctypes.c_uint64]),
    "fa_selftest_wait_timeout": (_i, [_vp]),
    "fa_set_decode_split": (_i, [_i]),
}

# name -> packer of its argument struct: pointers and sizes, int64 strides, ints, eps or scale, ints
PACKED = {
    "fa_qk_norm_rope": struct.Struct("8P8q11ifi").pack,
    "fa_qk_norm_rope_append": struct.Struct("13P11q14ifi").pack,
    "fa_qk_norm_rope_bwd": struct.Struct("14P14q11if3i").pack,
    "fa_paged_decode_shared": struct.Struct("11P8ifi").pack,
    "fa_paged_decode_scored": struct.Struct("10P7ifi").pack,
    "fa_paged_evict": struct.Struct("12P9i").pack,
}


class FAError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn}: {_status_string(status)} (status {status})")


_lib = None


def lib() -> ctypes.CDLL:
    """Load libfa_b200.so (raises if it was not built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with `python -m exact_attention_128_b200.build` "
                "(there is no non-CUDA implementation of this library)"
            )
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in EXPORTED.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def _status_string(s: int) -> str:
    return lib().fa_status_string(int(s)).decode()


def _check(fn: str, status: int):
    if status != FA_OK:
        raise FAError(fn, status)


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def _cuda4(name, t, dtype=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")


def fwd(q, k, v, causal: bool = False, scale: float | None = None, out=None, lse=None):
    """Forward pass: returns (o [B,Hq,Nq,d] of q's dtype, lse [B,Hq,Nq] fp32)."""
    for n, t in (("q", q), ("k", k), ("v", v)):
        _cuda4(n, t, q.dtype)
    if q.dim() != 4 or k.dim() != 4 or v.shape != k.shape:
        raise ValueError("expected q [B,Hq,Nq,d] and k, v [B,Hkv,Nkv,d]")
    B, Hq, Nq, d = q.shape
    Hkv, Nkv = k.shape[1], k.shape[2]
    if k.shape[0] != B or k.shape[3] != d:
        raise ValueError("q and k disagree on batch or head dim")
    if q.dtype not in _DT:
        raise ValueError(f"unsupported dtype {q.dtype}")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    o = out if out is not None else torch.empty_like(q)
    lse = lse if lse is not None else torch.empty((B, Hq, Nq), device=q.device, dtype=torch.float32)
    st = lib().fa_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, Hq, Hkv, Nq, Nkv, d,
                      float(scale), int(bool(causal)), _DT[q.dtype], _stream())
    _check("fa_fwd", st)
    return o, lse


def bwd_workspace_size(B, Hq, Nq, d) -> int:
    return int(lib().fa_bwd_workspace_size(B, Hq, Nq, d))


def bwd(q, k, v, o, lse, do, causal: bool = False, scale: float | None = None,
        grad_dtype: torch.dtype = torch.float32, workspace=None):
    """Backward pass of fwd: returns (dq, dk, dv) of dtype grad_dtype."""
    for n, t in (("q", q), ("k", k), ("v", v), ("o", o), ("do", do)):
        _cuda4(n, t, q.dtype)
    _cuda4("lse", lse, torch.float32)
    B, Hq, Nq, d = q.shape
    Hkv, Nkv = k.shape[1], k.shape[2]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if grad_dtype not in _DT:
        raise ValueError(f"unsupported grad dtype {grad_dtype}")
    dq = torch.empty(q.shape, device=q.device, dtype=grad_dtype)
    dk = torch.empty(k.shape, device=q.device, dtype=grad_dtype)
    dv = torch.empty(v.shape, device=q.device, dtype=grad_dtype)
    need = bwd_workspace_size(B, Hq, Nq, d)
    if workspace is None:
        workspace = torch.empty(max(need, 1), device=q.device, dtype=torch.uint8)
    st = lib().fa_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(do), _ptr(dq), _ptr(dk), _ptr(dv),
                      _DT[grad_dtype], B, Hq, Hkv, Nq, Nkv, d, float(scale), int(bool(causal)), _DT[q.dtype],
                      _ptr(workspace), workspace.numel() * workspace.element_size(), _stream())
    _check("fa_bwd", st)
    return dq, dk, dv


def paged_decode_workspace_size(R, Hq, d, max_blocks_per_seq, block_size) -> int:
    return int(lib().fa_paged_decode_workspace_size(R, Hq, d, max_blocks_per_seq, block_size))


def paged_decode(q, k_cache, v_cache, block_table, ctx_lens, scale: float | None = None,
                 with_lse: bool = True, workspace=None, out=None):
    """One decode step: q [R,Hq,d], caches [num_blocks,Hkv,block_size,d] -> (o [R,Hq,d], lse [R,Hq])."""
    _cuda4("q", q, torch.bfloat16)
    _cuda4("k_cache", k_cache, torch.bfloat16)
    _cuda4("v_cache", v_cache, torch.bfloat16)
    _cuda4("block_table", block_table, torch.int32)
    _cuda4("ctx_lens", ctx_lens, torch.int32)
    if v_cache.shape != k_cache.shape:
        raise ValueError("k_cache and v_cache must have the same shape")
    R, Hq, d = q.shape
    num_blocks, Hkv, bs, _ = k_cache.shape
    maxb = block_table.shape[1]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    o = out if out is not None else torch.empty_like(q)
    lse = torch.empty((R, Hq), device=q.device, dtype=torch.float32) if with_lse else None
    need = paged_decode_workspace_size(R, Hq, d, maxb, bs)
    if workspace is None:
        workspace = torch.empty(max(need, 1), device=q.device, dtype=torch.uint8)
    st = lib().fa_paged_decode(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table), _ptr(ctx_lens),
                               _ptr(o), _ptr(lse), R, Hq, Hkv, d, bs, maxb, num_blocks, float(scale),
                               FA_DTYPE_BF16, _ptr(workspace), workspace.numel() * workspace.element_size(),
                               _stream())
    _check("fa_paged_decode", st)
    return o, lse


def paged_kv_append(k_new, v_new, k_cache, v_cache, block_table, positions):
    """Write one new token per request into the paged caches in place (slot positions[r])."""
    _cuda4("k_new", k_new, torch.bfloat16)
    _cuda4("v_new", v_new, torch.bfloat16)
    _cuda4("k_cache", k_cache, torch.bfloat16)
    _cuda4("v_cache", v_cache, torch.bfloat16)
    _cuda4("block_table", block_table, torch.int32)
    _cuda4("positions", positions, torch.int32)
    if k_new.shape != v_new.shape or k_cache.shape != v_cache.shape:
        raise ValueError("k/v shapes disagree")
    R, Hkv, d = k_new.shape
    num_blocks, _, bs, _ = k_cache.shape
    st = lib().fa_paged_kv_append(_ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache), _ptr(block_table),
                                  _ptr(positions), R, Hkv, d, bs, block_table.shape[1], num_blocks, FA_DTYPE_BF16,
                                  _stream())
    _check("fa_paged_kv_append", st)


def paged_prefill(q, k_cache, v_cache, block_table, ctx_lens, q_lens, causal: bool = True,
                  scale: float | None = None, out=None, lse=None):
    """Prefill over a paged KV cache: q [R,Hq,Nq_max,d] (request r's rows < q_lens[r] are its
    last q_lens[r] positions), caches [num_blocks,Hkv,block_size,d] -> (o, lse [R,Hq,Nq_max]).
    Rows >= q_lens[r] of o and lse are undefined."""
    _cuda4("q", q, torch.bfloat16)
    _cuda4("k_cache", k_cache, torch.bfloat16)
    _cuda4("v_cache", v_cache, torch.bfloat16)
    _cuda4("block_table", block_table, torch.int32)
    _cuda4("ctx_lens", ctx_lens, torch.int32)
    _cuda4("q_lens", q_lens, torch.int32)
    if q.dim() != 4 or k_cache.dim() != 4 or v_cache.shape != k_cache.shape:
        raise ValueError("expected q [R,Hq,Nq_max,d] and caches [num_blocks,Hkv,block_size,d]")
    R, Hq, Nq, d = q.shape
    num_blocks, Hkv, bs, _ = k_cache.shape
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    o = out if out is not None else torch.empty_like(q)
    if lse is None:
        lse = torch.empty((R, Hq, Nq), device=q.device, dtype=torch.float32)
    st = lib().fa_paged_prefill(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table), _ptr(ctx_lens),
                                _ptr(q_lens), _ptr(o), _ptr(lse), R, Hq, Hkv, Nq, d, bs, block_table.shape[1],
                                num_blocks, float(scale), int(bool(causal)), FA_DTYPE_BF16, _stream())
    _check("fa_paged_prefill", st)
    return o, lse


# ------------------------------------------------------------------------------------
# The passes around attention.  Every tensor of a call lives on one device, which need
# not be the current one; the call runs on that device's current stream.
# ------------------------------------------------------------------------------------
def _expect(name, t, shape, dtype, device):
    """Address of a contiguous tensor of this shape and type on the CUDA device of this index."""
    try:
        if t.shape == shape and t.dtype is dtype and t.get_device() == device >= 0 and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    raise ValueError(f"{name} must be a contiguous {dtype} CUDA tensor of shape {tuple(shape)} on device {device}, got "
                     f"{_described(t)}")


def _described(t):
    if not isinstance(t, torch.Tensor):
        return type(t).__name__
    return f"{t.dtype} {tuple(t.shape)} with strides {t.stride()} on {t.device}"


def _device(name, t, dim):
    """Index of the CUDA device of the tensor that a call's others are held against."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dim() != dim:
        raise ValueError(f"{name} must be a CUDA tensor of {dim} dimensions, got {_described(t)}")
    return t.get_device()


_current_device = getattr(torch._C, "_cuda_getDevice", None)  # (absent from a build of torch without CUDA)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _call(name, device, *args):
    """Run one entry point on the device of this index and its current stream."""
    fn = getattr(_lib or lib(), name)
    try:
        packed = PACKED[name](*args)
    except (struct.error, OverflowError) as e:
        raise ValueError(f"{name}: a size or option is out of its C type's range: {e}") from None
    if device == _current_device():
        st = fn(packed, _raw_stream(device))
    else:
        with torch.cuda.device(device):
            st = fn(packed, _raw_stream(device))
    if st:
        raise FAError(name, st)


@functools.lru_cache(maxsize=1024)
def _size(name, *args):
    """A workspace size: it depends on its arguments alone."""
    try:
        return int(getattr(lib(), name)(*args))
    except ctypes.ArgumentError as e:
        raise ValueError(f"{name}: {e}") from None


def _workspace(workspace, need, like):
    """(address, bytes) of the caller's workspace, or of a new one; the last item keeps it alive."""
    if workspace is None:
        if not need:
            return 0, 0, None
        workspace = like.new_empty(need, dtype=torch.uint8)
        return workspace.data_ptr(), need, workspace
    if workspace.get_device() != like.get_device() or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {like.device}, got {_described(workspace)}")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


def _rows(name, t, dtype, device, shape):
    """Address and {batch, head, token} strides of a [B,H,N,d] view whose rows are contiguous."""
    try:
        if t.shape == shape and t.dtype is dtype and t.get_device() == device:
            sb, sh, sn, sd = t.stride()
            if sd == 1 or shape[3] == 1:
                # a dimension of size 1 has no stride of its own
                return t.data_ptr(), (sb if shape[0] > 1 else 0, sh if shape[1] > 1 else 0,
                                      sn if shape[2] > 1 else 0)
    except AttributeError:
        pass
    raise ValueError(f"{name} must be {dtype} {tuple(shape)} with a contiguous last dimension on device {device}, got "
                     f"{_described(t)}")


def rope_frequencies(rotary_dim: int, base: float = 10000.0, device="cuda"):
    """Radians per position of the rotary_dim / 2 pairs, base^(-2i / rotary_dim), in 64 bits."""
    if rotary_dim <= 0 or rotary_dim % 2:
        raise ValueError(f"rotary_dim must be positive and even, got {rotary_dim}")
    i = torch.arange(rotary_dim // 2, device=device, dtype=torch.float64)
    return torch.exp(i * (-2.0 * math.log(base) / rotary_dim))


_ZEROS = {1: (0, 0), 2: (0,), 3: ()}


def _rope_args(device, positions, inv_freq, sections, B, N):
    """Rotary arguments in their C form: position pointer and strides, frequencies, sections."""
    try:
        half = inv_freq.shape[0]
        shape = positions.shape
        dims = len(shape)
    except (AttributeError, IndexError):
        raise ValueError(f"inv_freq must be a tensor [rotary_dim / 2], positions one of [N], [B,N] or [axes,B,N], got "
                         f"{_described(inv_freq)} and {_described(positions)}") from None
    freq = _expect("inv_freq", inv_freq, (half,), torch.float64, device)
    axes = shape[0] if dims == 3 else 1
    sec = (half,) if sections is None else tuple(sections)
    if len(sec) != axes or not 1 <= axes <= 3 or sum(sec) != half:
        raise ValueError(f"{axes} axes of positions need {axes} sections (1 to 3) that sum to {half}, got {sections}")
    if shape != ((axes, B, N) if dims == 3 else (B, N) if dims == 2 else (N,)):
        raise ValueError(f"positions must be [N], [B,N] or [axes,B,N] with B = {B} and N = {N}, got {tuple(shape)}")
    strides = positions.stride()
    if positions.dtype is not torch.int32 or positions.get_device() != device or (N > 1 and strides[-1] != 1):
        raise ValueError(f"positions must be int32 on device {device} with a contiguous last dimension, got "
                         f"{_described(positions)}")
    return (positions.data_ptr(), strides[0] if axes > 1 else 0, strides[-2] if dims > 1 and B > 1 else 0, freq,
            2 * half, sec + _ZEROS[axes], axes)


def _rope_weights(q_weight, k_weight, d, dtype, device):
    if q_weight is None and k_weight is None:
        return 0, 0
    if q_weight is None or k_weight is None:
        raise ValueError("q_weight and k_weight come together, or neither")
    return _expect("q_weight", q_weight, (d,), dtype, device), _expect("k_weight", k_weight, (d,), dtype, device)


def _heads(name, t):
    """Size of dimension 1 of a [B,H,N,d] tensor or cache."""
    if not isinstance(t, torch.Tensor) or t.dim() != 4:
        raise ValueError(f"{name} must be a CUDA tensor of 4 dimensions, got {_described(t)}")
    return t.shape[1]


def qk_norm_rope(q, k, q_weight, k_weight, positions, inv_freq, sections=None, interleaved: bool = False,
                 eps: float = 1e-6, q_out=None, k_out=None):
    """Per-head RMS norm and rotation: q [B,Hq,N,d], k [B,Hkv,N,d] (views with contiguous rows, as
    of a fused projection) -> contiguous (q', k') for fwd.  Weights [d], or None for both: the
    rotation alone.  positions int32 [N], [B,N] or [axes,B,N] with one section per axis;
    inv_freq float64 [rotary_dim / 2] (see rope_frequencies)."""
    device = _device("q", q, 4)
    B, Hq, N, d = shape = q.shape
    dtype, Hkv = q.dtype, _heads("k", k)
    kshape = (B, Hkv, N, d)
    qp, qs = _rows("q", q, dtype, device, shape)
    kp, ks = _rows("k", k, dtype, device, kshape)
    if dtype not in _DT:
        raise ValueError(f"unsupported dtype {dtype}")
    pos, sa, sb, freq, rd, sec, axes = _rope_args(device, positions, inv_freq, sections, B, N)
    wq, wk = _rope_weights(q_weight, k_weight, d, dtype, device)
    if q_out is None:
        q_out = q.new_empty(shape)
    if k_out is None:
        k_out = k.new_empty(kshape)
    qo = _expect("q_out", q_out, shape, dtype, device)
    ko = _expect("k_out", k_out, kshape, dtype, device)
    _call("fa_qk_norm_rope", device, qp, kp, wq, wk, pos, freq, qo, ko, *qs, *ks, sa, sb, B, Hq, Hkv, N, d, rd, *sec,
          axes, 1 if interleaved else 0, eps, _DT[dtype])
    return q_out, k_out


def qk_norm_rope_bwd(dq_out, dk_out, q, k, q_weight, k_weight, positions, inv_freq, sections=None,
                     interleaved: bool = False, eps: float = 1e-6, grad_dtype: torch.dtype | None = None, dq=None,
                     dk=None, workspace=None):
    """Gradients of qk_norm_rope: (dq, dk, dq_weight, dk_weight) from dq_out, dk_out (contiguous, as
    bwd returns them).  dq and dk have grad_dtype (default: q's) and lie in memory as q and k do (a
    projection's [B,N,H,d], or contiguous), or are the [B,H,N,d] views given; the weight gradients
    are fp32 [d] (None without weights)."""
    device = _device("q", q, 4)
    B, Hq, N, d = shape = q.shape
    dtype, Hkv = q.dtype, _heads("k", k)
    kshape = (B, Hkv, N, d)
    qp, qs = _rows("q", q, dtype, device, shape)
    kp, ks = _rows("k", k, dtype, device, kshape)
    if grad_dtype is None:
        grad_dtype = dtype
    dout_dtype = dq_out.dtype if isinstance(dq_out, torch.Tensor) else None
    if dtype not in _DT or grad_dtype not in _DT or dout_dtype not in _DT:
        raise ValueError(f"unsupported dtypes: {dtype} with gradients {dout_dtype} -> {grad_dtype}")
    dqo = _expect("dq_out", dq_out, shape, dout_dtype, device)
    dko = _expect("dk_out", dk_out, kshape, dout_dtype, device)
    pos, sa, sb, freq, rd, sec, axes = _rope_args(device, positions, inv_freq, sections, B, N)
    wq, wk = _rope_weights(q_weight, k_weight, d, dtype, device)
    if dq is None:
        dq = torch.empty_like(q, dtype=grad_dtype)  # (dense, its dimensions in the order of q's)
    if dk is None:
        dk = torch.empty_like(k, dtype=grad_dtype)
    dqp, dqs = _rows("dq", dq, grad_dtype, device, shape)
    dkp, dks = _rows("dk", dk, grad_dtype, device, kshape)
    dwq = dwk = keep = None
    dwqp = dwkp = ws = ws_bytes = 0
    if wq:
        dwq, dwk = q.new_empty(d, dtype=torch.float32), q.new_empty(d, dtype=torch.float32)
        dwqp, dwkp = dwq.data_ptr(), dwk.data_ptr()
        ws, ws_bytes, keep = _workspace(workspace, _size("fa_qk_norm_rope_bwd_workspace_size", d), q)
    _call("fa_qk_norm_rope_bwd", device, dqo, dko, qp, kp, wq, wk, pos, freq, dqp, dkp, dwqp, dwkp, ws, ws_bytes, *qs,
          *ks, *dqs, *dks, sa, sb, B, Hq, Hkv, N, d, rd, *sec, axes, 1 if interleaved else 0, eps, _DT[dtype],
          _DT[dout_dtype], _DT[grad_dtype])
    return dq, dk, dwq, dwk


def qk_norm_rope_append(q, k, v, q_weight, k_weight, positions, inv_freq, k_cache, v_cache, block_table, ctx_lens,
                        q_lens, sections=None, interleaved: bool = False, eps: float = 1e-6, q_out=None):
    """qk_norm_rope of R requests' newest tokens (q [R,Hq,Nq_max,d], k and v [R,Hkv,Nq_max,d], bf16
    views) with k' and v written into the paged caches: token i of request r at cache position
    ctx_lens[r] - q_lens[r] + i.  Returns q' [R,Hq,Nq_max,d], whose rows i >= q_lens[r] are left as
    q_out holds them (undefined where q_out is None)."""
    device = _device("q", q, 4)
    R, Hq, N, d = shape = q.shape
    Hkv, bf16 = _heads("k", k), torch.bfloat16
    kshape = (R, Hkv, N, d)
    qp, qs = _rows("q", q, bf16, device, shape)
    kp, ks = _rows("k", k, bf16, device, kshape)
    vp, vs = _rows("v", v, bf16, device, kshape)
    pos, sa, sb, freq, rd, sec, axes = _rope_args(device, positions, inv_freq, sections, R, N)
    wq, wk = _rope_weights(q_weight, k_weight, d, bf16, device)
    num_blocks, bs, maxb, kc, vc, bt, ctx = _cache_args(k_cache, v_cache, block_table, ctx_lens, R, Hkv, d, device)
    ql = _expect("q_lens", q_lens, (R,), torch.int32, device)
    if q_out is None:
        q_out = q.new_empty(shape)
    qo = _expect("q_out", q_out, shape, bf16, device)
    _call("fa_qk_norm_rope_append", device, qp, kp, vp, wq, wk, pos, freq, kc, vc, bt, ctx, ql, qo, *qs, *ks, *vs, sa,
          sb, R, Hq, Hkv, N, d, bs, maxb, num_blocks, rd, *sec, axes, 1 if interleaved else 0, eps, FA_DTYPE_BF16)
    return q_out


def _cache_args(k_cache, v_cache, block_table, ctx_lens, R, Hkv, d, device):
    try:
        shape = k_cache.shape
        num_blocks, _, bs, _ = shape
        maxb = block_table.shape[1]
    except (AttributeError, ValueError, IndexError):
        raise ValueError(f"caches must be [num_blocks,Hkv,block_size,d] and block_table [R,max_blocks], got "
                         f"{_described(k_cache)} and {_described(block_table)}") from None
    if shape[1] != Hkv or shape[3] != d:
        raise ValueError(f"caches must be [num_blocks,{Hkv},block_size,{d}], got {_described(k_cache)}")
    kc = _expect("k_cache", k_cache, shape, torch.bfloat16, device)
    vc = _expect("v_cache", v_cache, shape, torch.bfloat16, device)
    bt = _expect("block_table", block_table, (R, maxb), torch.int32, device)
    return num_blocks, bs, maxb, kc, vc, bt, _expect("ctx_lens", ctx_lens, (R,), torch.int32, device)


def paged_decode_shared_workspace_size(R, Hq, Hkv, d, max_prefix_blocks, max_blocks_per_seq, block_size) -> int:
    return _size("fa_paged_decode_shared_workspace_size", R, Hq, Hkv, d, max_prefix_blocks, max_blocks_per_seq,
                 block_size)


def _decode_outputs(q, shape, device, with_lse, out):
    if out is None:
        out = torch.empty_like(q)
    op = _expect("out", out, shape, torch.bfloat16, device)
    if not with_lse:
        return out, None, op, 0
    lse = q.new_empty(shape[:2], dtype=torch.float32)
    return out, lse, op, lse.data_ptr()


def paged_decode_shared(q, k_cache, v_cache, prefix_table, prefix_len, block_table, ctx_lens,
                        scale: float | None = None, with_lse: bool = True, workspace=None, out=None):
    """One decode step of R requests behind a common prefix, which is computed once for all:
    prefix_table [max_prefix_blocks] and prefix_len [1] (device, int32) name its tokens, block_table
    and ctx_lens each request's own ones; either length may be 0 -> (o [R,Hq,d], lse [R,Hq])."""
    device = _device("q", q, 3)
    R, Hq, d = shape = q.shape
    Hkv, i32 = _heads("k_cache", k_cache), torch.int32
    qp = _expect("q", q, shape, torch.bfloat16, device)
    num_blocks, bs, maxb, kc, vc, bt, ctx = _cache_args(k_cache, v_cache, block_table, ctx_lens, R, Hkv, d, device)
    pb = prefix_table.shape[0] if isinstance(prefix_table, torch.Tensor) and prefix_table.dim() == 1 else 0
    pt = _expect("prefix_table", prefix_table, (pb,), i32, device)
    pl = _expect("prefix_len", prefix_len, (1,), i32, device)
    need = _size("fa_paged_decode_shared_workspace_size", R, Hq, Hkv, d, pb, maxb, bs)
    ws, ws_bytes, keep = _workspace(workspace, need, q)
    o, lse, op, lp = _decode_outputs(q, shape, device, with_lse, out)
    _call("fa_paged_decode_shared", device, qp, kc, vc, pt, pl, bt, ctx, op, lp, ws, ws_bytes, R, Hq, Hkv, d, bs, pb,
          maxb, num_blocks, d ** -0.5 if scale is None else scale, FA_DTYPE_BF16)
    return o, lse


def paged_decode_scored_workspace_size(R, Hq, Hkv, d, max_blocks_per_seq, block_size) -> int:
    return _size("fa_paged_decode_scored_workspace_size", R, Hq, Hkv, d, max_blocks_per_seq, block_size)


def paged_decode_scored(q, k_cache, v_cache, block_table, ctx_lens, weights, scale: float | None = None,
                        with_lse: bool = True, workspace=None, out=None):
    """A decode step that adds to weights [R,Hkv,max_blocks*16] (fp32, in place) the attention each
    cached token gets, summed over the query heads of its kv head -> (o [R,Hq,d], lse [R,Hq])."""
    device = _device("q", q, 3)
    R, Hq, d = shape = q.shape
    Hkv = _heads("k_cache", k_cache)
    qp = _expect("q", q, shape, torch.bfloat16, device)
    num_blocks, bs, maxb, kc, vc, bt, ctx = _cache_args(k_cache, v_cache, block_table, ctx_lens, R, Hkv, d, device)
    w = _expect("weights", weights, (R, Hkv, maxb * bs), torch.float32, device)
    need = _size("fa_paged_decode_scored_workspace_size", R, Hq, Hkv, d, maxb, bs)
    ws, ws_bytes, keep = _workspace(workspace, need, q)
    o, lse, op, lp = _decode_outputs(q, shape, device, with_lse, out)
    _call("fa_paged_decode_scored", device, qp, kc, vc, bt, ctx, w, op, lp, ws, ws_bytes, R, Hq, Hkv, d, bs, maxb,
          num_blocks, d ** -0.5 if scale is None else scale, FA_DTYPE_BF16)
    return o, lse


def paged_evict_workspace_size(R, Hkv, max_blocks_per_seq, keep) -> int:
    return _size("fa_paged_evict_workspace_size", R, Hkv, max_blocks_per_seq, keep)


def paged_evict(k_cache, v_cache, block_table, ctx_lens, seq_lens, weights, slot_pos, keep: int, recent: int,
                weights_out=None, slot_pos_out=None, new_ctx=None, workspace=None):
    """Keep, per request and kv head, the tokens of the `recent` newest positions and the heaviest
    others, `keep` in all: moves their rows in the caches and returns (new_ctx [R], weights,
    slot_pos) for the next steps.  seq_lens [R]: tokens of each sequence so far, evicted ones
    included; slot_pos int32 [R,Hkv,max_blocks*16]: -1 everywhere at the start."""
    device = _device("k_cache", k_cache, 4)
    _, Hkv, _, d = k_cache.shape
    f32, i32 = torch.float32, torch.int32
    R = block_table.shape[0] if isinstance(block_table, torch.Tensor) and block_table.dim() == 2 else 0
    num_blocks, bs, maxb, kc, vc, bt, ctx = _cache_args(k_cache, v_cache, block_table, ctx_lens, R, Hkv, d, device)
    shape = (R, Hkv, maxb * bs)
    seq = _expect("seq_lens", seq_lens, (R,), i32, device)
    w, sp = _expect("weights", weights, shape, f32, device), _expect("slot_pos", slot_pos, shape, i32, device)
    if weights_out is None:
        weights_out = torch.empty_like(weights)
    if slot_pos_out is None:
        slot_pos_out = torch.empty_like(slot_pos)
    if new_ctx is None:
        new_ctx = torch.empty_like(ctx_lens)
    wo = _expect("weights_out", weights_out, shape, f32, device)
    so = _expect("slot_pos_out", slot_pos_out, shape, i32, device)
    nc = _expect("new_ctx", new_ctx, (R,), i32, device)
    need = _size("fa_paged_evict_workspace_size", R, Hkv, maxb, keep)
    ws, ws_bytes, alive = _workspace(workspace, need, k_cache)
    _call("fa_paged_evict", device, kc, vc, bt, ctx, seq, w, sp, wo, so, nc, ws, ws_bytes, R, Hkv, d, bs, maxb,
          num_blocks, keep, recent, FA_DTYPE_BF16)
    return new_ctx, weights_out, slot_pos_out


def device_status(reset: bool = True) -> int:
    return int(lib().fa_device_status(int(bool(reset))))


def set_decode_split(blocks: int) -> int:
    """Cache blocks per decode split (multiple of 4 in [32, 128]; 0 = default); returns the old value."""
    old = int(lib().fa_set_decode_split(int(blocks)))
    if old < 0:
        raise ValueError(f"decode split of {blocks} blocks is out of range")
    return old


def set_wait_limit_ns(ns: int):
    lib().fa_set_wait_limit_ns(int(ns))


def selftest_wait_timeout():
    _check("fa_selftest_wait_timeout", lib().fa_selftest_wait_timeout(_stream()))
