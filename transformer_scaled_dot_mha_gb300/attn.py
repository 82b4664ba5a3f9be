"""Python binding of libattn_gb300.so: the C entry points of include/attn_gb300.h
under the same names, plus tensor-shaped wrappers.

This module only marshals arguments (tensor shapes, data pointers, the current
CUDA stream) and turns status codes into exceptions; every step of the
attention computation runs in the library's kernels. There is no fallback: if
the library is missing or fails to load, every call raises.
"""
from __future__ import annotations

import ctypes
import math
import os

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libattn_gb300.so")

ATTN_OK, ATTN_ERR_INVALID, ATTN_ERR_UNSUPPORTED, ATTN_ERR_CUDA, ATTN_ERR_TIMEOUT = 0, -1, -2, -3, -4
MASK_NONE, MASK_CAUSAL, MASK_KEY_PADDING = 0, 1, 2
ROPE_INTERLEAVED, CACHE_E4M3 = 1, 2  # flags of the rotation and of the paged cache
BWD_DETERMINISTIC = 1  # attn_bwd flag: the two-kernel schedule, bit-identical on every run

_lib = None


class AttnError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {status_string(status)} ({status})")
        self.status = status


def lib() -> ctypes.CDLL:
    """The loaded CUDA library (loaded once)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built: run `python -c 'import __graft_entry__ as g; g.build()'`")
        L = ctypes.CDLL(LIB_PATH)
        vp, i, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
        L.attn_fwd.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, f, i, vp, vp]
        L.attn_fwd.restype = i
        L.attn_fwd_host_workspace_size.argtypes = [i, i, i, i, i, i]
        L.attn_fwd_host_workspace_size.restype = ctypes.c_size_t
        L.attn_fwd_host.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, f, i, vp, vp, ctypes.c_size_t, vp]
        L.attn_fwd_host.restype = i
        L.attn_fwd_local.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, i, i, vp, vp]
        L.attn_fwd_local.restype = i
        L.attn_fwd_f32.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, f, i, vp, vp]
        L.attn_fwd_f32.restype = i
        L.attn_decode_workspace_size.argtypes = [i, i, i, i, i]
        L.attn_decode_workspace_size.restype = ctypes.c_size_t
        L.attn_decode.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, vp, vp, ctypes.c_size_t, vp]
        L.attn_decode.restype = i
        L.attn_decode_noalloc.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, vp, vp]
        L.attn_decode_noalloc.restype = i
        L.attn_bwd_workspace_size.argtypes = [i, i, i, i, i]
        L.attn_bwd_workspace_size.restype = ctypes.c_size_t
        L.attn_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, f, i, vp, i, vp,
                               ctypes.c_size_t, vp]
        L.attn_bwd.restype = i
        L.attn_bwd_local.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, f, i, i, vp, i, vp,
                                     ctypes.c_size_t, vp]
        L.attn_bwd_local.restype = i
        L.attn_bwd_host_workspace_size.argtypes = [i, i, i, i, i, i, i]
        L.attn_bwd_host_workspace_size.restype = ctypes.c_size_t
        L.attn_bwd_host.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, f, i, vp, i, vp,
                                    ctypes.c_size_t, vp]
        L.attn_bwd_host.restype = i
        L.attn_weights.argtypes = [vp, vp, vp, vp, i, i, i, i, i, f, i, vp, vp]
        L.attn_weights.restype = i
        L.attn_linear.argtypes = [vp, vp, vp, vp, i, i, i, vp]
        L.attn_linear.restype = i
        L.attn_mha_workspace_size.argtypes = [i, i, i, i, i, i]
        L.attn_mha_workspace_size.restype = ctypes.c_size_t
        L.attn_mha_fwd.argtypes = [vp] * 11 + [i, i, i, i, i, i, i, f, i, vp, vp, ctypes.c_size_t, vp]
        L.attn_mha_fwd.restype = i
        i64, sz = ctypes.c_int64, ctypes.c_size_t
        # q, k, strides, weights, eps, cos_sin, n_pos, d_rot, positions
        rope = [vp, vp, i64, i64, vp, vp, f, vp, i, i, vp]
        L.attn_norm_rope.argtypes = rope + [vp, vp, i, i, i, i, i, i, vp]
        L.attn_norm_rope.restype = i
        L.attn_norm_rope_bwd_workspace_size.argtypes = [i, i, i, i, i]
        L.attn_norm_rope_bwd_workspace_size.restype = sz
        L.attn_norm_rope_bwd.argtypes = rope + [vp, vp, vp, vp, i64, i64, vp, vp, i, i, i, i, i, i, vp, sz, vp]
        L.attn_norm_rope_bwd.restype = i
        L.attn_paged_append.argtypes = [vp, vp, vp, i64, i64, i64, vp, vp, f, vp, i, i, vp, vp, vp, i, i, vp, vp, vp,
                                        i, i, vp, vp, i, i, i, i, i, vp]
        L.attn_paged_append.restype = i
        L.attn_paged_decode_workspace_size.argtypes = [i, i, i, i, i]
        L.attn_paged_decode_workspace_size.restype = sz
        L.attn_paged_decode.argtypes = [vp] * 7 + [i] * 8 + [f, i, i, vp, vp, i, vp, sz, vp]
        L.attn_paged_decode.restype = i
        L.attn_packed_fwd_workspace_size.argtypes = [i, i, i, i, i]
        L.attn_packed_fwd_workspace_size.restype = sz
        L.attn_packed_fwd.argtypes = [vp] * 5 + [i64] * 8 + [vp, vp] + [i] * 6 + [f, i, i, vp, sz, vp]
        L.attn_packed_fwd.restype = i
        L.attn_packed_bwd_workspace_size.argtypes = [i, i, i, i, i, i]
        L.attn_packed_bwd_workspace_size.restype = sz
        L.attn_packed_bwd.argtypes = [vp] * 9 + [ctypes.POINTER(i64), vp, vp] + [i] * 6 + [f, i, i, vp, sz, vp]
        L.attn_packed_bwd.restype = i
        L.attn_paged_chunk_workspace_size.argtypes = [i, i, i, i, i]
        L.attn_paged_chunk_workspace_size.restype = sz
        L.attn_paged_chunk.argtypes = [vp] * 8 + [i] * 8 + [f, i, i, vp, vp, i, vp, sz, vp]
        L.attn_paged_chunk.restype = i
        L.attn_fault_status.argtypes = [vp, i, ctypes.POINTER(ctypes.c_uint32)]
        L.attn_fault_status.restype = i
        L.attn_status_string.argtypes = [i]
        L.attn_status_string.restype = ctypes.c_char_p
        L.attn_internal_arm_wait_timeout.argtypes = [ctypes.c_ulonglong, i]
        L.attn_internal_arm_wait_timeout.restype = None
        L.attn_internal_arm_chunk_give_up.argtypes = [i]
        L.attn_internal_arm_chunk_give_up.restype = None
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().attn_status_string(int(status)).decode()


def _short_ways():
    """(current device, its current stream's handle): torch's own short ways, which save 0.3 and 3 us a
    call but are no public names; the public ones where they are missing."""
    return (getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device),
            getattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: torch.cuda.current_stream(dev).cuda_stream))


_current_device, _current_stream = _short_ways()


def _stream_handle(stream) -> int:
    if stream is None:
        return _current_stream(torch.cuda.current_device())
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _check(t, name, dtype, ndim=4):
    if t.dtype != dtype or t.dim() != ndim or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {ndim}-D CUDA {dtype} tensor, got {t.dtype} {tuple(t.shape)}")


def _call(fn, q, k, v, out, lse, scale, mask_mode, key_lens, stream, dtype, where):
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (out, "out")):
        _check(t, n, dtype)
    B, H, n_q, d_k = q.shape
    n_k, d_v = k.shape[2], v.shape[3]
    if k.shape != (B, H, n_k, d_k) or v.shape != (B, H, n_k, d_v) or out.shape != (B, H, n_q, d_v):
        raise ValueError(f"shape mismatch: q{tuple(q.shape)} k{tuple(k.shape)} v{tuple(v.shape)} out{tuple(out.shape)}")
    if lse is not None:
        _check(lse, "lse", torch.float32, 3)
        if lse.shape != (B, H, n_q):
            raise ValueError("lse must have shape [B, H, n_q]")
    if key_lens is not None:
        _check(key_lens, "key_lens", torch.int32, 1)
        if key_lens.shape != (B,):
            raise ValueError("key_lens must have shape [B]")
    if scale is None:
        scale = 1.0 / math.sqrt(d_k)
    st = fn(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, H, n_q, n_k, d_k, d_v, float(scale), int(mask_mode),
            _ptr(key_lens), _stream_handle(stream))
    if st != ATTN_OK:
        raise AttnError(st, where)
    return out


def attn_fwd(q, k, v, out, lse=None, scale=None, mask_mode=MASK_NONE, key_lens=None, stream=None):
    """bf16 forward into caller-provided ``out`` (and optional fp32 ``lse``)."""
    return _call(lib().attn_fwd, q, k, v, out, lse, scale, mask_mode, key_lens, stream, torch.bfloat16, "attn_fwd")


def attn_fwd_host_workspace_size(B, H, n_q, n_k, d, mask_mode=MASK_NONE) -> int:
    return int(lib().attn_fwd_host_workspace_size(B, H, n_q, n_k, d, int(mask_mode)))


def attn_fwd_host(q, k, v, out, workspace, lse=None, scale=None, mask_mode=MASK_NONE, key_lens=None, stream=None):
    """bf16 forward on HOST tensors (pinned recommended): q, k, v, key_lens are read
    and out, lse written in host memory; the chunked copy/compute pipeline runs on
    the GPU with ``workspace`` (a CUDA uint8 tensor of attn_fwd_host_workspace_size
    bytes) and is asynchronous on ``stream``."""
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (out, "out")):
        if t.dtype != torch.bfloat16 or t.dim() != 4 or t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{n} must be a contiguous 4-D host bf16 tensor, got {t.dtype} {tuple(t.shape)}")
    B, H, n_q, d_k = q.shape
    n_k, d_v = k.shape[2], v.shape[3]
    if k.shape != (B, H, n_k, d_k) or v.shape != (B, H, n_k, d_v) or out.shape != (B, H, n_q, d_v):
        raise ValueError(f"shape mismatch: q{tuple(q.shape)} k{tuple(k.shape)} v{tuple(v.shape)} out{tuple(out.shape)}")
    if lse is not None and (lse.dtype != torch.float32 or lse.is_cuda or not lse.is_contiguous()
                            or lse.shape != (B, H, n_q)):
        raise ValueError("lse must be a contiguous host float32 tensor of shape [B, H, n_q]")
    if key_lens is not None and (key_lens.dtype != torch.int32 or key_lens.is_cuda or key_lens.shape != (B,)):
        raise ValueError("key_lens must be a host int32 tensor of shape [B]")
    if workspace.dtype != torch.uint8 or not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA uint8 tensor")
    if scale is None:
        scale = 1.0 / math.sqrt(d_k)
    st = lib().attn_fwd_host(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, H, n_q, n_k, d_k, d_v,
                             float(scale), int(mask_mode), _ptr(key_lens), _ptr(workspace), workspace.numel(),
                             _stream_handle(stream))
    if st != ATTN_OK:
        raise AttnError(st, "attn_fwd_host")
    return out


def attn_fwd_local(q, k, v, out, window, lse=None, scale=None, mask_mode=MASK_NONE, key_lens=None, stream=None):
    """Local-window (restricted) self-attention, bf16: key j is legal for query i only
    if |i - j| <= window (plus mask_mode)."""
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (out, "out")):
        _check(t, n, torch.bfloat16)
    B, H, n, d_k = q.shape
    d_v = v.shape[3]
    if k.shape != (B, H, n, d_k) or v.shape != (B, H, n, d_v) or out.shape != (B, H, n, d_v):
        raise ValueError("local attention is self-attention: q, k, v, out must share B, H, n")
    if lse is not None:
        _check(lse, "lse", torch.float32, 3)
    if key_lens is not None:
        _check(key_lens, "key_lens", torch.int32, 1)
    if scale is None:
        scale = 1.0 / math.sqrt(d_k)
    st = lib().attn_fwd_local(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, H, n, d_k, d_v, float(scale),
                              int(window), int(mask_mode), _ptr(key_lens), _stream_handle(stream))
    if st != ATTN_OK:
        raise AttnError(st, "attn_fwd_local")
    return out


def attn_fwd_f32(q, k, v, out, lse=None, scale=None, mask_mode=MASK_NONE, key_lens=None, stream=None):
    """float32 forward into caller-provided ``out`` (and optional ``lse``)."""
    return _call(lib().attn_fwd_f32, q, k, v, out, lse, scale, mask_mode, key_lens, stream, torch.float32,
                 "attn_fwd_f32")


def attention(q, k, v, scale=None, mask_mode=MASK_NONE, key_lens=None, with_lse=False, stream=None):
    """Allocating convenience wrapper: returns ``out`` (and ``lse``) for bf16 or float32 inputs."""
    B, H, n_q, _ = q.shape
    out = torch.empty((B, H, n_q, v.shape[3]), dtype=q.dtype, device=q.device)
    lse = torch.empty((B, H, n_q), dtype=torch.float32, device=q.device) if with_lse else None
    fn = attn_fwd if q.dtype == torch.bfloat16 else attn_fwd_f32
    fn(q, k, v, out, lse, scale, mask_mode, key_lens, stream)
    return (out, lse) if with_lse else out


def attn_decode_workspace_size(B, H, n_q, n_max, d) -> int:
    return int(lib().attn_decode_workspace_size(B, H, n_q, n_max, d))


def attn_decode(q, k_cache, v_cache, out, cache_lens, workspace, lse=None, scale=None, stream=None):
    """One decoding step: ``q [B,H,n_q,d]`` against caches ``[B,H,n_max,d]`` (bf16),
    ``cache_lens`` int32 ``[B]``, caller-provided ``workspace`` (a CUDA uint8 tensor of
    at least ``attn_decode_workspace_size`` bytes) and ``out`` (and optional ``lse``)."""
    for t, n in ((q, "q"), (k_cache, "k_cache"), (v_cache, "v_cache"), (out, "out")):
        _check(t, n, torch.bfloat16)
    B, H, n_q, d = q.shape
    n_max = k_cache.shape[2]
    if k_cache.shape != (B, H, n_max, d) or v_cache.shape != (B, H, n_max, d) or out.shape != q.shape:
        raise ValueError("shape mismatch between q, caches and out")
    _check(cache_lens, "cache_lens", torch.int32, 1)
    if lse is not None:
        _check(lse, "lse", torch.float32, 3)
    if not (workspace.is_cuda and workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous CUDA tensor")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    nbytes = workspace.numel() * workspace.element_size()
    st = lib().attn_decode(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(out), _ptr(lse), B, H, n_q, n_max, d,
                           float(scale), _ptr(cache_lens), _ptr(workspace), nbytes, _stream_handle(stream))
    if st != ATTN_OK:
        raise AttnError(st, "attn_decode")
    return out


NOALLOC_MAX_BYTES = 4 << 20  # ATTN_DECODE_NOALLOC_MAX_BYTES


def attn_decode_noalloc(q, k_cache, v_cache, out, cache_lens, lse=None, scale=None, stream=None):
    """attn_decode without a workspace argument, for callers that cannot allocate
    device memory (e.g. while capturing a CUDA graph): the library uses its own
    static device buffer of NOALLOC_MAX_BYTES, shared by every call on the device,
    so calls must not overlap on the GPU. The first call on a device does a
    one-time set-up and should come before any stream capture."""
    for t, n in ((q, "q"), (k_cache, "k_cache"), (v_cache, "v_cache"), (out, "out")):
        _check(t, n, torch.bfloat16)
    B, H, n_q, d = q.shape
    n_max = k_cache.shape[2]
    if k_cache.shape != (B, H, n_max, d) or v_cache.shape != (B, H, n_max, d) or out.shape != q.shape:
        raise ValueError("shape mismatch between q, caches and out")
    _check(cache_lens, "cache_lens", torch.int32, 1)
    if lse is not None:
        _check(lse, "lse", torch.float32, 3)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    st = lib().attn_decode_noalloc(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(out), _ptr(lse), B, H, n_q, n_max,
                                   d, float(scale), _ptr(cache_lens), _stream_handle(stream))
    if st != ATTN_OK:
        raise AttnError(st, "attn_decode_noalloc")
    return out


def attn_bwd_workspace_size(B, H, n_q, d=64, flags=0) -> int:
    return int(lib().attn_bwd_workspace_size(B, H, n_q, d, int(flags)))


def attn_bwd(q, k, v, out, dout, lse, dq, dk, dv, workspace, scale=None, mask_mode=MASK_NONE, key_lens=None,
             stream=None, flags=0):
    """Gradients of attn_fwd into caller-provided ``dq``, ``dk``, ``dv`` (bf16, shaped like
    q, k, v), given ``dout`` and the forward's ``out`` and fp32 ``lse``; ``workspace`` is a
    CUDA tensor of at least ``attn_bwd_workspace_size(B, H, n_q, d, flags)`` bytes;
    ``flags`` = BWD_DETERMINISTIC selects the bit-reproducible schedule."""
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (out, "out"), (dout, "dout"), (dq, "dq"), (dk, "dk"), (dv, "dv")):
        _check(t, n, torch.bfloat16)
    B, H, n_q, d_k = q.shape
    n_k, d_v = k.shape[2], v.shape[3]
    if (k.shape != (B, H, n_k, d_k) or v.shape != (B, H, n_k, d_v) or out.shape != (B, H, n_q, d_v)
            or dout.shape != out.shape or dq.shape != q.shape or dk.shape != k.shape or dv.shape != v.shape):
        raise ValueError("shape mismatch between q, k, v, out, dout and the gradients")
    _check(lse, "lse", torch.float32, 3)
    if lse.shape != (B, H, n_q):
        raise ValueError("lse must have shape [B, H, n_q]")
    if key_lens is not None:
        _check(key_lens, "key_lens", torch.int32, 1)
        if key_lens.shape != (B,):
            raise ValueError("key_lens must have shape [B]")
    if not (workspace.is_cuda and workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous CUDA tensor")
    if scale is None:
        scale = 1.0 / math.sqrt(d_k)
    nbytes = workspace.numel() * workspace.element_size()
    st = lib().attn_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(dout), _ptr(lse), _ptr(dq), _ptr(dk), _ptr(dv),
                        B, H, n_q, n_k, d_k, d_v, float(scale), int(mask_mode), _ptr(key_lens), int(flags),
                        _ptr(workspace), nbytes, _stream_handle(stream))
    if st != ATTN_OK:
        raise AttnError(st, "attn_bwd")
    return dq, dk, dv


def attn_bwd_local(q, k, v, out, dout, lse, dq, dk, dv, workspace, window, scale=None, mask_mode=MASK_NONE,
                   key_lens=None, stream=None, flags=0):
    """Gradients of attn_fwd_local (key j legal for query i only if |i - j| <= window, plus
    mask_mode); arguments and workspace as in attn_bwd, with n_q = n_k."""
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (out, "out"), (dout, "dout"), (dq, "dq"), (dk, "dk"), (dv, "dv")):
        _check(t, n, torch.bfloat16)
    B, H, n, d_k = q.shape
    d_v = v.shape[3]
    if (k.shape != (B, H, n, d_k) or v.shape != (B, H, n, d_v) or out.shape != (B, H, n, d_v)
            or dout.shape != out.shape or dq.shape != q.shape or dk.shape != k.shape or dv.shape != v.shape):
        raise ValueError("local attention is self-attention: q, k, v, out, dout and the gradients share B, H, n")
    _check(lse, "lse", torch.float32, 3)
    if lse.shape != (B, H, n):
        raise ValueError("lse must have shape [B, H, n]")
    if key_lens is not None:
        _check(key_lens, "key_lens", torch.int32, 1)
    if not (workspace.is_cuda and workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous CUDA tensor")
    if scale is None:
        scale = 1.0 / math.sqrt(d_k)
    nbytes = workspace.numel() * workspace.element_size()
    st = lib().attn_bwd_local(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(dout), _ptr(lse), _ptr(dq), _ptr(dk),
                              _ptr(dv), B, H, n, d_k, d_v, float(scale), int(window), int(mask_mode), _ptr(key_lens),
                              int(flags), _ptr(workspace), nbytes, _stream_handle(stream))
    if st != ATTN_OK:
        raise AttnError(st, "attn_bwd_local")
    return dq, dk, dv


def attn_bwd_host_workspace_size(B, H, n_q, n_k, d, mask_mode=MASK_NONE, flags=0) -> int:
    return int(lib().attn_bwd_host_workspace_size(B, H, n_q, n_k, d, int(mask_mode), int(flags)))


def attn_bwd_host(q, k, v, out, dout, lse, dq, dk, dv, workspace, scale=None, mask_mode=MASK_NONE, key_lens=None,
                  stream=None, flags=0):
    """attn_bwd on HOST tensors (pinned recommended): q, k, v, out, dout (bf16), lse
    (float32) and key_lens are read and dq, dk, dv written in host memory; the chunked
    copy/compute pipeline runs on the GPU with ``workspace`` (a CUDA uint8 tensor of
    attn_bwd_host_workspace_size bytes) and is asynchronous on ``stream``."""
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (out, "out"), (dout, "dout"), (dq, "dq"), (dk, "dk"), (dv, "dv")):
        if t.dtype != torch.bfloat16 or t.dim() != 4 or t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{n} must be a contiguous 4-D host bf16 tensor, got {t.dtype} {tuple(t.shape)}")
    B, H, n_q, d_k = q.shape
    n_k, d_v = k.shape[2], v.shape[3]
    if (k.shape != (B, H, n_k, d_k) or v.shape != (B, H, n_k, d_v) or out.shape != (B, H, n_q, d_v)
            or dout.shape != out.shape or dq.shape != q.shape or dk.shape != k.shape or dv.shape != v.shape):
        raise ValueError("shape mismatch between q, k, v, out, dout and the gradients")
    if lse.dtype != torch.float32 or lse.is_cuda or not lse.is_contiguous() or lse.shape != (B, H, n_q):
        raise ValueError("lse must be a contiguous host float32 tensor of shape [B, H, n_q]")
    if key_lens is not None and (key_lens.dtype != torch.int32 or key_lens.is_cuda or key_lens.shape != (B,)):
        raise ValueError("key_lens must be a host int32 tensor of shape [B]")
    if workspace.dtype != torch.uint8 or not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA uint8 tensor")
    if scale is None:
        scale = 1.0 / math.sqrt(d_k)
    st = lib().attn_bwd_host(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(dout), _ptr(lse), _ptr(dq), _ptr(dk),
                             _ptr(dv), B, H, n_q, n_k, d_k, d_v, float(scale), int(mask_mode), _ptr(key_lens),
                             int(flags), _ptr(workspace), workspace.numel(), _stream_handle(stream))
    if st != ATTN_OK:
        raise AttnError(st, "attn_bwd_host")
    return dq, dk, dv


def attn_mha_workspace_size(B, n_q, n_k, d_model, H, d) -> int:
    return int(lib().attn_mha_workspace_size(B, n_q, n_k, d_model, H, d))


def attn_mha_fwd(x_q, x_kv, w_q, w_k, w_v, w_o, out, H, workspace, b_q=None, b_k=None, b_v=None, b_o=None,
                 scale=None, mask_mode=MASK_NONE, key_lens=None, stream=None):
    """Multi-head attention layer into caller-provided ``out [B, n_q, d_model]`` (bf16):
    ``x_q [B,n_q,d_model]``, ``x_kv [B,n_k,d_model]``, ``w_q, w_k, w_v [d_model, H*d]``,
    ``w_o [H*d, d_model]`` (the paper's x W orientation), optional biases, and a CUDA
    ``workspace`` of at least ``attn_mha_workspace_size`` bytes."""
    for t, n in ((x_q, "x_q"), (x_kv, "x_kv"), (out, "out")):
        _check(t, n, torch.bfloat16, 3)
    for t, n in ((w_q, "w_q"), (w_k, "w_k"), (w_v, "w_v"), (w_o, "w_o")):
        _check(t, n, torch.bfloat16, 2)
    for t, n in ((b_q, "b_q"), (b_k, "b_k"), (b_v, "b_v"), (b_o, "b_o")):
        if t is not None:
            _check(t, n, torch.bfloat16, 1)
    B, n_q, d_model = x_q.shape
    n_k = x_kv.shape[1]
    d_k, d_v = w_q.shape[1] // H, w_v.shape[1] // H
    if (x_kv.shape != (B, n_k, d_model) or w_q.shape != (d_model, H * d_k) or w_k.shape != w_q.shape
            or w_v.shape != (d_model, H * d_v) or w_o.shape != (H * d_v, d_model) or out.shape != x_q.shape):
        raise ValueError("inconsistent multi-head attention shapes")
    if key_lens is not None:
        _check(key_lens, "key_lens", torch.int32, 1)
    if not (workspace.is_cuda and workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous CUDA tensor")
    if scale is None:
        scale = 1.0 / math.sqrt(d_k)
    nbytes = workspace.numel() * workspace.element_size()
    st = lib().attn_mha_fwd(_ptr(x_q), _ptr(x_kv), _ptr(w_q), _ptr(b_q), _ptr(w_k), _ptr(b_k), _ptr(w_v), _ptr(b_v),
                            _ptr(w_o), _ptr(b_o), _ptr(out), B, n_q, n_k, d_model, H, d_k, d_v, float(scale),
                            int(mask_mode), _ptr(key_lens), _ptr(workspace), nbytes, _stream_handle(stream))
    if st != ATTN_OK:
        raise AttnError(st, "attn_mha_fwd")
    return out


def attn_weights(q, k, lse, w, scale=None, mask_mode=MASK_NONE, key_lens=None, stream=None):
    """The softmax weights ``w [B, H, n_q, n_k]`` (float32, caller-provided) of bf16
    ``q``, ``k`` given the ``lse`` attn_fwd returned for the same inputs and mask."""
    _check(q, "q", torch.bfloat16)
    _check(k, "k", torch.bfloat16)
    _check(lse, "lse", torch.float32, 3)
    _check(w, "w", torch.float32)
    B, H, n_q, d = q.shape
    n_k = k.shape[2]
    if k.shape != (B, H, n_k, d) or lse.shape != (B, H, n_q) or w.shape != (B, H, n_q, n_k):
        raise ValueError(f"shape mismatch: q{tuple(q.shape)} k{tuple(k.shape)} lse{tuple(lse.shape)} w{tuple(w.shape)}")
    if key_lens is not None:
        _check(key_lens, "key_lens", torch.int32, 1)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    st = lib().attn_weights(_ptr(q), _ptr(k), _ptr(lse), _ptr(w), B, H, n_q, n_k, d, float(scale), int(mask_mode),
                            _ptr(key_lens), _stream_handle(stream))
    if st != ATTN_OK:
        raise AttnError(st, "attn_weights")
    return w


def attn_linear(x, w, y, bias=None, stream=None):
    """One projection ``y [M, N] = x [M, K] w [K, N] + bias [N]`` (bf16, row-major,
    caller-provided ``y``)."""
    _check(x, "x", torch.bfloat16, 2)
    _check(w, "w", torch.bfloat16, 2)
    _check(y, "y", torch.bfloat16, 2)
    if bias is not None:
        _check(bias, "bias", torch.bfloat16, 1)
    M, K = x.shape
    N = w.shape[1]
    if w.shape != (K, N) or y.shape != (M, N) or (bias is not None and bias.shape != (N,)):
        raise ValueError(f"shape mismatch: x{tuple(x.shape)} w{tuple(w.shape)} y{tuple(y.shape)}")
    st = lib().attn_linear(_ptr(x), _ptr(w), _ptr(bias), _ptr(y), M, N, K, _stream_handle(stream))
    if st != ATTN_OK:
        raise AttnError(st, "attn_linear")
    return y


def _device_of(t) -> int:
    """The device of a call's tensors: the current one, where its launches go."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"the tensors must be on a CUDA device, got {t.device}")
    if dev != _current_device():
        raise ValueError(f"the tensors are on {t.device}, the current device is cuda:{torch.cuda.current_device()}")
    return dev


_INT_MAX = 2 ** 31 - 1


def _int32(x) -> int:
    """The nearest number that a C int holds (ctypes would drop the upper bits)."""
    x = int(x)
    return x if -_INT_MAX <= x <= _INT_MAX else _INT_MAX if x > 0 else -_INT_MAX


def _raw_stream(stream, dev) -> int:
    return _current_stream(dev) if stream is None else _stream_handle(stream)


def _need(t, name, dtype, shape, dev):
    """Data pointer of a contiguous tensor of that type, shape and device."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {list(shape)} on cuda:{dev}, got "
                         f"{t.dtype} {list(t.shape)} with strides {t.stride()} on {t.device}")
    return t.data_ptr()


def _need_rows(t, name, shape, dev):
    """Data pointer and token stride of bf16 head rows by token, ``[..., heads, d]``: a token's
    heads side by side, tokens one stride apart (a view of a fused projection)."""
    st = t.stride()
    if t.dtype is torch.bfloat16 and t.shape == shape and t.get_device() == dev and st[-1] == 1:
        n, h, d = shape[-3:]
        if h == 1 or st[-2] == d:
            if len(shape) == 3 or shape[0] == 1:
                return t.data_ptr(), st[-3] if n > 1 else h * d
            if n == 1:
                return t.data_ptr(), st[0]
            if st[0] == n * st[1]:
                return t.data_ptr(), st[1]
    raise ValueError(f"{name} must be a bfloat16 tensor of shape {list(shape)} on cuda:{dev}, a token's heads side by "
                     f"side and tokens one stride apart, got {t.dtype} {list(t.shape)} with strides {st} on {t.device}")


def _need_table(cos_sin, dev):
    """Pointer, positions and columns of a rotation table; none without one."""
    if cos_sin is None:
        return None, 0, 0
    if cos_sin.dim() != 2:
        raise ValueError(f"cos_sin must be [n_pos, d_rot], got {list(cos_sin.shape)}")
    shape = cos_sin.shape
    return _need(cos_sin, "cos_sin", torch.float32, shape, dev), shape[0], shape[1]


def _need_workspace(workspace, dev):
    if workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on cuda:{dev}")
    return workspace.data_ptr(), workspace.nbytes


def attn_norm_rope(q, k, q_out, k_out, cos_sin, q_weight=None, k_weight=None, positions=None, eps=1e-6,
                   interleaved=False, stream=None):
    """RMS norm of every head (with weights) and position rotation, bf16: ``q [B, n, h_q, d]``
    and ``k [B, n, h_kv, d]`` token-major (views of a fused projection are fine) into
    ``q_out [B, h_q, n, d]`` and ``k_out [B, h_kv, n, d]``. ``cos_sin`` is float32
    ``[n_pos, d_rot]`` (cosines, then sines; None: no rotation), ``positions`` int32 ``[B, n]``
    or None for 0 .. n - 1; ``interleaved`` turns adjacent columns instead of the halves."""
    dev, bf16 = _device_of(q), torch.bfloat16
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError(f"q, k must be [B, n, heads, d], got {list(q.shape)} {list(k.shape)}")
    B, n, h_q, d = q.shape
    h_kv = k.shape[2]
    q_ptr, q_stride = _need_rows(q, "q", (B, n, h_q, d), dev)
    k_ptr, k_stride = _need_rows(k, "k", (B, n, h_kv, d), dev)
    table, n_pos, d_rot = _need_table(cos_sin, dev)
    st = lib().attn_norm_rope(
        q_ptr, k_ptr, q_stride, k_stride,
        None if q_weight is None else _need(q_weight, "q_weight", bf16, (d,), dev),
        None if k_weight is None else _need(k_weight, "k_weight", bf16, (d,), dev),
        float(eps), table, n_pos, d_rot,
        None if positions is None else _need(positions, "positions", torch.int32, (B, n), dev),
        _need(q_out, "q_out", bf16, (B, h_q, n, d), dev), _need(k_out, "k_out", bf16, (B, h_kv, n, d), dev),
        B, n, h_q, h_kv, d, ROPE_INTERLEAVED if interleaved else 0, _raw_stream(stream, dev))
    if st != ATTN_OK:
        raise AttnError(st, "attn_norm_rope")
    return q_out, k_out


def attn_norm_rope_bwd_workspace_size(B, n, h_q, h_kv, d) -> int:
    return int(lib().attn_norm_rope_bwd_workspace_size(B, n, h_q, h_kv, d))


def attn_norm_rope_bwd(q, k, dq_out, dk_out, dq, dk, workspace, cos_sin, q_weight=None, k_weight=None, dq_weight=None,
                       dk_weight=None, positions=None, eps=1e-6, interleaved=False, stream=None):
    """Gradients of attn_norm_rope: ``dq_out``, ``dk_out`` (shaped like its outputs) into
    ``dq``, ``dk`` (token-major like ``q``, ``k``) and, with a norm, float32 ``dq_weight``,
    ``dk_weight [d]``; ``workspace``: a CUDA tensor of at least
    ``attn_norm_rope_bwd_workspace_size`` bytes (None without a norm)."""
    dev, bf16, f32 = _device_of(q), torch.bfloat16, torch.float32
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError(f"q, k must be [B, n, heads, d], got {list(q.shape)} {list(k.shape)}")
    B, n, h_q, d = q.shape
    h_kv = k.shape[2]
    q_shape, k_shape = (B, n, h_q, d), (B, n, h_kv, d)
    q_ptr, q_stride = _need_rows(q, "q", q_shape, dev)
    k_ptr, k_stride = _need_rows(k, "k", k_shape, dev)
    dq_ptr, dq_stride = _need_rows(dq, "dq", q_shape, dev)
    dk_ptr, dk_stride = _need_rows(dk, "dk", k_shape, dev)
    table, n_pos, d_rot = _need_table(cos_sin, dev)
    ws_ptr, ws_bytes = (None, 0) if workspace is None else _need_workspace(workspace, dev)
    st = lib().attn_norm_rope_bwd(
        q_ptr, k_ptr, q_stride, k_stride,
        None if q_weight is None else _need(q_weight, "q_weight", bf16, (d,), dev),
        None if k_weight is None else _need(k_weight, "k_weight", bf16, (d,), dev),
        float(eps), table, n_pos, d_rot,
        None if positions is None else _need(positions, "positions", torch.int32, (B, n), dev),
        _need(dq_out, "dq_out", bf16, (B, h_q, n, d), dev), _need(dk_out, "dk_out", bf16, (B, h_kv, n, d), dev),
        dq_ptr, dk_ptr, dq_stride, dk_stride,
        None if dq_weight is None else _need(dq_weight, "dq_weight", f32, (d,), dev),
        None if dk_weight is None else _need(dk_weight, "dk_weight", f32, (d,), dev),
        B, n, h_q, h_kv, d, ROPE_INTERLEAVED if interleaved else 0, ws_ptr, ws_bytes, _raw_stream(stream, dev))
    if st != ATTN_OK:
        raise AttnError(st, "attn_norm_rope_bwd")
    return dq, dk


def _need_pages(k_pages, v_pages, k_scale, v_scale, h_kv, d, dev):
    """A paged cache ``[n_pages, h_kv, page_size, d]`` in bf16, or in float8_e4m3fn with its scales:
    flags, n_pages, page_size, the pages' and scales' pointers."""
    kind = k_pages.dtype
    e4m3 = kind is torch.float8_e4m3fn
    if k_pages.dim() != 4 or not (e4m3 or kind is torch.bfloat16):
        raise ValueError(f"k_pages must be [n_pages, h_kv, page_size, d] in bfloat16 or float8_e4m3fn, got {kind} "
                         f"{list(k_pages.shape)}")
    if (k_scale is not None) != e4m3 or (v_scale is not None) != e4m3:
        raise ValueError("k_scale and v_scale are required with an e4m3 cache, and only there")
    n_pages, _, page_size, _ = k_pages.shape
    shape = (n_pages, h_kv, page_size, d)
    k_ptr, v_ptr = _need(k_pages, "k_pages", kind, shape, dev), _need(v_pages, "v_pages", kind, shape, dev)
    if not e4m3:
        return 0, n_pages, page_size, k_ptr, v_ptr, None, None
    return (CACHE_E4M3, n_pages, page_size, k_ptr, v_ptr, _need(k_scale, "k_scale", torch.float32, (h_kv,), dev),
            _need(v_scale, "v_scale", torch.float32, (h_kv,), dev))


def attn_paged_append(k, v, k_pages, v_pages, positions, page_table, seq_ids=None, q=None, q_out=None, cos_sin=None,
                      q_weight=None, k_weight=None, k_scale=None, v_scale=None, eps=1e-6, interleaved=False,
                      stream=None):
    """Writes new tokens' keys (normalised and rotated as in attn_norm_rope) and values,
    ``k, v [T, h_kv, d]`` bf16, into the pages ``k_pages, v_pages [n_pages, h_kv, page_size, d]``
    (bf16, or float8_e4m3fn with the float32 scales ``k_scale, v_scale [h_kv]``), and the
    tokens' queries ``q [T, h_q, d]`` into ``q_out`` (contiguous). ``positions`` int32 ``[T]``
    (negative: padding, skipped), ``seq_ids`` int32 ``[T]`` (None: token x is sequence x's),
    ``page_table`` int32 ``[n_seqs, max_pages]``."""
    dev, bf16, i32 = _device_of(k), torch.bfloat16, torch.int32
    if k.dim() != 3 or page_table.dim() != 2:
        raise ValueError(f"k must be [T, h_kv, d], page_table [n_seqs, max_pages], got {list(k.shape)} "
                         f"{list(page_table.shape)}")
    T, h_kv, d = k.shape
    k_ptr, k_stride = _need_rows(k, "k", (T, h_kv, d), dev)
    v_ptr, v_stride = _need_rows(v, "v", (T, h_kv, d), dev)
    flags, n_pages, page_size, kp, vp, ks, vs = _need_pages(k_pages, v_pages, k_scale, v_scale, h_kv, d, dev)
    q_ptr = q_to = None
    h_q = q_stride = 0
    if (q is None) != (q_out is None):
        raise ValueError("q and q_out go together")
    if q is not None:
        if q.dim() != 3:
            raise ValueError(f"q must be [T, h_q, d], got {list(q.shape)}")
        h_q = q.shape[1]
        q_ptr, q_stride = _need_rows(q, "q", (T, h_q, d), dev)
        q_to = _need(q_out, "q_out", bf16, (T, h_q, d), dev)
    table, n_pos, d_rot = _need_table(cos_sin, dev)
    n_seqs, max_pages = page_table.shape
    st = lib().attn_paged_append(
        q_ptr, k_ptr, v_ptr, q_stride, k_stride, v_stride,
        None if q_weight is None else _need(q_weight, "q_weight", bf16, (d,), dev),
        None if k_weight is None else _need(k_weight, "k_weight", bf16, (d,), dev),
        float(eps), table, n_pos, d_rot, _need(positions, "positions", i32, (T,), dev),
        None if seq_ids is None else _need(seq_ids, "seq_ids", i32, (T,), dev),
        _need(page_table, "page_table", i32, (n_seqs, max_pages), dev), _int32(n_seqs), _int32(max_pages), q_to, kp, vp,
        n_pages, page_size, ks, vs, T, h_q, h_kv, d, flags | (ROPE_INTERLEAVED if interleaved else 0),
        _raw_stream(stream, dev))
    if st != ATTN_OK:
        raise AttnError(st, "attn_paged_append")
    return q_out


def attn_paged_decode_workspace_size(B, n_q, h_q, h_kv, d) -> int:
    return int(lib().attn_paged_decode_workspace_size(B, n_q, h_q, h_kv, d))


def attn_paged_decode(q, k_pages, v_pages, out, page_table, cache_lens, workspace, lse=None, scale=None, window=-1,
                      sinks=0, k_scale=None, v_scale=None, stream=None):
    """The newest ``n_q`` tokens of each sequence, ``q [B, n_q, h_q, d]`` bf16, attend over the
    paged cache (see attn_paged_append) of ``cache_lens`` int32 ``[B]`` tokens, the new ones
    included, into ``out`` (like ``q``) and optional float32 ``lse [B, n_q, h_q]``. ``window`` >= 0:
    only keys within that distance and the first ``sinks``. ``workspace``: a CUDA tensor of
    at least ``attn_paged_decode_workspace_size`` bytes."""
    dev, i32 = _device_of(q), torch.int32
    if q.dim() != 4 or k_pages.dim() != 4 or page_table.dim() != 2:
        raise ValueError(f"q must be [B, n_q, h_q, d], the pages [n_pages, h_kv, page_size, d], page_table "
                         f"[B, max_pages], got {list(q.shape)} {list(k_pages.shape)} {list(page_table.shape)}")
    B, n_q, h_q, d = shape = q.shape
    h_kv, max_pages = k_pages.shape[1], page_table.shape[1]
    flags, n_pages, page_size, kp, vp, ks, vs = _need_pages(k_pages, v_pages, k_scale, v_scale, h_kv, d, dev)
    ws_ptr, ws_bytes = _need_workspace(workspace, dev)
    st = lib().attn_paged_decode(
        _need(q, "q", torch.bfloat16, shape, dev), kp, vp, _need(out, "out", torch.bfloat16, shape, dev),
        None if lse is None else _need(lse, "lse", torch.float32, (B, n_q, h_q), dev),
        _need(page_table, "page_table", i32, (B, max_pages), dev), _need(cache_lens, "cache_lens", i32, (B,), dev),
        B, n_q, h_q, h_kv, d, n_pages, page_size, _int32(max_pages),
        1.0 / math.sqrt(d) if scale is None else float(scale), _int32(window), _int32(sinks), ks, vs, flags, ws_ptr,
        ws_bytes, _raw_stream(stream, dev))
    if st != ATTN_OK:
        raise AttnError(st, "attn_paged_decode")
    return out


def _need_heads(t, name, shape, dev):
    """Data pointer, token stride and head stride of a bf16 ``[tokens, heads, d]`` tensor, tokens or
    heads outermost."""
    st = t.stride()
    if t.dtype is not torch.bfloat16 or t.shape != shape or t.get_device() != dev or st[2] != 1:
        raise ValueError(f"{name} must be a bfloat16 tensor of shape {list(shape)} on cuda:{dev} with d side by side, got "
                         f"{t.dtype} {list(t.shape)} with strides {st} on {t.device}")
    return t.data_ptr(), st[0], st[1]


def _need_starts(starts, name, dev):
    """Data pointer and number of sequences of int32 offsets ``[n_seqs + 1]``."""
    if starts.dim() != 1 or starts.shape[0] < 2:
        raise ValueError(f"{name} must be [n_seqs + 1], got {list(starts.shape)}")
    return _need(starts, name, torch.int32, starts.shape, dev), starts.shape[0] - 1


def attn_packed_fwd_workspace_size(T_q, n_seqs, h_q, h_kv, d) -> int:
    return int(lib().attn_packed_fwd_workspace_size(_int32(T_q), _int32(n_seqs), _int32(h_q), _int32(h_kv), _int32(d)))


def attn_packed_fwd(q, k, v, out, q_starts, workspace, k_starts=None, lse=None, scale=None, mask_mode=MASK_NONE,
                    window=-1, stream=None):
    """Attention of packed sequences with shared key/value heads, bf16: ``q [T_q, h_q, d]`` and
    ``k, v [T_k, h_kv, d]`` (views with tokens or heads outermost) into ``out`` (shaped like ``q``) and
    optional float32 ``lse [T_q, h_q]``. Sequence b's queries are rows ``q_starts[b]`` to
    ``q_starts[b + 1] - 1`` (int32 ``[n_seqs + 1]``), its keys likewise by ``k_starts`` (None: the same
    rows). ``mask_mode`` MASK_NONE or MASK_CAUSAL, the last query at the last key's position;
    ``window`` >= 0: only keys within that distance. ``workspace``: a CUDA tensor of at least
    ``attn_packed_fwd_workspace_size`` bytes."""
    dev = _device_of(q)
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError(f"q must be [T_q, h_q, d], k [T_k, h_kv, d], got {list(q.shape)} {list(k.shape)}")
    T_q, h_q, d = q_shape = q.shape
    T_k, h_kv, _ = k.shape
    k_shape = (T_k, h_kv, d)
    q_ptr, *q_st = _need_heads(q, "q", q_shape, dev)
    k_ptr, *k_st = _need_heads(k, "k", k_shape, dev)
    v_ptr, *v_st = _need_heads(v, "v", k_shape, dev)
    o_ptr, *o_st = _need_heads(out, "out", q_shape, dev)
    starts, n_seqs = _need_starts(q_starts, "q_starts", dev)
    ws_ptr, ws_bytes = _need_workspace(workspace, dev)
    st = lib().attn_packed_fwd(
        q_ptr, k_ptr, v_ptr, o_ptr, None if lse is None else _need(lse, "lse", torch.float32, (T_q, h_q), dev), *q_st,
        *k_st, *v_st, *o_st, starts,
        None if k_starts is None else _need(k_starts, "k_starts", torch.int32, (n_seqs + 1,), dev), _int32(n_seqs),
        _int32(T_q), _int32(T_k), h_q, h_kv, d, 1.0 / math.sqrt(d) if scale is None else float(scale), int(mask_mode),
        _int32(window), ws_ptr, ws_bytes, _raw_stream(stream, dev))
    if st != ATTN_OK:
        raise AttnError(st, "attn_packed_fwd")
    return out


def attn_packed_bwd_workspace_size(T_q, T_k, n_seqs, h_q, h_kv, d) -> int:
    return int(lib().attn_packed_bwd_workspace_size(_int32(T_q), _int32(T_k), _int32(n_seqs), _int32(h_q), _int32(h_kv),
                                                    _int32(d)))


_SixteenStrides = ctypes.c_int64 * 16


def attn_packed_bwd(q, k, v, out, dout, lse, dq, dk, dv, q_starts, workspace, k_starts=None, scale=None,
                    mask_mode=MASK_NONE, window=-1, stream=None):
    """Gradients of attn_packed_fwd into ``dq`` (shaped like ``q``), ``dk`` and ``dv`` (like ``k``, ``v``), given
    ``dout`` and the forward's ``out`` and float32 ``lse``; views as there. ``workspace``: a CUDA tensor of
    at least ``attn_packed_bwd_workspace_size`` bytes."""
    dev = _device_of(q)
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError(f"q must be [T_q, h_q, d], k [T_k, h_kv, d], got {list(q.shape)} {list(k.shape)}")
    T_q, h_q, d = q_shape = q.shape
    T_k, h_kv, _ = k.shape
    k_shape = (T_k, h_kv, d)
    ptrs, strides = [], []
    for t, name, shape in ((q, "q", q_shape), (k, "k", k_shape), (v, "v", k_shape), (out, "out", q_shape),
                           (dout, "dout", q_shape), (dq, "dq", q_shape), (dk, "dk", k_shape), (dv, "dv", k_shape)):
        ptr, ts, hs = _need_heads(t, name, shape, dev)
        ptrs.append(ptr)
        strides += (ts, hs)
    starts, n_seqs = _need_starts(q_starts, "q_starts", dev)
    ws_ptr, ws_bytes = _need_workspace(workspace, dev)
    st = lib().attn_packed_bwd(
        *ptrs[:5], _need(lse, "lse", torch.float32, (T_q, h_q), dev), *ptrs[5:], _SixteenStrides(*strides), starts,
        None if k_starts is None else _need(k_starts, "k_starts", torch.int32, (n_seqs + 1,), dev), _int32(n_seqs),
        _int32(T_q), _int32(T_k), h_q, h_kv, d, 1.0 / math.sqrt(d) if scale is None else float(scale), int(mask_mode),
        _int32(window), ws_ptr, ws_bytes, _raw_stream(stream, dev))
    if st != ATTN_OK:
        raise AttnError(st, "attn_packed_bwd")
    return dq, dk, dv


def attn_paged_chunk_workspace_size(T, n_seqs, h_q, h_kv, d) -> int:
    return int(lib().attn_paged_chunk_workspace_size(_int32(T), _int32(n_seqs), _int32(h_q), _int32(h_kv), _int32(d)))


def attn_paged_chunk(q, k_pages, v_pages, out, q_starts, page_table, cache_lens, workspace, lse=None, scale=None,
                     window=-1, sinks=0, k_scale=None, v_scale=None, stream=None):
    """New tokens of every sequence, any number of them, attend over the paged cache (see
    attn_paged_append) that holds them already: ``q [T, h_q, d]`` bf16 into ``out`` (like ``q``) and
    optional float32 ``lse [T, h_q]``. Sequence b's new tokens are rows ``q_starts[b]`` to
    ``q_starts[b + 1] - 1`` (int32 ``[n_seqs + 1]``), the last of its ``cache_lens[b]`` cached ones (int32
    ``[n_seqs]``); ``page_table`` int32 ``[n_seqs, max_pages]``. ``window`` >= 0: only keys within that
    distance and the first ``sinks``. ``workspace``: a CUDA tensor of at least
    ``attn_paged_chunk_workspace_size`` bytes."""
    dev, i32 = _device_of(q), torch.int32
    if q.dim() != 3 or k_pages.dim() != 4 or page_table.dim() != 2:
        raise ValueError(f"q must be [T, h_q, d], the pages [n_pages, h_kv, page_size, d], page_table [n_seqs, max_pages], "
                         f"got {list(q.shape)} {list(k_pages.shape)} {list(page_table.shape)}")
    T, h_q, d = shape = q.shape
    h_kv, max_pages = k_pages.shape[1], page_table.shape[1]
    starts, n_seqs = _need_starts(q_starts, "q_starts", dev)
    flags, n_pages, page_size, kp, vp, ks, vs = _need_pages(k_pages, v_pages, k_scale, v_scale, h_kv, d, dev)
    ws_ptr, ws_bytes = _need_workspace(workspace, dev)
    st = lib().attn_paged_chunk(
        _need(q, "q", torch.bfloat16, shape, dev), kp, vp, _need(out, "out", torch.bfloat16, shape, dev),
        None if lse is None else _need(lse, "lse", torch.float32, (T, h_q), dev), starts,
        _need(page_table, "page_table", i32, (n_seqs, max_pages), dev),
        _need(cache_lens, "cache_lens", i32, (n_seqs,), dev), _int32(n_seqs), _int32(T), h_q, h_kv, d, n_pages, page_size,
        _int32(max_pages), 1.0 / math.sqrt(d) if scale is None else float(scale), _int32(window), _int32(sinks), ks, vs,
        flags, ws_ptr, ws_bytes, _raw_stream(stream, dev))
    if st != ATTN_OK:
        raise AttnError(st, "attn_paged_chunk")
    return out


def _internal_arm_wait_timeout(wait_ns: int, skip_v_tile: int) -> None:
    """Test hook (not part of the C ABI header): the next plain d = 64 forward launch
    made on this host thread gives up its waits after ``wait_ns`` and never copies the
    V tile of K/V tile ``skip_v_tile``, so it ends through the bounded-wait abort path."""
    lib().attn_internal_arm_wait_timeout(int(wait_ns), int(skip_v_tile))


def _internal_arm_chunk_give_up(v_tile: int) -> None:
    """Test hook (not part of the C ABI header): in the next attn_paged_chunk call made on this host thread the
    copying warps of V give up before their tile ``v_tile``, as if a wait had run out there."""
    lib().attn_internal_arm_chunk_give_up(int(v_tile))


def attn_fault_status(stream=None, clear=True):
    """(status, raw fault bits) after synchronising ``stream``."""
    code = ctypes.c_uint32(0)
    st = lib().attn_fault_status(_stream_handle(stream), int(clear), ctypes.byref(code))
    return st, code.value
