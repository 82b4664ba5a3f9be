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
        L.attn_fault_status.argtypes = [vp, i, ctypes.POINTER(ctypes.c_uint32)]
        L.attn_fault_status.restype = i
        L.attn_status_string.argtypes = [i]
        L.attn_status_string.restype = ctypes.c_char_p
        L.attn_internal_arm_wait_timeout.argtypes = [ctypes.c_ulonglong, i]
        L.attn_internal_arm_wait_timeout.restype = None
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().attn_status_string(int(status)).decode()


def _stream_handle(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
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


def _same_device(first, *others):
    """The launch goes to the current device: every tensor has to be there."""
    dev = first.get_device()
    if dev != torch.cuda.current_device():
        raise ValueError(f"the tensors are on cuda:{dev}, the current device is cuda:{torch.cuda.current_device()}")
    for t in others:
        if t is not None and t.get_device() != dev:
            raise ValueError("all tensors must be on one device")


def _check_rows(t, name, ndim):
    """bf16 head rows by token, [..., heads, d]: a token's heads side by side, tokens one stride apart."""
    if t.dtype != torch.bfloat16 or t.dim() != ndim or not t.is_cuda:
        raise ValueError(f"{name} must be a {ndim}-D CUDA bfloat16 tensor, got {t.dtype} {tuple(t.shape)}")
    st, sh = t.stride(), t.shape
    if (st[-1] != 1 or (sh[-2] != 1 and st[-2] != sh[-1])
            or (ndim == 4 and sh[0] != 1 and sh[1] != 1 and st[0] != sh[1] * st[1])):
        raise ValueError(f"{name}: a token's heads must lie side by side and tokens one stride apart, got strides {st}")


def _row_stride(t):
    """Elements between tokens; of a single token, those of its heads."""
    if t.dim() == 4 and t.shape[1] == 1:
        return t.stride(0) if t.shape[0] > 1 else t.shape[2] * t.shape[3]
    return t.stride(-3) if t.shape[-3] > 1 else t.shape[-2] * t.shape[-1]


def _check_rotation(cos_sin, q_weight, k_weight, d):
    for t, n in ((q_weight, "q_weight"), (k_weight, "k_weight")):
        if t is not None:
            _check(t, n, torch.bfloat16, 1)
            if t.shape[0] != d:
                raise ValueError(f"{n} must have shape [{d}]")
    if cos_sin is None:
        return 0, 0
    _check(cos_sin, "cos_sin", torch.float32, 2)
    return cos_sin.shape


def attn_norm_rope(q, k, q_out, k_out, cos_sin, q_weight=None, k_weight=None, positions=None, eps=1e-6,
                   interleaved=False, stream=None):
    """RMS norm of every head (with weights) and position rotation, bf16: ``q [B, n, h_q, d]``
    and ``k [B, n, h_kv, d]`` token-major (views of a fused projection are fine) into
    ``q_out [B, h_q, n, d]`` and ``k_out [B, h_kv, n, d]``. ``cos_sin`` is float32
    ``[n_pos, d_rot]`` (cosines, then sines; None: no rotation), ``positions`` int32 ``[B, n]``
    or None for 0 .. n - 1; ``interleaved`` turns adjacent columns instead of the halves."""
    _check_rows(q, "q", 4)
    _check_rows(k, "k", 4)
    _check(q_out, "q_out", torch.bfloat16)
    _check(k_out, "k_out", torch.bfloat16)
    B, n, h_q, d = q.shape
    h_kv = k.shape[2]
    if k.shape != (B, n, h_kv, d) or q_out.shape != (B, h_q, n, d) or k_out.shape != (B, h_kv, n, d):
        raise ValueError(f"shape mismatch: q{tuple(q.shape)} k{tuple(k.shape)} q_out{tuple(q_out.shape)} "
                         f"k_out{tuple(k_out.shape)}")
    n_pos, d_rot = _check_rotation(cos_sin, q_weight, k_weight, d)
    if positions is not None:
        _check(positions, "positions", torch.int32, 2)
        if positions.shape != (B, n):
            raise ValueError("positions must have shape [B, n]")
    _same_device(q, k, q_out, k_out, cos_sin, q_weight, k_weight, positions)
    st = lib().attn_norm_rope(_ptr(q), _ptr(k), _row_stride(q), _row_stride(k), _ptr(q_weight), _ptr(k_weight),
                              float(eps), _ptr(cos_sin), n_pos, d_rot, _ptr(positions), _ptr(q_out), _ptr(k_out), B, n,
                              h_q, h_kv, d, ROPE_INTERLEAVED if interleaved else 0, _stream_handle(stream))
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
    for t, m in ((q, "q"), (k, "k"), (dq, "dq"), (dk, "dk")):
        _check_rows(t, m, 4)
    _check(dq_out, "dq_out", torch.bfloat16)
    _check(dk_out, "dk_out", torch.bfloat16)
    B, n, h_q, d = q.shape
    h_kv = k.shape[2]
    if (k.shape != (B, n, h_kv, d) or dq_out.shape != (B, h_q, n, d) or dk_out.shape != (B, h_kv, n, d)
            or dq.shape != q.shape or dk.shape != k.shape):
        raise ValueError("shape mismatch between q, k, their gradients and the outputs' gradients")
    n_pos, d_rot = _check_rotation(cos_sin, q_weight, k_weight, d)
    for t, m in ((dq_weight, "dq_weight"), (dk_weight, "dk_weight")):
        if t is not None:
            _check(t, m, torch.float32, 1)
            if t.shape[0] != d:
                raise ValueError(f"{m} must have shape [{d}]")
    if positions is not None:
        _check(positions, "positions", torch.int32, 2)
        if positions.shape != (B, n):
            raise ValueError("positions must have shape [B, n]")
    if workspace is not None and not (workspace.is_cuda and workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous CUDA tensor")
    _same_device(q, k, dq_out, dk_out, dq, dk, workspace, cos_sin, q_weight, k_weight, dq_weight, dk_weight, positions)
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib().attn_norm_rope_bwd(_ptr(q), _ptr(k), _row_stride(q), _row_stride(k), _ptr(q_weight), _ptr(k_weight),
                                  float(eps), _ptr(cos_sin), n_pos, d_rot, _ptr(positions), _ptr(dq_out), _ptr(dk_out),
                                  _ptr(dq), _ptr(dk), _row_stride(dq), _row_stride(dk), _ptr(dq_weight),
                                  _ptr(dk_weight), B, n, h_q, h_kv, d, ROPE_INTERLEAVED if interleaved else 0,
                                  _ptr(workspace), nbytes, _stream_handle(stream))
    if st != ATTN_OK:
        raise AttnError(st, "attn_norm_rope_bwd")
    return dq, dk


def _check_pages(k_pages, v_pages, k_scale, v_scale, page_table, h_kv, d):
    """Flags of a paged cache ``[n_pages, h_kv, page_size, d]`` in bf16 or float8_e4m3fn."""
    e4m3 = k_pages.dtype == torch.float8_e4m3fn
    for t, n in ((k_pages, "k_pages"), (v_pages, "v_pages")):
        _check(t, n, torch.float8_e4m3fn if e4m3 else torch.bfloat16)
    if k_pages.shape != v_pages.shape or k_pages.shape[1] != h_kv or k_pages.shape[3] != d:
        raise ValueError(f"k_pages, v_pages must be [n_pages, {h_kv}, page_size, {d}], got {tuple(k_pages.shape)} "
                         f"{tuple(v_pages.shape)}")
    _check(page_table, "page_table", torch.int32, 2)
    for t, n in ((k_scale, "k_scale"), (v_scale, "v_scale")):
        if (t is not None) != e4m3:
            raise ValueError(f"{n} is required with an e4m3 cache, and only there")
        if t is not None:
            _check(t, n, torch.float32, 1)
            if t.shape[0] != h_kv:
                raise ValueError(f"{n} must have shape [{h_kv}]")
    return CACHE_E4M3 if e4m3 else 0


def attn_paged_append(k, v, k_pages, v_pages, positions, page_table, seq_ids=None, q=None, q_out=None, cos_sin=None,
                      q_weight=None, k_weight=None, k_scale=None, v_scale=None, eps=1e-6, interleaved=False,
                      stream=None):
    """Writes new tokens' keys (normalised and rotated as in attn_norm_rope) and values,
    ``k, v [T, h_kv, d]`` bf16, into the pages ``k_pages, v_pages [n_pages, h_kv, page_size, d]``
    (bf16, or float8_e4m3fn with the float32 scales ``k_scale, v_scale [h_kv]``), and the
    tokens' queries ``q [T, h_q, d]`` into ``q_out`` (contiguous). ``positions`` int32 ``[T]``
    (negative: padding, skipped), ``seq_ids`` int32 ``[T]`` (None: token x is sequence x's),
    ``page_table`` int32 ``[n_seqs, max_pages]``."""
    _check_rows(k, "k", 3)
    _check_rows(v, "v", 3)
    T, h_kv, d = k.shape
    if v.shape != k.shape:
        raise ValueError(f"shape mismatch: k{tuple(k.shape)} v{tuple(v.shape)}")
    flags = _check_pages(k_pages, v_pages, k_scale, v_scale, page_table, h_kv, d)
    h_q = q_stride = 0
    if (q is None) != (q_out is None):
        raise ValueError("q and q_out go together")
    if q is not None:
        _check_rows(q, "q", 3)
        _check(q_out, "q_out", torch.bfloat16, 3)
        h_q, q_stride = q.shape[1], _row_stride(q)
        if q.shape != (T, h_q, d) or q_out.shape != q.shape:
            raise ValueError(f"shape mismatch: q{tuple(q.shape)} q_out{tuple(q_out.shape)} k{tuple(k.shape)}")
    n_pos, d_rot = _check_rotation(cos_sin, q_weight, k_weight, d)
    _check(positions, "positions", torch.int32, 1)
    if positions.shape[0] != T:
        raise ValueError("positions must have shape [T]")
    if seq_ids is not None:
        _check(seq_ids, "seq_ids", torch.int32, 1)
        if seq_ids.shape[0] != T:
            raise ValueError("seq_ids must have shape [T]")
    _same_device(k, v, k_pages, v_pages, positions, page_table, seq_ids, q, q_out, cos_sin, q_weight, k_weight,
                 k_scale, v_scale)
    st = lib().attn_paged_append(_ptr(q), _ptr(k), _ptr(v), q_stride, _row_stride(k), _row_stride(v), _ptr(q_weight),
                                 _ptr(k_weight), float(eps), _ptr(cos_sin), n_pos, d_rot, _ptr(positions),
                                 _ptr(seq_ids), _ptr(page_table), page_table.shape[0], page_table.shape[1],
                                 _ptr(q_out), _ptr(k_pages), _ptr(v_pages), k_pages.shape[0], k_pages.shape[2],
                                 _ptr(k_scale), _ptr(v_scale), T, h_q, h_kv, d,
                                 flags | (ROPE_INTERLEAVED if interleaved else 0), _stream_handle(stream))
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
    _check(q, "q", torch.bfloat16)
    _check(out, "out", torch.bfloat16)
    B, n_q, h_q, d = q.shape
    h_kv = k_pages.shape[1] if k_pages.dim() == 4 else 0
    flags = _check_pages(k_pages, v_pages, k_scale, v_scale, page_table, h_kv, d)
    _check(cache_lens, "cache_lens", torch.int32, 1)
    if out.shape != q.shape or page_table.shape[0] != B or cache_lens.shape[0] != B:
        raise ValueError("shape mismatch between q, out, page_table and cache_lens")
    if lse is not None:
        _check(lse, "lse", torch.float32, 3)
        if lse.shape != (B, n_q, h_q):
            raise ValueError("lse must have shape [B, n_q, h_q]")
    if not (workspace.is_cuda and workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous CUDA tensor")
    _same_device(q, k_pages, v_pages, out, page_table, cache_lens, workspace, lse, k_scale, v_scale)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    st = lib().attn_paged_decode(_ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(out), _ptr(lse), _ptr(page_table),
                                 _ptr(cache_lens), B, n_q, h_q, h_kv, d, k_pages.shape[0], k_pages.shape[2],
                                 page_table.shape[1], float(scale), int(window), int(sinks), _ptr(k_scale),
                                 _ptr(v_scale), flags, _ptr(workspace), workspace.numel() * workspace.element_size(),
                                 _stream_handle(stream))
    if st != ATTN_OK:
        raise AttnError(st, "attn_paged_decode")
    return out


def _internal_arm_wait_timeout(wait_ns: int, skip_v_tile: int) -> None:
    """Test hook (not part of the C ABI header): the next plain d = 64 forward launch
    made on this host thread gives up its waits after ``wait_ns`` and never copies the
    V tile of K/V tile ``skip_v_tile``, so it ends through the bounded-wait abort path."""
    lib().attn_internal_arm_wait_timeout(int(wait_ns), int(skip_v_tile))


def attn_fault_status(stream=None, clear=True):
    """(status, raw fault bits) after synchronising ``stream``."""
    code = ctypes.c_uint32(0)
    st = lib().attn_fault_status(_stream_handle(stream), int(clear), ctypes.byref(code))
    return st, code.value
