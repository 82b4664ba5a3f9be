"""The entry points for packed sequences and chunks over a paged cache reject bad arguments with the
documented status codes, without a GPU (argument validation returns before any CUDA call; the
placeholder pointers are never read)."""
import ctypes

import pytest
import torch

from transformer_scaled_dot_mha_gb300 import attn, build


@pytest.fixture(scope="module")
def L():
    build.build()
    return attn.lib()


BIG = 1 << 34  # more than any workspace that is asked for here
PACKED = dict(q=16, k=32, v=48, out=64, lse=80, q_stride=512, q_head=64, k_stride=512, k_head=64, v_stride=512,
              v_head=64, out_stride=256, out_head=64, q_starts=96, k_starts=None, n_seqs=3, T_q=40, T_k=40, h_q=4,
              h_kv=2, d=64, scale=0.125, mask_mode=1, window=-1, ws=256, nbytes=BIG, stream=None)


@pytest.mark.parametrize("bad", [
    dict(q=None), dict(k=None), dict(v=None), dict(out=None), dict(q_starts=None), dict(ws=None), dict(q=24), dict(k=8),
    dict(out=72), dict(lse=82), dict(q_starts=98), dict(k_starts=33), dict(ws=128),
    dict(q_stride=516), dict(q_head=60), dict(q_stride=0), dict(k_stride=-512), dict(q_head=0), dict(v_head=32),
    dict(q_stride=192), dict(k_stride=64, k_head=128), dict(out_stride=64, out_head=64), dict(q_stride=1 << 50),
    dict(n_seqs=0), dict(T_q=0), dict(T_k=0), dict(h_q=0), dict(h_kv=0), dict(h_q=5), dict(d=0), dict(h_kv=-2),
    dict(T_q=1 << 28), dict(T_k=1 << 28), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("inf")),
    dict(scale=float("nan")), dict(mask_mode=2), dict(mask_mode=3), dict(mask_mode=-1), dict(window=-2), dict(nbytes=1000),
])
def test_packed_fwd_invalid_arguments(L, bad):
    assert L.attn_packed_fwd(*dict(PACKED, **bad).values()) == attn.ATTN_ERR_INVALID


def test_packed_fwd_unsupported_shapes(L):
    for bad in (dict(d=96), dict(d=256), dict(h_q=129, h_kv=1), dict(n_seqs=1 << 27, h_q=16, h_kv=8)):
        assert L.attn_packed_fwd(*dict(PACKED, **bad).values()) == attn.ATTN_ERR_UNSUPPORTED, bad


BWD = dict(q=16, k=32, v=48, out=64, dout=80, lse=96, dq=112, dk=128, dv=144, strides=[512, 64] * 8, q_starts=160,
           k_starts=None, n_seqs=3, T_q=40, T_k=40, h_q=4, h_kv=2, d=64, scale=0.125, mask_mode=1, window=-1, ws=256,
           nbytes=BIG, stream=None)


def bwd(L, **bad):
    a = dict(BWD, **bad)
    if a["strides"] is not None:
        a["strides"] = (ctypes.c_int64 * 16)(*a["strides"])
    return L.attn_packed_bwd(*a.values())


@pytest.mark.parametrize("bad", [
    *[{x: None} for x in ("q", "k", "v", "out", "dout", "lse", "dq", "dk", "dv", "strides", "q_starts", "ws")],
    *[{x: 24} for x in ("q", "k", "v", "out", "dout", "dq", "dk", "dv", "ws")],
    *[dict(strides=[512, 64] * i + [128, 64] + [512, 64] * (7 - i)) for i in (0, 3, 4, 5)],  # 4 heads in 128 columns
    *[dict(strides=[512, 64] * i + [64, 64] + [512, 64] * (7 - i)) for i in (1, 2, 6, 7)],
    dict(strides=[512, 60] + [512, 64] * 7), dict(lse=97), dict(q_starts=161), dict(k_starts=2), dict(n_seqs=0),
    dict(T_q=0), dict(T_k=1 << 28), dict(h_q=3), dict(scale=0.0), dict(scale=float("nan")), dict(mask_mode=2),
    dict(window=-5), dict(nbytes=1 << 20),
])
def test_packed_bwd_invalid_arguments(L, bad):
    assert bwd(L, **bad) == attn.ATTN_ERR_INVALID


def test_packed_bwd_unsupported_shapes(L):
    for bad in (dict(d=96), dict(h_q=129, h_kv=1)):
        assert bwd(L, **bad) == attn.ATTN_ERR_UNSUPPORTED, bad


def test_packed_bwd_workspace_size():
    size = attn.attn_packed_bwd_workspace_size
    assert size(0, 1, 1, 1, 1, 64) == 0 and size(1, 0, 1, 1, 1, 64) == 0 and size(1, 1, 0, 1, 1, 64) == 0
    assert size(1, 1, 1, 3, 2, 64) == 0 and size(1, 1, 1, 1, 1, 32) == 0
    assert 0 < size(1, 1, 1, 8, 8, 128) < size(1 << 20, 1 << 20, 100, 8, 8, 128)


def test_workspace_sizes(L):
    for size in (attn.attn_packed_fwd_workspace_size, attn.attn_paged_chunk_workspace_size):
        assert size(0, 1, 1, 1, 64) == 0 and size(1, 0, 1, 1, 64) == 0 and size(1, 1, 3, 2, 64) == 0
        assert size(1, 1, 1, 1, 96) == 0 and size(1, 1, 129, 1, 64) == 0 and size(1 << 31, 1, 1, 1, 64) == 0
        a, b = size(1, 1, 8, 8, 64), size(1 << 20, 1000, 8, 8, 64)
        assert 0 < a < b < a + (1 << 24)  # the list grows with the tokens, the partial results do not


CHUNK = dict(q=16, kp=32, vp=48, out=64, lse=None, q_starts=80, table=96, lens=112, n_seqs=3, T=40, h_q=4, h_kv=2, d=64,
             n_pages=9, page_size=16, max_pages=4, scale=0.125, window=-1, sinks=0, k_scale=None, v_scale=None, flags=0,
             ws=256, nbytes=BIG, stream=None)


@pytest.mark.parametrize("bad", [
    dict(q=None), dict(kp=None), dict(vp=None), dict(out=None), dict(q_starts=None), dict(table=None), dict(lens=None),
    dict(ws=None), dict(q=8), dict(kp=24), dict(out=72), dict(lse=2), dict(q_starts=82), dict(table=97), dict(lens=114),
    dict(ws=16), dict(n_seqs=0), dict(T=0), dict(h_q=3), dict(h_kv=0), dict(d=-64), dict(n_pages=0), dict(page_size=0),
    dict(max_pages=0), dict(n_pages=1 << 30), dict(max_pages=1 << 30), dict(scale=0.0), dict(scale=float("nan")),
    dict(window=-2), dict(sinks=-1), dict(k_scale=128), dict(flags=2), dict(flags=2, k_scale=128), dict(flags=1),
    dict(flags=2, k_scale=128, v_scale=130), dict(nbytes=1000), dict(T=1 << 28),
])
def test_paged_chunk_invalid_arguments(L, bad):
    assert L.attn_paged_chunk(*dict(CHUNK, **bad).values()) == attn.ATTN_ERR_INVALID


def test_paged_chunk_unsupported_shapes(L):
    for bad in (dict(d=96), dict(h_q=258, h_kv=2)):
        assert L.attn_paged_chunk(*dict(CHUNK, **bad).values()) == attn.ATTN_ERR_UNSUPPORTED, bad


def test_host_tensors_are_refused_as_values():
    x, pages, i32 = torch.zeros(3, 2, 64, dtype=torch.bfloat16), torch.zeros(1, 2, 16, 64, dtype=torch.bfloat16), torch.int32
    at = torch.zeros(2, dtype=i32)
    with pytest.raises(ValueError, match="CUDA"):
        attn.attn_packed_fwd(x, x, x, x, at, x)
    with pytest.raises(ValueError, match="CUDA"):
        attn.attn_paged_chunk(x, pages, pages, x, at, torch.zeros(1, 1, dtype=i32), torch.zeros(1, dtype=i32), x)
