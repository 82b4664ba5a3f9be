"""The norm + rotation, paged append and paged decode entry points reject bad arguments with
the documented status codes, without a GPU (argument validation returns before any CUDA
call; the placeholder pointers are never read)."""
import pytest

from transformer_scaled_dot_mha_gb300 import attn, build


@pytest.fixture(scope="module")
def L():
    build.build()
    return attn.lib()


ROPE = dict(q=16, k=32, q_stride=512, k_stride=512, q_weight=48, k_weight=64, eps=1e-6, cos_sin=80, n_pos=10, d_rot=64,
            positions=None, q_out=96, k_out=112, B=2, n=10, h_q=4, h_kv=2, d=64, flags=0, stream=None)


@pytest.mark.parametrize("bad", [
    dict(q=None), dict(k=None), dict(q_out=None), dict(k_out=None), dict(q=24), dict(k_out=104),
    dict(q_stride=255), dict(q_stride=248), dict(k_stride=100), dict(k_stride=1 << 50),
    dict(q_weight=None), dict(k_weight=None), dict(q_weight=50), dict(eps=-1e-6), dict(eps=float("nan")),
    dict(cos_sin=None), dict(cos_sin=84), dict(n_pos=0), dict(n_pos=9), dict(d_rot=-16), dict(d_rot=80),
    dict(positions=2), dict(B=0), dict(n=-1), dict(h_q=0), dict(h_kv=0), dict(d=0), dict(flags=2), dict(flags=4),
    dict(B=1 << 20, n=1 << 20, positions=128),
])
def test_norm_rope_invalid_arguments(L, bad):
    assert L.attn_norm_rope(*dict(ROPE, **bad).values()) == attn.ATTN_ERR_INVALID


def test_norm_rope_unsupported_shapes(L):
    for bad in (dict(d=96, d_rot=64), dict(d_rot=24), dict(d=256)):
        a = dict(ROPE, q_stride=1024, k_stride=1024, **bad)
        assert L.attn_norm_rope(*a.values()) == attn.ATTN_ERR_UNSUPPORTED


def test_norm_rope_bwd_argument_checks(L):
    size = attn.attn_norm_rope_bwd_workspace_size
    need = size(2, 10, 4, 2, 64)
    assert need > 0 and need % (64 * 4) == 0
    assert size(0, 1, 1, 1, 64) == 0 and size(1, 1, 1, 0, 64) == 0 and size(1, 1, 1, 1, 96) == 0
    assert size(16, 1 << 20, 32, 8, 128) <= (4 * 152 + 2) * 128 * 4  # does not grow with the tokens
    a = {x: ROPE[x] for x in list(ROPE)[:11]}
    a |= dict(dq_out=96, dk_out=112, dq=128, dk=144, dq_stride=512, dk_stride=512, dq_weight=160, dk_weight=176)
    a |= {x: ROPE[x] for x in ("B", "n", "h_q", "h_kv", "d", "flags")} | dict(ws=192, nbytes=need, stream=None)
    for bad in (dict(dq_out=None), dict(dk_out=None), dict(dq=None), dict(dk=None), dict(dq_weight=None),
                dict(dk_weight=None), dict(ws=None), dict(ws=200), dict(nbytes=need - 1), dict(dq_stride=128),
                dict(dk_stride=129), dict(q=None), dict(flags=8), dict(q_weight=None),
                dict(q_weight=None, k_weight=None)):  # no norm, yet gradients of its weights asked for
        assert L.attn_norm_rope_bwd(*dict(a, **bad).values()) == attn.ATTN_ERR_INVALID, bad
    assert L.attn_norm_rope_bwd(*dict(a, d=96, q_stride=1024, k_stride=1024).values()) == attn.ATTN_ERR_UNSUPPORTED


APPEND = dict(q=16, k=32, v=48, q_stride=256, k_stride=128, v_stride=128, q_weight=64, k_weight=80, eps=1e-6,
              cos_sin=96, n_pos=10, d_rot=64, positions=112, seq_ids=128, page_table=144, n_seqs=3, max_pages=4, q_out=160,
              k_pages=176, v_pages=192, n_pages=9, page_size=16, k_scale=None, v_scale=None, T=5, h_q=4, h_kv=2, d=64,
              flags=0, stream=None)


@pytest.mark.parametrize("bad", [
    dict(k=None), dict(v=None), dict(k_pages=None), dict(v_pages=None), dict(positions=None), dict(page_table=None),
    dict(q_out=None), dict(q=None), dict(q=None, q_out=None), dict(q_weight=None), dict(k_weight=None),
    dict(seq_ids=None), dict(seq_ids=2), dict(positions=2), dict(page_table=2), dict(k_pages=8), dict(v=40),
    dict(q_stride=64), dict(k_stride=127), dict(v_stride=0), dict(T=0), dict(h_q=0), dict(h_kv=0), dict(n_seqs=0),
    dict(max_pages=0), dict(n_pages=0), dict(page_size=0), dict(page_size=-16), dict(k_scale=208), dict(v_scale=208),
    dict(flags=2), dict(flags=2, k_scale=208), dict(flags=2, k_scale=208, v_scale=2), dict(flags=4),
    dict(n_pages=1 << 27), dict(max_pages=1 << 27), dict(cos_sin=None), dict(eps=float("inf")),
])
def test_paged_append_invalid_arguments(L, bad):
    assert L.attn_paged_append(*dict(APPEND, **bad).values()) == attn.ATTN_ERR_INVALID


DECODE = dict(q=16, k_pages=32, v_pages=48, out=64, lse=None, page_table=80, cache_lens=96, B=3, n_q=2, h_q=4, h_kv=2,
              d=64, n_pages=9, page_size=16, max_pages=4, scale=0.125, window=-1, sinks=0, k_scale=None, v_scale=None,
              flags=0, ws=112, nbytes=1 << 30, stream=None)


@pytest.mark.parametrize("bad", [
    dict(q=None), dict(k_pages=None), dict(v_pages=None), dict(out=None), dict(page_table=None), dict(cache_lens=None),
    dict(ws=None), dict(q=8), dict(out=72), dict(ws=104), dict(lse=2), dict(cache_lens=2), dict(B=0), dict(n_q=0),
    dict(h_q=0), dict(h_q=5), dict(h_kv=0), dict(d=0), dict(n_pages=0), dict(page_size=0), dict(max_pages=0),
    dict(scale=float("nan")), dict(window=-2), dict(sinks=-1), dict(flags=1), dict(flags=2), dict(k_scale=128),
    dict(flags=2, k_scale=128), dict(nbytes=0), dict(max_pages=1 << 27), dict(n_pages=1 << 27),
])
def test_paged_decode_invalid_arguments(L, bad):
    assert L.attn_paged_decode(*dict(DECODE, **bad).values()) == attn.ATTN_ERR_INVALID


def test_paged_unsupported_shapes_and_workspace(L):
    for bad in (dict(n_q=17), dict(d=96), dict(d=256), dict(h_q=2 * 8193),
                dict(B=1 << 20, max_pages=1 << 26)):  # more tiles than 32 bits count
        assert L.attn_paged_decode(*dict(DECODE, **bad).values()) == attn.ATTN_ERR_UNSUPPORTED
    assert L.attn_paged_append(*dict(APPEND, d=96, q_stride=512, k_stride=512, v_stride=512).values()) == \
        attn.ATTN_ERR_UNSUPPORTED
    assert L.attn_paged_append(*dict(APPEND, d_rot=24).values()) == attn.ATTN_ERR_UNSUPPORTED
    size = attn.attn_paged_decode_workspace_size
    need = size(3, 2, 4, 2, 64)
    assert need > 0 and need == size(3000, 2, 4, 2, 64)
    assert L.attn_paged_decode(*dict(DECODE, nbytes=need - 1).values()) == attn.ATTN_ERR_INVALID
    assert size(0, 1, 1, 1, 64) == 0 and size(1, 17, 1, 1, 64) == 0 and size(1, 1, 3, 2, 64) == 0
    assert size(1, 1, 1, 1, 96) == 0 and size(1, 1, 8193, 1, 64) == 0
