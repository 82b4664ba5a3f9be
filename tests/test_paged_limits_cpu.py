"""Sizes at the limits of the norm + rotation, paged append and paged decode entry points:
refused or accepted as documented, without a GPU (the checks return before any CUDA call)."""
import pytest

from test_paged_abi_cpu import APPEND, ROPE, L  # noqa: F401 (a fixture)
from transformer_scaled_dot_mha_gb300 import attn

WIDE = 1 << 25  # heads of 64 columns: 2^31 elements, beyond a row's 32-bit column offsets


@pytest.mark.parametrize("heads", ["h_q", "h_kv"])
def test_rows_of_more_than_31_bits_are_refused(L, heads):  # noqa: F811
    stride = "q_stride" if heads == "h_q" else "k_stride"
    wide = {"B": 1, "n": 1, heads: WIDE, stride: WIDE * 64}
    assert L.attn_norm_rope(*dict(ROPE, **wide).values()) == attn.ATTN_ERR_INVALID
    assert attn.attn_norm_rope_bwd_workspace_size(1, 1, wide.get("h_q", 4), wide.get("h_kv", 4), 64) == 0
    assert attn.attn_norm_rope_bwd_workspace_size(1, 1, WIDE - 1, WIDE - 1, 64) > 0
    a = {x: ROPE[x] for x in list(ROPE)[:11]}
    a |= dict(dq_out=96, dk_out=112, dq=128, dk=144, dq_stride=WIDE * 64, dk_stride=WIDE * 64, dq_weight=160,
              dk_weight=176)
    a |= {x: ROPE[x] for x in ("B", "n", "h_q", "h_kv", "d", "flags")} | dict(ws=192, nbytes=1 << 30, stream=None)
    assert L.attn_norm_rope_bwd(*dict(a, **wide).values()) == attn.ATTN_ERR_INVALID
    wide = {"T": 1, heads: WIDE, "q_stride": WIDE * 64, "k_stride": WIDE * 64, "v_stride": WIDE * 64, "n_pages": 1,
            "page_size": 1}
    assert L.attn_paged_append(*dict(APPEND, **wide).values()) == attn.ATTN_ERR_INVALID
