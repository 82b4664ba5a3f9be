"""Strides whose products with the tokens or heads leave 64 bits are refused, not wrapped, without a GPU."""
import pytest

from test_packed_abi_cpu import BWD, L, PACKED, bwd  # noqa: F401
from transformer_scaled_dot_mha_gb300 import attn

TOKENS = (1 << 26) + 1  # times 2^38: 2^64 and the rest


@pytest.mark.parametrize("bad", [
    dict(q_stride=1 << 38, T_q=TOKENS, h_q=1, h_kv=1), dict(out_stride=1 << 38, T_q=TOKENS, h_q=1, h_kv=1),
    dict(k_stride=1 << 38, T_k=TOKENS, h_q=1, h_kv=1), dict(v_stride=1 << 38, T_k=TOKENS, h_kv=1),
    dict(q_head=1 << 38, k_head=1 << 38, v_head=1 << 38, out_head=1 << 38, T_q=1, T_k=1, h_q=TOKENS, h_kv=TOKENS),
])
def test_packed_fwd(L, bad):  # noqa: F811
    assert L.attn_packed_fwd(*dict(PACKED, nbytes=1 << 60, **bad).values()) == attn.ATTN_ERR_INVALID


@pytest.mark.parametrize("operand", range(8))
def test_packed_bwd(L, operand):  # noqa: F811
    strides = [64, 64] * operand + [1 << 38, 64] + [64, 64] * (7 - operand)
    assert bwd(L, strides=strides, h_q=1, h_kv=1, T_q=TOKENS, T_k=TOKENS, nbytes=1 << 60) == attn.ATTN_ERR_INVALID
