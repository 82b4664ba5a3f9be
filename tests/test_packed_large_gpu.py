"""Packed arrays of more than 2^31 numbers: sequences at their end get the bits that small arrays of the same rows give."""
import pytest
import torch

from transformer_scaled_dot_mha_gb300 import attn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    attn.lib()


def call(arrays, lse, at, causal):
    q, k, v, out, dout, dq, dk, dv = arrays
    (T_q, h_q, d), (T_k, h_kv, _), n = q.shape, k.shape, at.shape[0] - 1
    size = max(attn.attn_packed_fwd_workspace_size(T_q, n, h_q, h_kv, d), attn.attn_packed_bwd_workspace_size(T_q, T_k, n, h_q, h_kv, d))
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    mask = attn.MASK_CAUSAL if causal else attn.MASK_NONE
    attn.attn_packed_fwd(q, k, v, out, at, ws, lse=lse, mask_mode=mask)
    attn.attn_packed_bwd(q, k, v, out, dout, lse, dq, dk, dv, at, ws, mask_mode=mask)
    torch.cuda.synchronize()
    assert attn.attn_fault_status() == (attn.ATTN_OK, 0)


@pytest.mark.parametrize("d,T", [(64, 280000), (128, 140000)])
@pytest.mark.parametrize("h_kv", [128, 16])
@pytest.mark.parametrize("layout", ["tokens", "heads"])
def test_rows_beyond_32_bits(d, T, h_kv, layout):
    h_q, first, n = 128, T - 701, 701
    dev = dict(dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(d)
    at = torch.tensor([0, 300, 301, n], dtype=torch.int32, device="cuda")
    heads = (h_q, h_kv, h_kv, h_q, h_q, h_q, h_kv, h_kv)
    small = [torch.randn(n, h, d, generator=g, device="cuda").bfloat16() for h in heads]
    small_lse = torch.empty(n, h_q, device="cuda")
    call(small, small_lse, at, True)
    large = []
    for x, h in zip(small, heads):
        y = torch.empty(T, h, d, **dev) if layout == "tokens" else torch.empty(h, T, d, **dev).transpose(0, 1)
        y[first:] = x
        y[first - 1] = 7.0
        large.append(y)
    lse = torch.empty(T, h_q, device="cuda")
    call(large, lse, at + first, True)
    assert torch.equal(lse[first:], small_lse)
    for i in (3, 5, 6, 7):
        assert torch.equal(large[i][first:], small[i]) and torch.all(large[i][first - 1] == 7.0)
