"""The binding's argument handling for norm + rotation and the paged cache, as far as it goes
without a GPU."""
import pytest
import torch

from transformer_scaled_dot_mha_gb300 import attn


def zeros(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


def test_host_tensors_are_refused_as_values():
    """As by every other entry point: a ValueError, with or without a GPU in the machine."""
    i32 = torch.int32
    x, out, rows, pages = zeros(1, 2, 1, 64), zeros(1, 1, 2, 64), zeros(2, 1, 64), zeros(1, 1, 16, 64)
    calls = [
        lambda: attn.attn_norm_rope(x, x, out, out, None),
        lambda: attn.attn_norm_rope_bwd(x, x, out, out, x, x, None, None),
        lambda: attn.attn_paged_append(rows, rows, pages, pages, zeros(2, dtype=i32), zeros(2, 1, dtype=i32)),
        lambda: attn.attn_paged_decode(x, pages, pages, x, zeros(1, 1, dtype=i32), zeros(1, dtype=i32), x),
    ]
    for call in calls:
        with pytest.raises(ValueError, match="CUDA"):
            call()
