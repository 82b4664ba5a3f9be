"""The bounded-wait abort path of attn_paged_chunk, taken with copies in flight.

A warp that gives up raises its CTA's abort flag; every role then stops, the copies in flight land before the CTA
returns, and nothing more is written. Here the copying warps of V give up by themselves before a given tile (the
library's test-only instantiation), while those of K, and their own boxes of the tiles before, are under way.
"""
import pytest
import torch

from test_chunk_gpu import make, run, same
from transformer_scaled_dot_mha_gb300 import attn

pytestmark = pytest.mark.gpu

FAULT_PACKED = 512


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    attn.lib()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("page", [4, 16, 64])
def test_gives_up_with_copies_in_flight(d, e4m3, page):
    """320 units of 19 or 20 tiles, none of which is cut, for 152 CTAs: all of them give up in their first unit."""
    new, lens = [1] * 40, [2400 + 4 * i for i in range(40)]
    q, q_at, kp, vp, table, ln, sc = case = make(43, new, lens, 16, 8, d, page, e4m3, back=0)
    want = run(*case)
    at = torch.tensor(q_at, dtype=torch.int32, device="cuda")
    ws = torch.empty(attn.attn_paged_chunk_workspace_size(40, 40, 16, 8, d), dtype=torch.uint8, device="cuda")
    for tile in (0, 1, 2, 3, 4, 5, 9, 17):
        out, lse = torch.full_like(q, 7.0), torch.full((40, 16), 7.0, device="cuda")
        call = lambda: attn.attn_paged_chunk(q, kp, vp, out, at, table, ln, ws, lse=lse, k_scale=sc[0], v_scale=sc[1])  # noqa: E731
        attn._internal_arm_chunk_give_up(tile)
        call()
        assert attn.attn_fault_status() == (attn.ATTN_ERR_TIMEOUT, FAULT_PACKED)
        assert torch.all(out == 7.0) and torch.all(lse == 7.0)
        call()  # the next one, on the same workspace, is an ordinary one
        assert attn.attn_fault_status() == (attn.ATTN_OK, 0)
        assert same(out, want[0]) and same(lse, want[1])


@pytest.mark.parametrize("e4m3", [False, True])
def test_gives_up_among_pieces(e4m3):
    """A unit that is cut, given up in its pieces: reported, and the next call is right."""
    q, q_at, kp, vp, table, ln, sc = case = make(44, [3, 200], [30001, 700], 4, 2, 128, 16, e4m3, back=0)
    want = run(*case)
    attn._internal_arm_chunk_give_up(1)
    out, lse = torch.empty_like(q), torch.empty(203, 4, device="cuda")
    at = torch.tensor(q_at, dtype=torch.int32, device="cuda")
    ws = torch.empty(attn.attn_paged_chunk_workspace_size(203, 2, 4, 2, 128), dtype=torch.uint8, device="cuda")
    attn.attn_paged_chunk(q, kp, vp, out, at, table, ln, ws, lse=lse, k_scale=sc[0], v_scale=sc[1])
    assert attn.attn_fault_status() == (attn.ATTN_ERR_TIMEOUT, FAULT_PACKED)
    got = run(*case)
    assert same(got[0], want[0]) and same(got[1], want[1])
