"""What rows of other sequences hold does not reach a sequence, one kind of poison at a time, forward and backward; and
offsets that decrease without naming a row twice."""
import math

import pytest
import torch

import packed_reference as ref
from test_packed_bwd_gpu import backward
from test_packed_gpu import INF, NAN, make, run
from transformer_scaled_dot_mha_gb300 import attn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    attn.lib()


LENS = [70, 30, 129, 5, 200, 60]
POISONED, CLEAN = (1, 3), (0, 2, 4, 5)


def rows(at, b):
    return slice(at[b], at[b + 1])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal,window", [(True, -1), (False, -1), (True, 20), (False, 64)])
@pytest.mark.parametrize("bad", [NAN, INF, -INF])
def test_forward(d, causal, window, bad):
    q, k, v, at, _ = make(12, LENS, None, 4, 2, d)
    want, want_lse = run(q, k, v, at, at, causal, window)
    for x in (q, k, v):
        kept = x.clone()
        for b in POISONED:
            x[rows(at, b)] = bad
        got, lse = run(q, k, v, at, at, causal, window)
        for b in CLEAN:
            assert torch.equal(got[rows(at, b)], want[rows(at, b)]) and torch.equal(lse[rows(at, b)], want_lse[rows(at, b)])
        x.copy_(kept)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal,window", [(True, -1), (False, -1), (True, 20), (False, 64)])
@pytest.mark.parametrize("bad", [NAN, INF, -INF])
def test_backward(d, causal, window, bad):
    q, k, v, at, _ = make(12, LENS, None, 6, 2, d)
    out, lse = run(q, k, v, at, at, causal, window)
    dout = torch.randn(q.shape, generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    want = backward(q, k, v, out, lse, dout, at, at, causal, window)
    for x in (q, k, v, out, lse, dout):
        kept = x.clone()
        for b in POISONED:
            x[rows(at, b)] = bad
        got = backward(q, k, v, out, lse, dout, at, at, causal, window)
        for b in CLEAN:
            for y, w in zip(got, want):
                assert torch.equal(y[rows(at, b)], w[rows(at, b)])
        x.copy_(kept)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T", [300, 200])
def test_a_sequence_that_ends_before_it_starts(d, T):
    """Offsets 120, 60, T: the first sequence is empty, the second has rows 60 to T - 1. (T = 200: without a work list.)"""
    q, k, v, _, _ = make(13, [T], None, 2, 1, d)
    at = torch.tensor([120, 60, T], dtype=torch.int32, device="cuda")
    dout = torch.randn(q.shape, generator=torch.Generator().manual_seed(4)).bfloat16().cuda()
    out, lse = torch.full_like(q, 7.0), torch.full((T, 2), 7.0, device="cuda")
    grads = [torch.full_like(x, 7.0) for x in (q, k, v)]
    ws = torch.empty(max(attn.attn_packed_fwd_workspace_size(T, 2, 2, 1, d), attn.attn_packed_bwd_workspace_size(T, T, 2, 2, 1, d)),
                     dtype=torch.uint8, device="cuda")
    attn.attn_packed_fwd(q, k, v, out, at, ws, lse=lse, mask_mode=attn.MASK_CAUSAL)
    attn.attn_packed_bwd(q, k, v, out, dout, lse, *grads, at, ws, mask_mode=attn.MASK_CAUSAL)
    torch.cuda.synchronize()
    assert attn.attn_fault_status() == (attn.ATTN_OK, 0)
    meant = [60, 60, T]
    ref.check(out, lse, *ref.packed(q, k, v, meant, meant, 1 / math.sqrt(d), True))
    ref.check_grads(grads, *ref.packed_bwd(q, k, v, out, lse, dout, meant, meant, 1 / math.sqrt(d), True))
    for x in (out, lse, *grads):
        assert torch.all(x[:60] == 7.0)
