"""attn_paged_chunk where a CTA works through units with keys and units without any, in turn: new tokens whose
sequence has no cached keys (padding, or more new tokens than cached ones) between others."""
import pytest
import torch

from test_chunk_gpu import make, run, same, verify
from test_packed_gpu import starts
from transformer_scaled_dot_mha_gb300 import attn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    attn.lib()


def long_caches(seed, new, lens, h_q, h_kv, d, page, e4m3):
    """As make, for lengths whose pages would be gigabytes: a pool of few pages that the table names again and again."""
    q, q_at, kp, vp, _, _, sc = make(seed, new, [40 * page] * len(new), h_q, h_kv, d, page, e4m3, back=3)
    g = torch.Generator().manual_seed(seed)
    pool = kp.shape[0] - 2  # the others hold poison
    good = torch.isfinite(kp.float()).flatten(1).all(1).nonzero()[:, 0].cpu()
    assert len(good) == pool
    table = good[torch.randint(0, pool, (len(new), -(-max(lens) // page)), generator=g)].to(torch.int32).cuda()
    return q, q_at, kp, vp, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), sc


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("page", [4, 16, 64, 128])
def test_no_keys_between_pieces(d, e4m3, page):
    """The cut list: 7813 tiles for each of two heads, then units without keys, then 235 tiles for each head, in shares of
    106 tiles. One CTA has the last 44 tiles of the first sequence, the empty units and the first 60 tiles of the last."""
    for new in ([1, 1, 1], [1, 70, 1], [1, 200, 2]):
        verify(*long_caches(41, new, [1000003, 0, 30000], 4, 2, d, page, e4m3))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("page", [1, 4, 16, 64, 128])
@pytest.mark.parametrize("most", [1, 20])
def test_no_keys_between_short_sequences(d, e4m3, page, most):
    """Whole units, dealt as CTAs ask: those of one tile and those of none cost the same and come in any order."""
    g = torch.Generator().manual_seed(page)
    new = torch.randint(1, most + 1, (100,), generator=g).tolist()
    lens = torch.randint(1, 129, (100,), generator=g).tolist()
    lens[::5] = [0] * 20
    lens[3::7] = [min(x, n) for x, n in zip(lens[3::7], range(14))]  # fewer cached tokens than new ones
    q, q_at, kp, vp, table, ln, sc = case = make(42, new, lens, 8, 8, d, page, e4m3)
    verify(*case)
    want = run(*case)
    out, lse, at = want[0].clone(), want[1].clone(), torch.tensor(starts(new), dtype=torch.int32, device="cuda")
    ws = torch.empty(attn.attn_paged_chunk_workspace_size(q.shape[0], 100, 8, 8, d), dtype=torch.uint8, device="cuda")
    for _ in range(20):
        out.fill_(7.0)
        attn.attn_paged_chunk(q, kp, vp, out, at, table, ln, ws, lse=lse, k_scale=sc[0], v_scale=sc[1])
        assert same(out, want[0]) and same(lse, want[1])
    assert attn.attn_fault_status() == (attn.ATTN_OK, 0)
