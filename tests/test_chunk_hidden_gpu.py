"""attn_paged_chunk under a sliding window: pages of which no new token may see a row are not used. They may belong to
other sequences by now, and hold anything."""
import pytest
import torch

from test_chunk_gpu import INF, NAN, make, run, same, verify
from transformer_scaled_dot_mha_gb300 import attn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    attn.lib()


def hidden(new, lens, page, window, sinks):
    """(sequence, page) of every page whose rows are all before the windows and behind the first tokens."""
    return [(b, x) for b, (n, total) in enumerate(zip(new, lens)) for x in range(-(-sinks // page), (total - n - window) // page)]


CASES = [  # new tokens, lengths, window, sinks
    ([1, 1, 40, 300], [700, 129, 600, 1000], 0, 0),
    ([1, 3, 40, 300, 2], [700, 129, 500, 1000, 90], 37, 4),
    ([1, 3, 40, 300, 2], [701, 130, 501, 1003, 5000], 100, 130),
    ([1, 1, 5, 260], [257, 128, 385, 2000], 127, 1),
    ([2, 600], [640, 3000], 1000, 0),
]


@pytest.mark.parametrize("new,lens,window,sinks", CASES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("page", [1, 4, 8, 20, 64, 256])
def test_pages_that_no_token_may_see(new, lens, window, sinks, d, e4m3, page):
    q, q_at, kp, vp, table, ln, sc = make(45, new, lens, 4, 2, d, page, e4m3)
    kp, vp = (torch.cat([x, x[:3]]) for x in (kp, vp))  # three pages of another sequence
    case = q, q_at, kp, vp, table, ln, sc
    want = run(*case, window, sinks)
    for i, bad in enumerate((NAN, NAN, NAN) if e4m3 else (NAN, INF, -INF)):
        for x in (kp, vp):
            x[i - 3] = torch.full(x.shape[1:], bad).to(x.dtype)
    pages = hidden(new, lens, page, window, sinks)
    assert pages
    b, x = torch.tensor(pages, device="cuda").T
    table[b, x] = kp.shape[0] - 3 + torch.arange(len(pages), device="cuda", dtype=torch.int32) % 3
    got = run(*case, window, sinks)
    assert same(got[0], want[0]) and same(got[1], want[1])
    if not e4m3:  # (torch's cast to 8 bits makes NaN of what is too large, also in keys that some tokens see)
        assert torch.isfinite(got[0][:q_at[-1]]).all()
        verify(*case, window, sinks)
