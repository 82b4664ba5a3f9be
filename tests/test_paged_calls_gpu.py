"""Calls of attn_paged_decode that its documentation allows and its other tests do not make."""
import math

import pytest
import torch

import paged_reference as ref
from test_paged_gpu import check, make, run
from transformer_scaled_dot_mha_gb300 import attn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    attn.lib()


@pytest.mark.parametrize("window,sinks", [(2 ** 32 + 1, 0), (2 ** 31, 0), (2 ** 63 - 1, 2 ** 32), (2, 2 ** 32 + 1)])
def test_windows_and_sinks_beyond_32_bits(window, sinks):
    """A window or a number of first tokens that no int holds reaches every key, as the widest does."""
    q, kp, vp, table, ln, sc = make(91, [90, 3], 1, 4, 2, 64, 16)
    got = run(q, kp, vp, table, ln, sc, None, window, sinks)
    check(*got, *ref.paged_decode(q, kp, vp, table, ln, 0.125, window, sinks))


@pytest.mark.parametrize("B,h_q,h_kv,d,capacity,longest,n_q,e4m3", [
    (342, 8, 8, 64, 1024, 1000, 1, False),   # 1.5 pairs per resident warp, 32 tiles: not split
    (115, 8, 8, 64, 768, 700, 2, False),     # half a pair per warp, 24 tiles
    (70, 16, 16, 128, 384, 380, 1, False),
    (60, 64, 16, 128, 768, 500, 3, True),    # 12 rows of a pair, 24 tiles of 8-bit keys
    (40, 8, 8, 128, 4096, 40, 1, False),     # short sequences under a large capacity: split
])
def test_batches_around_the_rules_for_unsplit_pairs(B, h_q, h_kv, d, capacity, longest, n_q, e4m3):
    """The capacity (the page table's width), the number of pairs and the row count choose between
    a warp per pair and the list of parts: ragged, with empty sequences, on both sides."""
    g = torch.Generator().manual_seed(B)
    lens = torch.randint(1, longest, (B,), generator=g).tolist()
    lens[0], lens[B // 3], lens[B - 1], lens[5] = 0, 0, 0, longest
    q, kp, vp, table, ln, sc = make(B, lens, n_q, h_q, h_kv, d, 64, e4m3, max_pages=capacity // 64)
    assert table.shape[1] == capacity // 64
    check(*run(q, kp, vp, table, ln, sc), *ref.paged_decode(q, kp, vp, table, ln, 1 / math.sqrt(d), -1, 0, *sc))


@pytest.mark.parametrize("e4m3", [False, True])
def test_millions_of_keys(e4m3):
    """2^24 + 3 keys of one sequence in a table of 2^26 pages of 16: all entries name one of three
    pages, so that key j's weight is known. Sums of 2^24 weights in fp32, cut into parts of at most
    2^14 keys: at most 2^12 additions one after the other, 2^-11 of the terms' sizes even if
    every one loses an eighth of a unit (2^-23 each); the output's rounding is 2^-8 of it."""
    q, kp, vp, _, _, sc = make(92, [48], 1, 2, 1, 64, 16, e4m3)
    n = 2 ** 24 + 3
    table = torch.arange(2 ** 26, dtype=torch.int32, device="cuda").remainder_(3)[None]
    kp, vp = (x[:3].float().nan_to_num(0.5).to(x.dtype) for x in (kp, vp))  # unused rows hold NaN
    out, lse = run(q, kp, vp, table, torch.tensor([n], dtype=torch.int32), sc)
    k, v = (x.float().double().transpose(1, 2).reshape(48, 64) for x in (kp, vp))
    if e4m3:
        k, v = k * sc[0].double(), v * sc[1].double()
    count = torch.tensor([n // 48 + (j < n % 48) for j in range(48)]).double()
    for h in range(2):
        s = 0.125 * (k @ q[0, 0, h].double())
        w = count * torch.exp(s - s.max())
        want = (w @ v) / w.sum()
        size = (w @ v.abs()) / w.sum()
        assert torch.all((out[0, 0, h].double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -10 * size)
        assert abs(lse[0, 0, h] - (s.max() + w.sum().log())) <= 2.0 ** -10


def test_two_graphs_share_a_workspace():
    """Captured calls that replay one after the other may use one workspace."""
    cases = [make(93 + i, [900, 40 + i, 1400], 1, 8, 2, 64, 16) for i in range(2)]
    want = [run(*c)[0] for c in cases]
    held = [[x.cuda() if torch.is_tensor(x) else x for x in c] for c in cases]
    outs = [torch.empty_like(c[0]) for c in held]
    ws = torch.empty(attn.attn_paged_decode_workspace_size(3, 1, 8, 2, 64), dtype=torch.uint8, device="cuda")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graphs = []
    for (q, kp, vp, table, ln, _), out in zip(held, outs):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=stream):
            attn.attn_paged_decode(q, kp, vp, out, table, ln, ws)
    with torch.cuda.stream(stream):
        for _ in range(10):
            for out in outs:
                out.fill_(7.0)
            for g in graphs:
                g.replay()
    stream.synchronize()
    for out, w in zip(outs, want):
        assert torch.equal(out.cpu(), w)
