"""attn_paged_chunk against the plain float64 form (packed_reference.py derives the tolerance), and with
the operators before and after it."""
import math

import pytest
import torch

import packed_reference as ref
from test_packed_gpu import starts
from test_paged_gpu import make as make_cache
from transformer_scaled_dot_mha_gb300 import attn

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    attn.lib()


def make(seed, new, lens, h_q, h_kv, d, page, e4m3=False, max_pages=0, back=40):
    """Everything on the GPU; rows behind the lengths, unused pages and table entries are poison."""
    _, kp, vp, table, ln, sc = make_cache(seed, lens, 1, h_q, h_kv, d, page, e4m3, max_pages)
    q_at = starts(new)
    g = torch.Generator().manual_seed(seed + 1)
    q = 1.5 * torch.randn(q_at[-1] + back, h_q, d, generator=g)
    q[q_at[-1]:] = NAN
    dev = lambda x: None if x is None else x.cuda()  # noqa: E731
    return dev(q.bfloat16()), q_at, dev(kp), dev(vp), dev(table), dev(ln), [dev(x) for x in sc]


def run(q, q_at, kp, vp, table, ln, sc, window=-1, sinks=0, scale=None, fill=255):
    T, h, d = q.shape
    out, lse = torch.full_like(q, 7.0), torch.full((T, h), 7.0, device="cuda")
    size = attn.attn_paged_chunk_workspace_size(T, len(q_at) - 1, h, kp.shape[1], d)
    ws = torch.full((size,), fill, dtype=torch.uint8, device="cuda")
    attn.attn_paged_chunk(q, kp, vp, out, torch.tensor(q_at, dtype=torch.int32, device="cuda"), table, ln, ws, lse=lse,
                          scale=scale, window=window, sinks=sinks, k_scale=sc[0], v_scale=sc[1])
    torch.cuda.synchronize()
    assert attn.attn_fault_status() == (attn.ATTN_OK, 0)
    return out, lse


def verify(q, q_at, kp, vp, table, ln, sc, window=-1, sinks=0):
    got, lse = run(q, q_at, kp, vp, table, ln, sc, window, sinks)
    ref.check(got, lse, *ref.chunk(q, q_at, kp, vp, table, ln, 1 / math.sqrt(q.shape[2]), window, sinks, *sc))
    assert torch.all(got[q_at[-1]:] == 7.0) and torch.all(lse[q_at[-1]:] == 7.0)
    again = run(q, q_at, kp, vp, table, ln, sc, window, sinks, fill=0)
    assert same(got, again[0]) and same(lse, again[1])


def same(x, y):  # bits: NaN stays NaN
    as_int = torch.int16 if x.dtype == torch.bfloat16 else torch.int32
    return torch.equal(x.contiguous().view(as_int), y.contiguous().view(as_int))


CASES = [  # new tokens, lengths, h_q, h_kv, d, page, window, sinks, max_pages
    ([1], [1], 1, 1, 64, 16, -1, 0, 0),
    ([17], [17], 8, 8, 64, 16, -1, 0, 0),
    ([1, 0, 5, 130, 0], [1, 40, 5, 200, 0], 8, 2, 128, 64, -1, 0, 0),
    ([1, 1, 1, 1], [127, 128, 129, 900], 8, 2, 128, 64, -1, 0, 0),
    ([100, 3, 257], [100, 50, 300], 7, 7, 64, 20, -1, 0, 0),
    ([100, 3, 257], [150, 3, 257], 6, 3, 128, 1, -1, 0, 0),
    ([100, 3], [150, 3], 6, 3, 64, 1, -1, 0, 0),
    ([60, 30], [360, 130], 5, 1, 64, 8, -1, 0, 0),
    ([60, 30], [360, 130], 14, 2, 128, 2, -1, 0, 0),
    ([200, 1, 64], [1300, 800, 64], 16, 2, 128, 256, -1, 0, 9),
    ([200, 1, 64], [1300, 800, 64], 4, 2, 64, 48, -1, 0, 0),
    ([5, 20], [3, 0], 4, 2, 64, 16, -1, 0, 0),                  # more new tokens than cached ones
    ([5, 300], [3, 140], 4, 2, 128, 16, -1, 0, 0),
    ([16, 1], [60001, 900], 8, 1, 128, 64, -1, 0, 0),           # few rows, a long axis
    ([3, 1], [40003, 20000], 2, 2, 64, 128, -1, 0, 0),
    ([200, 300], [1000, 300], 4, 2, 64, 16, 0, 0, 0),
    ([200, 300], [1000, 300], 4, 2, 64, 16, 100, 4, 0),
    ([200, 300, 1], [1500, 300, 999], 8, 2, 128, 32, 130, 200, 0),
    ([200, 300, 1], [1500, 300, 999], 2, 1, 128, 64, 600, 1, 0),
    ([40], [700], 4, 4, 64, 16, 50, 1000, 0),                   # more first tokens than keys
    ([40, 7], [700, 9], 128, 1, 64, 16, 33, 2, 0),
]


@pytest.mark.parametrize("new,lens,h_q,h_kv,d,page,window,sinks,max_pages", CASES)
@pytest.mark.parametrize("e4m3", [False, True])
def test_chunk(new, lens, h_q, h_kv, d, page, window, sinks, max_pages, e4m3):
    verify(*make(31, new, lens, h_q, h_kv, d, page, e4m3, max_pages), window, sinks)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("page", [4, 16, 256])
def test_entries_that_name_no_page(d, e4m3, page):
    """Keys of bad page table entries are illegal, in some rows all of them."""
    q, q_at, kp, vp, table, ln, sc = make(32, [300, 40, 5], [700, 300, 20], 4, 2, d, page, e4m3)
    table[0, 1::3] = -7
    table[0, 0] = kp.shape[0]
    table[1] = 1 << 29
    table[0, 2:3] = -2 ** 31  # the lowest number, like any other
    verify(q, q_at, kp, vp, table, ln, sc)
    verify(q, q_at, kp, vp, table, ln, sc, window=90, sinks=5)


@pytest.mark.parametrize("d", [64, 128])
def test_every_number_of_8_bits(d):
    """All 254 finite e4m3 numbers, subnormal ones among them, as keys and values, with equal weights."""
    codes = torch.arange(256, dtype=torch.uint8)
    codes = codes[(codes & 0x7f) != 0x7f]
    n = 300
    x = codes[torch.arange(n * d) % len(codes)].view(torch.float8_e4m3fn).view(1, 1, n, d)
    page = torch.zeros(1, 1, 300, d, dtype=torch.float8_e4m3fn)
    page.view(torch.uint8)[:] = x.view(torch.uint8)
    page = page.cuda()
    sc = [torch.tensor([2.0 ** -9], device="cuda"), torch.tensor([1.0], device="cuda")]
    q = torch.zeros(300, 1, d, dtype=torch.bfloat16, device="cuda")
    table, ln = torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.tensor([n], dtype=torch.int32, device="cuda")
    verify(q, [0, n], page, page, table, ln, sc)           # equal weights: running means of the values
    verify(q, [0, n], page, page, table, ln, sc, window=0)  # only the own key: its value, exactly
    got, _ = run(q, [0, n], page, page, table, ln, sc, window=0)
    assert torch.equal(got[:, 0].float(), page[0, 0].float())


def test_8_bit_nan_stays():
    """A NaN in the cache reaches the rows that see it, not other sequences'."""
    q, q_at, kp, vp, table, ln, sc = make(33, [20, 20], [150, 150], 2, 1, 64, 16, True)
    vp.view(torch.uint8)[int(table[0, 0]), 0, 3, 7] = 0x7f
    kp.view(torch.uint8)[int(table[0, 2]), 0, 3, 7] = 0xff
    got, lse = run(q, q_at, kp, vp, table, ln, sc)
    assert torch.isnan(got[:20]).any(-1).all() and torch.isnan(lse[:20]).all()
    assert torch.isfinite(got[20:40]).all()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("page", [4, 16, 64])
def test_pages_beyond_32_bits(e4m3, page):
    """A pool of more than 2^32 bytes whose last pages are in use: the bits of a small pool with the same pages."""
    q, q_at, kp, vp, table, ln, sc = make(35, [70, 3], [500, 130], 4, 2, 128, page, e4m3)
    per_page = kp[0].numel() * kp.element_size()
    n = (1 << 32) // per_page + 2 * kp.shape[0]
    want = run(q, q_at, kp, vp, table, ln, sc)
    big = []
    for x in (kp, vp):
        pool = torch.empty(n, *x.shape[1:], dtype=x.dtype, device="cuda")
        pool.view(torch.uint8)[n - x.shape[0]:] = x.view(torch.uint8)
        big.append(pool)
    got = run(q, q_at, *big, table + (n - kp.shape[0]), ln, sc)
    for x, y in zip(want, got):
        assert same(x[:73], y[:73])


@pytest.mark.parametrize("e4m3", [False, True])
def test_captured_calls_follow_the_lengths(e4m3):
    """Two graphs on one workspace, replayed with other lengths and offsets than at capture."""
    cases = [make(36 + i, [300, 20], [900, 700], 8, 2, 64, 16, e4m3, back=0) for i in range(2)]
    size = attn.attn_paged_chunk_workspace_size(320, 2, 8, 2, 64)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    at, ln = torch.tensor([0, 300, 320], dtype=torch.int32, device="cuda"), cases[0][5].clone()
    outs = [torch.zeros_like(c[0]) for c in cases]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graphs = []
    for (q, _, kp, vp, table, _, sc), out in zip(cases, outs):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=stream):
            attn.attn_paged_chunk(q, kp, vp, out, at, table, ln, ws, k_scale=sc[0], v_scale=sc[1])
    for new, lens in (([300, 20], [900, 700]), ([1, 319], [1, 640]), ([0, 1], [0, 77]), ([320, 0], [333, 5])):
        at.copy_(torch.tensor(starts(new), dtype=torch.int32))
        ln.copy_(torch.tensor(lens, dtype=torch.int32))
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            for g in graphs + graphs:
                g.replay()
        stream.synchronize()
        for (q, _, kp, vp, table, _, sc), out in zip(cases, outs):
            want, _ = run(q, starts(new), kp, vp, table, ln, sc)
            assert same(out[:sum(new)], want[:sum(new)])


def test_two_calls_at_once():
    """On two streams, each with a workspace of its own: the results of calls that run alone."""
    cases = [make(38 + i, [200, 1, 90], [900, 3000, 90], 8, 2, 128, 16, i == 1, back=0) for i in range(2)]
    want = [run(*c) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    at = torch.tensor(cases[0][1], dtype=torch.int32, device="cuda")
    state = []
    for q, *_ in cases:
        ws = torch.empty(attn.attn_paged_chunk_workspace_size(291, 3, 8, 2, 128), dtype=torch.uint8, device="cuda")
        state.append((torch.zeros_like(q), torch.zeros(291, 8, device="cuda"), ws))
    torch.cuda.synchronize()
    for _ in range(20):
        for stream, (q, _, kp, vp, table, ln, sc), (out, lse, ws) in zip(streams, cases, state):
            attn.attn_paged_chunk(q, kp, vp, out, at, table, ln, ws, lse=lse, k_scale=sc[0], v_scale=sc[1], stream=stream)
    torch.cuda.synchronize()
    for w, (out, lse, _) in zip(want, state):
        assert same(w[0], out) and same(w[1], lse)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("page", [4, 16])
def test_calls_in_a_row_over_more_than_the_l2(e4m3, page):
    """Hundreds of calls that nothing waits between, over caches that the L2 cannot hold."""
    new, lens = [65, 1, 1, 300, 1, 129], [9000, 20000, 41, 30000, 7777, 16000]
    q, q_at, kp, vp, table, ln, sc = make(40, new, lens, 16, 8, 128, page, e4m3, back=0)
    want = run(q, q_at, kp, vp, table, ln, sc)
    out, lse, at = torch.empty_like(want[0]), torch.empty_like(want[1]), torch.tensor(q_at, dtype=torch.int32, device="cuda")
    ws = torch.empty(attn.attn_paged_chunk_workspace_size(sum(new), 6, 16, 8, 128), dtype=torch.uint8, device="cuda")
    for _ in range(300):
        attn.attn_paged_chunk(q, kp, vp, out, at, table, ln, ws, lse=lse, k_scale=sc[0], v_scale=sc[1])
    torch.cuda.synchronize()
    assert attn.attn_fault_status() == (attn.ATTN_OK, 0)
    assert same(out, want[0]) and same(lse, want[1])


def test_as_one_decode_step():
    """One new token a sequence: what attn_paged_decode computes, up to both roundings."""
    q, q_at, kp, vp, table, ln, sc = make(34, [1] * 6, [1, 40, 300, 1025, 7, 2000], 8, 2, 128, 16, back=0)
    got, lse = run(q, q_at, kp, vp, table, ln, sc)
    out, lse2 = torch.empty_like(q).view(6, 1, 8, 128), torch.empty(6, 1, 8, device="cuda")
    ws = torch.empty(attn.attn_paged_decode_workspace_size(6, 1, 8, 2, 128), dtype=torch.uint8, device="cuda")
    attn.attn_paged_decode(q.view(6, 1, 8, 128), kp, vp, out, table, ln, ws, lse=lse2)
    want, want_lse, qb, lb = ref.chunk(q, q_at, kp, vp, table, ln, 1 / math.sqrt(128))
    assert torch.all((got.double() - out[:, 0].double()).abs() <= 12 * qb)
    assert torch.all((lse - lse2[:, 0]).abs() <= 2 * lb)


@pytest.mark.parametrize("e4m3", [False, True])
def test_prompt_in_pieces(e4m3):
    """Prompts appended and attended to in pieces of different sizes, then a decoding step: each row as
    attention over its whole prefix, with the cache's values."""
    h_q, h_kv, d, page, B = 8, 2, 64, 16, 3
    g = torch.Generator().manual_seed(35)
    pieces = [[50, 1, 0], [1, 200, 70], [130, 1, 1]]
    table = torch.randperm(60, generator=g)[:3 * 20].view(3, 20).to(torch.int32).cuda()
    kind = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    kp, vp = (torch.zeros(60, h_kv, page, d, device="cuda").to(kind) for _ in range(2))
    sc = [torch.full((h_kv,), 0.02, device="cuda") if e4m3 else None for _ in range(2)]
    lens = [0] * B
    for new in pieces:
        q_at = starts(new)
        T = q_at[-1] + 5  # a padded batch
        qkv = torch.randn(T, h_q + 2 * h_kv, d, generator=g).bfloat16().cuda()
        pos, seq = torch.full((T,), -1, dtype=torch.int32), torch.zeros(T, dtype=torch.int32)
        for b in range(B):
            pos[q_at[b]:q_at[b + 1]] = torch.arange(lens[b], lens[b] + new[b])
            seq[q_at[b]:q_at[b + 1]] = b
            lens[b] += new[b]
        q = torch.zeros(T, h_q, d, dtype=torch.bfloat16, device="cuda")
        attn.attn_paged_append(qkv[:, h_q:h_q + h_kv], qkv[:, h_q + h_kv:], kp, vp, pos.cuda(), table, seq_ids=seq.cuda(),
                               q=qkv[:, :h_q], q_out=q, k_scale=sc[0], v_scale=sc[1])
        verify(q, q_at, kp, vp, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), sc)
