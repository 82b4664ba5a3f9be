"""attn_packed_fwd against the plain float64 form (packed_reference.py derives the tolerance)."""
import math

import pytest
import torch

import packed_reference as ref
from transformer_scaled_dot_mha_gb300 import attn

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    attn.lib()


def starts(lens, first=0):
    at = [first]
    for n in lens:
        at.append(at[-1] + n)
    return at


def place(x, layout):
    """x [T, heads, d] as a view of token-major ("fused", with other columns beside) or head-major rows."""
    T, h, d = x.shape
    if layout == "heads":
        y = torch.empty(h, T, d, dtype=x.dtype, device=x.device).transpose(0, 1)
    else:
        y = torch.full((T, h + 2, d), NAN, dtype=x.dtype, device=x.device)[:, 1:1 + h]
    return y.copy_(x)


def make(seed, q_lens, k_lens, h_q, h_kv, d, layout="heads", front=0, back=0):
    """q, k, v on the GPU and their offsets; rows of no sequence are NaN and infinities."""
    g = torch.Generator().manual_seed(seed)
    q_at, k_at = starts(q_lens, front), starts(q_lens if k_lens is None else k_lens, front)
    def rows(at, h, scale):
        x = scale * torch.randn(max(1, at[-1] + back), h, d, generator=g)
        x[:at[0]], x[at[-1]:] = NAN, INF
        return place(x.bfloat16().cuda(), layout)
    return rows(q_at, h_q, 1.5), rows(k_at, h_kv, 1.0), rows(k_at, h_kv, 1.0), q_at, k_at


def run(q, k, v, q_at, k_at, causal=False, window=-1, scale=None, same=False, fill=255, with_lse=True):
    T, h, d = q.shape
    out = place(torch.full((T, h, d), 7.0, dtype=torch.bfloat16, device="cuda"), "fused")
    lse = torch.full((T, h), 7.0, device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    size = attn.attn_packed_fwd_workspace_size(T, len(q_at) - 1, h, k.shape[1], d)
    ws = torch.full((size,), fill, dtype=torch.uint8, device="cuda")
    attn.attn_packed_fwd(q, k, v, out, i32(q_at), ws, k_starts=None if same else i32(k_at), lse=lse if with_lse else None,
                         scale=scale, mask_mode=attn.MASK_CAUSAL if causal else attn.MASK_NONE, window=window)
    torch.cuda.synchronize()
    assert attn.attn_fault_status() == (attn.ATTN_OK, 0)
    return out, lse


def verify(q, k, v, q_at, k_at, causal=False, window=-1, scale=None, **kw):
    got, lse = run(q, k, v, q_at, k_at, causal, window, scale, **kw)
    want = ref.packed(q, k, v, q_at, k_at, 1 / math.sqrt(q.shape[2]) if scale is None else scale, causal, window)
    ref.check(got, lse, *want)
    none = torch.ones(q.shape[0], dtype=torch.bool, device="cuda")
    none[q_at[0]:q_at[-1]] = False
    assert torch.all(got[none] == 7.0) and torch.all(lse[none] == 7.0)
    again, lse2 = run(q, k, v, q_at, k_at, causal, window, scale, **dict(kw, fill=0))
    assert torch.equal(got, again) and torch.equal(lse, lse2)
    return got, lse


CASES = [  # q_lens, k_lens, h_q, h_kv, d, causal, window
    ([1], None, 1, 1, 64, True, -1),
    ([1], None, 1, 1, 128, True, -1),
    ([0, 1, 127, 128, 129, 0, 3], None, 2, 2, 64, True, -1),
    ([0, 1, 127, 128, 129, 0, 3], None, 2, 2, 128, True, -1),
    ([0, 1, 127, 128, 129, 0, 3], None, 2, 2, 64, False, -1),
    ([255, 256, 257, 40], None, 4, 1, 128, True, -1),
    ([255, 256, 257, 40], None, 4, 1, 128, False, -1),
    ([300, 5, 77], None, 6, 2, 64, True, -1),           # three heads a group: 126 rows a tile
    ([300, 5, 77], None, 7, 1, 128, True, -1),
    ([33, 64, 9], None, 5, 1, 64, False, -1),
    ([40, 3], None, 128, 1, 64, True, -1),              # one token a tile
    ([40, 3], None, 100, 1, 128, True, -1),             # 28 rows unused
    ([700, 1200, 90], None, 8, 2, 128, True, -1),
    ([700, 1200, 90], None, 8, 2, 64, True, -1),
    ([5, 0, 200, 1], [100, 30, 0, 1500], 4, 4, 64, False, -1),
    ([5, 0, 200, 1], [100, 30, 0, 1500], 4, 2, 128, False, -1),
    ([50, 200, 1, 130], [100, 30, 5, 0], 4, 2, 64, True, -1),   # more queries than keys: rows with none
    ([50, 200, 1, 600], [100, 30, 5, 300], 4, 2, 128, True, -1),
    ([2, 9], [5000, 3000], 2, 2, 64, False, -1),        # few rows, long axis
    ([2, 9], [5000, 3000], 8, 1, 128, True, -1),
    ([900, 300], None, 2, 1, 64, True, 0),
    ([900, 300], None, 2, 1, 128, True, 1),
    ([900, 300], None, 2, 2, 64, True, 130),
    ([900, 300, 1], None, 4, 1, 128, True, 257),
    ([900, 300, 1], None, 1, 1, 64, False, 100),
    ([900, 300, 1], None, 1, 1, 128, False, 64),
    ([300, 1000], [900, 200], 2, 1, 128, False, 70),    # windows before the first key
    ([300, 1000], [900, 200], 2, 1, 64, False, 70),
    ([300, 10], None, 2, 2, 64, False, 2 ** 40),
]


@pytest.mark.parametrize("q_lens,k_lens,h_q,h_kv,d,causal,window", CASES)
@pytest.mark.parametrize("layout", ["fused", "heads"])
def test_packed(q_lens, k_lens, h_q, h_kv, d, causal, window, layout):
    q, k, v, q_at, k_at = make(5, q_lens, k_lens, h_q, h_kv, d, layout, front=3 if layout == "heads" else 0, back=130)
    verify(q, k, v, q_at, k_at, causal, window, same=k_lens is None)


@pytest.mark.parametrize("d", [64, 128])
def test_many_short_sequences(d):
    """More sequences than the planning CTA has threads, and units than CTAs: dealt whole."""
    g = torch.Generator().manual_seed(d)
    lens = torch.randint(0, 40, (1500,), generator=g).tolist()
    lens[700] = 900
    q, k, v, q_at, k_at = make(6, lens, None, 4, 2, d)
    verify(q, k, v, q_at, k_at, True)


def test_thousands_of_sequences():
    """More sequences than the planning CTA's shared memory has room for."""
    g = torch.Generator().manual_seed(8)
    lens = torch.randint(0, 4, (5000,), generator=g).tolist()
    q, k, v, q_at, k_at = make(7, lens, None, 1, 1, 64)
    verify(q, k, v, q_at, k_at, True)


@pytest.mark.parametrize("d", [64, 128])
def test_one_long_among_many(d):
    """One sequence longer than a CTA's share of a full batch: the list is cut in the midst of many units."""
    lens = [60] * 700 + [9000] + [1] * 3
    k_lens = [60] * 700 + [30000] + [1] * 3
    lens[700] = 40
    q, k, v, q_at, k_at = make(9, lens, k_lens, 2, 2, d)
    verify(q, k, v, q_at, k_at, True)


@pytest.mark.parametrize("d,h_q,h_kv", [(64, 2, 1), (128, 4, 2)])
@pytest.mark.parametrize("causal", [True, False])
def test_long_sequences(d, h_q, h_kv, causal):
    q, k, v, q_at, k_at = make(10, [4099, 1, 2500], None, h_q, h_kv, d)
    verify(q, k, v, q_at, k_at, causal)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("size", [30.0, 300.0])
def test_large_scores(d, size):
    """Scores of hundreds: reference maxima that grow late, weights that are almost one-hot."""
    q, k, v, q_at, k_at = make(11, [600, 129], None, 2, 1, d)
    k[q_at[0]:q_at[-1]] *= torch.linspace(0.1, 1, q_at[-1] - q_at[0], device="cuda").bfloat16()[:, None, None]
    verify(q, k, v, q_at, k_at, True, scale=size / d)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
def test_other_sequences_do_not_reach(d, causal):
    """Sequences full of infinities and NaN between others, whose tiles hold their rows."""
    lens = [70, 30, 129, 5, 200, 60]
    q, k, v, q_at, k_at = make(12, lens, None, 4, 2, d)
    want, want_lse = run(q, k, v, q_at, k_at, causal)
    for x, bad in ((q, NAN), (k, INF), (v, -INF), (v, NAN)):
        x[q_at[1]:q_at[2]] = bad
        x[q_at[3]:q_at[4]] = bad
    got, lse = run(q, k, v, q_at, k_at, causal)
    for b in (0, 2, 4, 5):
        r = slice(q_at[b], q_at[b + 1])
        assert torch.equal(got[r], want[r]) and torch.equal(lse[r], want_lse[r])
    assert torch.isnan(got[q_at[1]:q_at[2]]).all()


@pytest.mark.parametrize("d", [64, 128])
def test_offsets_outside_the_arrays(d):
    """Offsets before, behind and against the order: clamped, empty; what remains is right."""
    q, k, v, _, _ = make(13, [300], None, 2, 1, d)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    for given, meant in (([-50, 100, 2 ** 31 - 1], [0, 100, 300]), ([10, 10, 290], [10, 10, 290]), ([400, 500, 300], None),
                         ([120, 60, 300], [120, 120, 300])):
        out, lse = torch.full_like(q, 7.0), torch.full((300, 2), 7.0, device="cuda")
        ws = torch.empty(attn.attn_packed_fwd_workspace_size(300, 2, 2, 1, d), dtype=torch.uint8, device="cuda")
        attn.attn_packed_fwd(q, k, v, out, i32(given), ws, lse=lse, mask_mode=attn.MASK_CAUSAL)
        torch.cuda.synchronize()
        assert attn.attn_fault_status() == (attn.ATTN_OK, 0)
        if meant is None:
            assert torch.all(out == 7.0) and torch.all(lse == 7.0)
        elif given != [120, 60, 300]:  # there the second sequence starts at 60
            ref.check(out, lse, *ref.packed(q, k, v, meant, meant, 1 / math.sqrt(d), True))


@pytest.mark.parametrize("d,h_q,h_kv", [(64, 1, 1), (128, 2, 1), (64, 3, 3), (128, 100, 1)])
@pytest.mark.parametrize("causal", [True, False])
def test_small_batches_of_many_sequences(d, h_q, h_kv, causal):
    """Up to a unit for every CTA: each finds its own, over more than one warp's width of sequences."""
    for lens in ([i % 3 for i in range(100)], [0] * 70 + [5, 0, 140], [0, 0, 0]):
        if sum(lens):
            verify(*make(22, lens, None, h_q, h_kv, d, back=3), causal)
        else:
            q, k, v, q_at, k_at = make(22, lens, None, h_q, h_kv, d, back=3)
            out, lse = run(q, k, v, q_at, k_at, causal)
            assert torch.all(out == 7.0) and torch.all(lse == 7.0)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T", [300, 40])
def test_offsets_that_name_rows_again(d, T):
    """Offsets that go back and forth would make more units than the work list has places for: nothing is written
    outside the workspace or the rows, forward and backward."""
    q, k, v, _, _ = make(21, [T], None, 2, 1, d)
    at = torch.tensor([0, T] * (200 if T == 300 else 50), dtype=torch.int32, device="cuda")
    n = at.shape[0] - 1
    dev = dict(dtype=torch.bfloat16, device="cuda")
    out, lse = torch.full((T + 2, 2, d), 7.0, **dev), torch.zeros(T, 2, device="cuda")
    grads = [torch.full((T + 2, h, d), 7.0, **dev) for h in (2, 1, 1)]

    def workspace(size):
        ws = torch.full((size + 512,), 91, dtype=torch.uint8, device="cuda")
        return ws, ws[:size]

    (w0, ws), (w1, ws_bwd) = (workspace(f) for f in (attn.attn_packed_fwd_workspace_size(T, n, 2, 1, d),
                                                     attn.attn_packed_bwd_workspace_size(T, T, n, 2, 1, d)))
    attn.attn_packed_fwd(q, k, v, out[:T], at, ws, lse=lse, mask_mode=attn.MASK_CAUSAL)
    attn.attn_packed_bwd(q, k, v, out[:T], q, lse, *(x[:T] for x in grads), at, ws_bwd, mask_mode=attn.MASK_CAUSAL)
    torch.cuda.synchronize()
    assert attn.attn_fault_status() == (attn.ATTN_OK, 0)
    assert torch.all(w0[-512:] == 91) and torch.all(w1[-512:] == 91)
    for x in (out, *grads):
        assert torch.all(x[T:] == 7.0)


def test_without_lse_and_on_another_stream():
    q, k, v, q_at, k_at = make(14, [500, 3, 800], None, 4, 2, 128)
    want, _ = run(q, k, v, q_at, k_at, True)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        got, lse = run(q, k, v, q_at, k_at, True, with_lse=False)
    stream.synchronize()
    assert torch.equal(got, want) and torch.all(lse == 7.0)


def test_two_graphs_share_a_workspace_and_lengths_change():
    """Captured calls follow the offsets that their memory holds when they are replayed."""
    cases = [make(15 + i, lens, None, 4, 2, 64, back=1400 - sum(lens)) for i, lens in
             enumerate(([700, 200], [100, 1300]))]
    ws = torch.empty(attn.attn_packed_fwd_workspace_size(1400, 2, 4, 2, 64), dtype=torch.uint8, device="cuda")
    at = torch.tensor(cases[0][3], dtype=torch.int32, device="cuda")
    outs = [torch.zeros(1400, 4, 64, dtype=torch.bfloat16, device="cuda") for _ in cases]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graphs = []
    for (q, k, v, _, _), out in zip(cases, outs):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=stream):
            attn.attn_packed_fwd(q, k, v, out, at, ws, mask_mode=attn.MASK_CAUSAL)
    for lens in ([700, 200], [1, 899], [0, 900]):
        q_at = starts(lens)
        at.copy_(torch.tensor(q_at, dtype=torch.int32))
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            for _ in range(3):
                for g in graphs:
                    g.replay()
        stream.synchronize()
        for (q, k, v, _, _), out in zip(cases, outs):
            if not torch.isfinite(q[:900]).all():
                continue
            want, _ = run(q, k, v, q_at, q_at, True)
            assert torch.equal(out[:900], want[:900])


@pytest.mark.parametrize("d", [64, 128])
def test_calls_in_a_row_over_more_than_the_l2(d):
    """Hundreds of calls that nothing waits between, over inputs that the L2 cannot hold: short row tiles
    and long key lists, whose copies come late. (Once a wait for a tile passed early here.)"""
    g = torch.Generator().manual_seed(19)
    h, i32 = 16, lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    q_lens = [1 + 257 * i // 47 for i in range(48)]
    k_lens = [[33 + 988 * int(i) // 47 for i in torch.randperm(48, generator=g)] for _ in range(3)]
    T_q, T_k = sum(q_lens), sum(k_lens[0])
    states = []
    for k_len in k_lens:
        q, k, v = (torch.randn(h, n, d, device="cuda").bfloat16().transpose(0, 1) for n in (T_q, T_k, T_k))
        ws = torch.empty(attn.attn_packed_fwd_workspace_size(T_q, 48, h, h, d), dtype=torch.uint8, device="cuda")
        states.append((q, k, v, torch.empty(T_q, h, d, dtype=torch.bfloat16, device="cuda"), i32(starts(q_lens)), ws,
                       i32(starts(k_len))))
    want = []
    for s in states:
        attn.attn_packed_fwd(*s[:6], k_starts=s[6])
        torch.cuda.synchronize()
        want.append(s[3].clone())
    for s, w, k_len in zip(states, want, k_lens):
        at, ka = starts(q_lens), starts(k_len)
        out, _, qb, _ = ref.packed(*s[:3], at, ka, 1 / math.sqrt(d), False)
        assert torch.all((w.double() - out).abs() <= 6 * qb)
    for i in range(600):
        s = states[i % 3]
        attn.attn_packed_fwd(*s[:6], k_starts=s[6])
    torch.cuda.synchronize()
    assert attn.attn_fault_status() == (attn.ATTN_OK, 0)
    for s, w in zip(states, want):
        assert torch.equal(s[3], w)
