"""attn_packed_bwd against the plain float64 form (packed_reference.py derives the tolerance), against
differences of the forward's formula, and as training uses it."""
import math

import pytest
import torch

import packed_reference as ref
from test_packed_gpu import CASES, make, place, run as forward, starts
from transformer_scaled_dot_mha_gb300 import attn

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    attn.lib()


def backward(q, k, v, out, lse, dout, q_at, k_at, causal, window, scale=None, same=False, fill=255, layout="heads"):
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    grads = [place(torch.full(x.shape, 7.0, dtype=torch.bfloat16, device="cuda"), layout) for x in (q, k, v)]
    (T_q, h_q, d), (T_k, h_kv, _) = q.shape, k.shape
    ws = torch.full((attn.attn_packed_bwd_workspace_size(T_q, T_k, len(q_at) - 1, h_q, h_kv, d),), fill, dtype=torch.uint8,
                    device="cuda")
    attn.attn_packed_bwd(q, k, v, out, dout, lse, *grads, i32(q_at), ws, k_starts=None if same else i32(k_at), scale=scale,
                         mask_mode=attn.MASK_CAUSAL if causal else attn.MASK_NONE, window=window)
    torch.cuda.synchronize()
    assert attn.attn_fault_status() == (attn.ATTN_OK, 0)
    return grads


def verify(q, k, v, q_at, k_at, causal=False, window=-1, scale=None, same=False, layout="heads"):
    out, lse = forward(q, k, v, q_at, k_at, causal, window, scale)
    none = torch.ones(q.shape[0], dtype=torch.bool, device="cuda")
    none[q_at[0]:q_at[-1]] = False
    out[none], lse[none] = NAN, NAN  # rows of no sequence are not used
    g = torch.Generator().manual_seed(77)
    dout = torch.randn(q.shape, generator=g).bfloat16().cuda()
    dout[none] = INF
    dout = place(dout, layout)
    got = backward(q, k, v, out, lse, dout, q_at, k_at, causal, window, scale, same, layout=layout)
    want, bounds = ref.packed_bwd(q, k, v, out, lse, dout, q_at, k_at, 1 / math.sqrt(q.shape[2]) if scale is None else scale,
                                  causal, window)
    ref.check_grads(got, want, bounds)
    for x, y in zip(got, backward(q, k, v, out, lse, dout, q_at, k_at, causal, window, scale, same, fill=0, layout=layout)):
        assert torch.equal(x, y)


@pytest.mark.parametrize("q_lens,k_lens,h_q,h_kv,d,causal,window", CASES)
def test_gradients(q_lens, k_lens, h_q, h_kv, d, causal, window):
    for layout in ("fused", "heads"):
        q, k, v, q_at, k_at = make(5, q_lens, k_lens, h_q, h_kv, d, layout, front=3 if layout == "heads" else 0, back=130)
        verify(q, k, v, q_at, k_at, causal, window, same=k_lens is None, layout=layout)


@pytest.mark.parametrize("d", [64, 128])
def test_many_short_sequences(d):
    g = torch.Generator().manual_seed(d)
    lens = torch.randint(0, 40, (1500,), generator=g).tolist()
    lens[700] = 900
    q, k, v, q_at, k_at = make(6, lens, None, 4, 2, d)
    verify(q, k, v, q_at, k_at, True)


@pytest.mark.parametrize("group", [5, 7, 12, 33, 48, 64, 65, 96, 127, 128])
def test_head_groups(group):
    """Groups that do not divide half a row tile, and those of which one token fills more than half."""
    for d, causal, window in ((64, True, -1), (128, True, 20)):
        q, k, v, q_at, k_at = make(group, [3, 0, 70, 1, 33], [5, 4, 200, 129, 0], group, 1, d, back=1)
        verify(q, k, v, q_at, k_at, causal, window)


@pytest.mark.parametrize("d", [64, 128])
def test_calls_in_a_row_over_more_than_the_l2(d):
    """Hundreds of calls that nothing waits between, over inputs that the L2 cannot hold, so that tiles come late: the
    same bits each time. (Once an issuer missed a tile's phase here, one call in ten thousand.)"""
    lens, h_q, h_kv = [1 + 470 * i % 3301 for i in range(24)], 12, 4
    T = sum(lens)
    at = torch.tensor(starts(lens), dtype=torch.int32, device="cuda")
    ws = torch.empty(attn.attn_packed_bwd_workspace_size(T, T, len(lens), h_q, h_kv, d), dtype=torch.uint8, device="cuda")
    states = []
    for seed in range(2):
        q, k, v, q_at, k_at = make(seed, lens, None, h_q, h_kv, d)
        out, lse = forward(q, k, v, q_at, k_at, True, 511)
        dout = torch.randn(q.shape, generator=torch.Generator().manual_seed(seed)).bfloat16().cuda()
        grads = [torch.empty_like(x) for x in (q, k, v)]
        states.append((q, k, v, out, dout, lse, *grads, at, ws))
    call = lambda s: attn.attn_packed_bwd(*s, mask_mode=attn.MASK_CAUSAL, window=511)  # noqa: E731
    want = []
    for s in states:
        call(s)
        torch.cuda.synchronize()
        want.append([x.clone() for x in s[6:9]])
    for i in range(400):
        call(states[i % 2])
    torch.cuda.synchronize()
    assert attn.attn_fault_status() == (attn.ATTN_OK, 0)
    for s, w in zip(states, want):
        for x, y in zip(s[6:9], w):
            assert torch.equal(x, y)


def test_two_calls_at_once_and_captured():
    """On two streams, then from two graphs on one workspace: the results of calls that run alone."""
    lens, h_q, h_kv, d = [700, 3, 0, 260], 6, 2, 64
    T = sum(lens)
    cases, want = [], []
    for seed in (50, 51):
        q, k, v, q_at, k_at = make(seed, lens, None, h_q, h_kv, d)
        out, lse = forward(q, k, v, q_at, k_at, True, -1)
        dout = torch.randn(q.shape, generator=torch.Generator().manual_seed(seed)).bfloat16().cuda()
        want.append(backward(q, k, v, out, lse, dout, q_at, k_at, True, -1))
        cases.append((q, k, v, out, dout, lse, *[torch.zeros_like(x) for x in (q, k, v)]))
    at = torch.tensor(starts(lens), dtype=torch.int32, device="cuda")
    size = attn.attn_packed_bwd_workspace_size(T, T, 4, h_q, h_kv, d)
    ws = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, c, w in zip(streams, cases, ws):
            attn.attn_packed_bwd(*c, at, w, mask_mode=attn.MASK_CAUSAL, stream=s)
    torch.cuda.synchronize()
    for c, w in zip(cases, want):
        for x, y in zip(c[6:], w):
            assert torch.equal(x, y)
            x.zero_()
    torch.cuda.synchronize()
    graphs = []
    for c in cases:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=streams[0]):
            attn.attn_packed_bwd(*c, at, ws[0], mask_mode=attn.MASK_CAUSAL)
    with torch.cuda.stream(streams[0]):
        for g in graphs + graphs:
            g.replay()
    torch.cuda.synchronize()
    for c, w in zip(cases, want):
        for x, y in zip(c[6:], w):
            assert torch.equal(x, y)


def test_thousands_of_sequences():
    g = torch.Generator().manual_seed(8)
    lens = torch.randint(0, 4, (5000,), generator=g).tolist()
    q, k, v, q_at, k_at = make(7, lens, None, 1, 1, 64)
    verify(q, k, v, q_at, k_at, True)


@pytest.mark.parametrize("d", [64, 128])
def test_one_long_among_many(d):
    lens, k_lens = [60] * 700 + [5000] + [1] * 3, [60] * 700 + [9000] + [1] * 3
    q, k, v, q_at, k_at = make(9, lens, k_lens, 2, 2, d)
    verify(q, k, v, q_at, k_at, True)


@pytest.mark.parametrize("d,h_q,h_kv", [(64, 2, 1), (128, 4, 2), (64, 3, 1)])
@pytest.mark.parametrize("causal", [True, False])
def test_long_sequences(d, h_q, h_kv, causal):
    q, k, v, q_at, k_at = make(10, [4099, 1, 2500], None, h_q, h_kv, d)
    verify(q, k, v, q_at, k_at, causal)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
def test_other_sequences_do_not_reach(d, causal):
    """Sequences full of infinities and NaN between others, whose tiles hold their rows."""
    lens = [70, 30, 129, 5, 200, 60]
    q, k, v, q_at, k_at = make(12, lens, None, 6, 2, d)
    out, lse = forward(q, k, v, q_at, k_at, causal)
    dout = torch.randn(q.shape, generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    want = backward(q, k, v, out, lse, dout, q_at, k_at, causal, -1)
    for x, bad in ((q, NAN), (k, INF), (v, NAN), (out, NAN), (lse, NAN), (lse, -INF), (dout, -INF), (dout, NAN)):
        x[q_at[1]:q_at[2]] = bad
        x[q_at[3]:q_at[4]] = bad
    got = backward(q, k, v, out, lse, dout, q_at, k_at, causal, -1)
    for b in (0, 2, 4, 5):
        r = slice(q_at[b], q_at[b + 1])
        for x, y in zip(got, want):
            assert torch.equal(x[r], y[r])


def test_against_differences():
    """dL / dx for L = sum(dO O) along random directions: the float64 forward's central differences."""
    q, k, v, q_at, k_at = make(16, [150, 40], None, 4, 2, 64)
    n = q_at[-1]
    out, lse = forward(q, k, v, q_at, k_at, True, 60)
    dout = torch.randn(q.shape, generator=torch.Generator().manual_seed(5)).bfloat16().cuda()
    grads = backward(q, k, v, out, lse, dout, q_at, k_at, True, 60)
    x = [t.double() for t in (q, k, v)]
    loss = lambda a: (ref.packed(*a, q_at, k_at, 0.125, True, 60)[0][:n] * dout[:n].double()).sum()  # noqa: E731
    _, bounds = ref.packed_bwd(q, k, v, out, lse, dout, q_at, k_at, 0.125, True, 60)
    for i in range(3):
        # the sign of the gradient as direction: every element counts; steps of 2^-10 leave an error of
        # third order, some 2^-20 of the terms' sizes
        step = grads[i].double().sign() * 2.0 ** -10
        up, down = ([t + s * step if j == i else t for j, t in enumerate(x)] for s in (1, -1))
        slope = (loss(up) - loss(down)) / 2
        want = (grads[i].double() * step).sum()
        # independent roundings of each element, and out's own rounding in D
        tol = 6 * 2.0 ** -10 * bounds[i][:n].norm() + 2.0 ** -9 * want.abs()
        assert (slope - want).abs() <= tol, (i, slope, want, tol)


def test_training_step_of_a_packed_batch():
    """Norm + rotation, attention and all their gradients, over one fused projection of packed tokens; two
    calls in a captured graph, with eager calls between, give the eager call's gradients."""
    h_q, h_kv, d, lens = 6, 2, 64, [70, 1, 300, 129]
    q_at = starts(lens)
    T = q_at[-1]
    g = torch.Generator().manual_seed(18)
    qkv = torch.randn(T, h_q + 2 * h_kv, d, generator=g).bfloat16().cuda()
    w = (1 + 0.1 * torch.randn(2, d, generator=g)).bfloat16().cuda()
    dout = torch.randn(T, h_q, d, generator=g).bfloat16().cuda()
    pos = torch.cat([torch.arange(n) for n in lens]).to(torch.int32).cuda()[None]
    angle = torch.arange(300, dtype=torch.float64)[:, None] * 1e4 ** (-torch.arange(32, dtype=torch.float64) / 32)
    table = torch.cat([angle.cos(), angle.sin()], 1).float().cuda()
    at = torch.tensor(q_at, dtype=torch.int32, device="cuda")
    qn, kn = (torch.empty(1, h, T, d, dtype=torch.bfloat16, device="cuda") for h in (h_q, h_kv))
    out, lse = torch.empty(T, h_q, d, dtype=torch.bfloat16, device="cuda"), torch.empty(T, h_q, device="cuda")
    dqn, dkn = torch.empty_like(qn), torch.empty_like(kn)
    dqkv, dw = torch.empty_like(qkv), torch.empty(2, d, device="cuda")
    size = max(attn.attn_packed_fwd_workspace_size(T, 4, h_q, h_kv, d), attn.attn_packed_bwd_workspace_size(T, T, 4, h_q, h_kv, d),
               attn.attn_norm_rope_bwd_workspace_size(1, T, h_q, h_kv, d))
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    x, dx = qkv[None], dqkv[None]
    v, dv = qkv[:, h_q + h_kv:], dqkv[:, h_q + h_kv:]

    def step():
        attn.attn_norm_rope(x[:, :, :h_q], x[:, :, h_q:h_q + h_kv], qn, kn, table, w[0], w[1], positions=pos)
        q, k = qn[0].transpose(0, 1), kn[0].transpose(0, 1)
        attn.attn_packed_fwd(q, k, v, out, at, ws, lse=lse, mask_mode=attn.MASK_CAUSAL)
        attn.attn_packed_bwd(q, k, v, out, dout, lse, dqn[0].transpose(0, 1), dkn[0].transpose(0, 1), dv, at, ws,
                             mask_mode=attn.MASK_CAUSAL)
        attn.attn_norm_rope_bwd(x[:, :, :h_q], x[:, :, h_q:h_q + h_kv], dqn, dkn, dx[:, :, :h_q], dx[:, :, h_q:h_q + h_kv],
                                ws, table, w[0], w[1], dw[0], dw[1], positions=pos)

    step()
    torch.cuda.synchronize()
    assert attn.attn_fault_status() == (attn.ATTN_OK, 0)
    eager, eager_w = dqkv.clone(), dw.clone()
    # the formulas in float64, through automatic differentiation
    leaf, wl = qkv.double().requires_grad_(), w.double().requires_grad_()
    c, s = table[pos[0].long()].double()[:, None].split(32, -1)
    y = leaf[:, :h_q + h_kv]
    y = y / (y.square().mean(-1, keepdim=True) + 1e-6).sqrt() * torch.cat([wl[:1].expand(h_q, d), wl[1:].expand(h_kv, d)])
    y = torch.cat([y[..., :32] * c - y[..., 32:] * s, y[..., 32:] * c + y[..., :32] * s], -1)
    loss = 0
    for b in range(4):
        r = slice(q_at[b], q_at[b + 1])
        z = torch.einsum("ihd,jhd->hij", y[r, :h_q], y[r, h_q:].repeat_interleave(3, 1)) / 8
        z = z.masked_fill(~torch.ones(lens[b], lens[b], dtype=torch.bool, device="cuda").tril(), -INF).softmax(-1)
        o = torch.einsum("hij,jhd->ihd", z, leaf[r, h_q + h_kv:].repeat_interleave(3, 1))
        loss = loss + (o * dout[r].double()).sum()
    loss.backward()
    # bf16 steps between the operators: three roundings one after the other (2^-9 each in the mean), the
    # attention's own P and dS
    for got, want in ((eager, leaf.grad), (eager_w, wl.grad)):
        assert (got.double() - want).norm() <= 2.0 ** -7 * want.norm()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        step()
        step()
    for _ in range(3):
        dqkv.zero_()
        dw.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(dqkv, eager) and torch.equal(dw, eager_w)
        step()
        torch.cuda.synchronize()
        assert torch.equal(dqkv, eager) and torch.equal(dw, eager_w)
