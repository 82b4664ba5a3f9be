"""attn_paged_decode against the plain float64 form (paged_reference.py derives the
tolerance): per element |err| <= 6 qbound, over a tensor ||err|| <= ||qbound||, each row's
lse within its bound. Then the operators together, as a generating program calls them."""
import math

import pytest
import torch

import paged_reference as ref
from transformer_scaled_dot_mha_gb300 import attn

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    attn.lib()


def make(seed, lens, n_q, h_q, h_kv, d, page, e4m3=False, max_pages=0, poison=True):
    """q, pages, table, lens, scales on the CPU. Rows behind every length, unused pages and
    table entries are poison: NaN, and page numbers that do not exist."""
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    need = [-(-x // page) for x in lens]
    total = sum(need) + 2
    order = torch.randperm(total, generator=g)
    table = torch.full((B, max(max(need), max_pages, 1)), -1, dtype=torch.int32)
    table[:, 1::2] = 1 << 30
    kp, vp = (torch.full((total, h_kv, page, d), NAN if poison else 0.0) for _ in range(2))
    at = 0
    for b, n in enumerate(need):
        for x in range(n):
            pid, rows = int(order[at]), min(page, lens[b] - x * page)
            table[b, x] = pid
            kp[pid, :, :rows] = torch.randn(h_kv, rows, d, generator=g)
            vp[pid, :, :rows] = torch.randn(h_kv, rows, d, generator=g)
            at += 1
    scales = [None, None]
    if e4m3:
        scales = [0.01 + 0.01 * torch.rand(h_kv, generator=g) for _ in range(2)]
        kp, vp = ((x / s[:, None, None]).to(torch.float8_e4m3fn) for x, s in zip((kp, vp), scales))
    else:
        kp, vp = kp.bfloat16(), vp.bfloat16()
    q = (1.5 * torch.randn(B, n_q, h_q, d, generator=g)).bfloat16()
    return q, kp, vp, table, torch.tensor(lens, dtype=torch.int32), scales


def run(q, kp, vp, table, lens, scales, scale=None, window=-1, sinks=0, fill=255):
    B, n_q, h_q, d = q.shape
    out = torch.full(q.shape, NAN, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B, n_q, h_q), NAN, device="cuda")
    size = attn.attn_paged_decode_workspace_size(B, n_q, h_q, kp.shape[1], d)
    ws = torch.full((size,), fill, dtype=torch.uint8, device="cuda")
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    attn.attn_paged_decode(dev(q), dev(kp), dev(vp), out, dev(table), dev(lens), ws, lse=lse, scale=scale,
                           window=window, sinks=sinks, k_scale=dev(scales[0]), v_scale=dev(scales[1]))
    torch.cuda.synchronize()
    return out.cpu(), lse.cpu()


def check(got, lse, want, want_lse, qb, lb):
    fin = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    err = torch.where(fin, got.double() - want, 0.0).abs()
    qb = torch.where(fin, qb, 0.0)
    assert torch.all(err <= 6 * qb + 1e-30), f"{(err / qb.clamp_min(1e-30)).max():.2f} of qbound"
    assert err.norm() <= qb.norm()
    none = want_lse == -INF
    assert torch.equal(none, lse == -INF)
    ok = torch.isfinite(want_lse)
    assert torch.all((lse.double() - want_lse)[ok].abs() <= lb[ok])


CASES = [  # lens, n_q, h_q, h_kv, d, page, window, sinks, e4m3, max_pages
    ([1], 1, 1, 1, 64, 16, -1, 0, False, 0),
    ([0, 1, 15, 16, 17, 31, 32, 33], 1, 8, 8, 64, 16, -1, 0, False, 0),
    ([5, 0, 130, 64], 1, 8, 2, 128, 64, -1, 0, False, 0),
    ([5, 0, 130, 64], 1, 8, 2, 128, 64, -1, 0, True, 0),
    ([100, 3, 257], 1, 7, 7, 64, 20, -1, 0, True, 0),
    ([100, 3, 257], 1, 6, 3, 128, 1, -1, 0, False, 0),
    ([700, 1300, 0, 90], 1, 16, 2, 128, 64, -1, 0, False, 0),       # split
    ([1500], 1, 8, 8, 64, 256, -1, 0, False, 64),
    ([2100, 40], 1, 5, 1, 64, 8, -1, 0, True, 300),
    ([33, 2, 0, 1, 600], 3, 4, 2, 64, 16, -1, 0, False, 0),          # some queries before the start
    ([33, 2, 0, 1, 1400], 16, 4, 2, 128, 32, -1, 0, False, 0),       # two row tiles
    ([900, 1100], 5, 8, 1, 128, 16, -1, 0, True, 0),                 # 40 rows
    ([50, 999, 1, 0], 1, 8, 4, 64, 16, 0, 0, False, 0),              # only the key itself
    ([50, 999, 4, 5, 0], 1, 8, 4, 64, 16, 100, 4, False, 0),
    ([50, 999, 4, 5, 0], 4, 8, 4, 64, 16, 33, 7, False, 0),
    ([1900, 300], 7, 2, 2, 128, 64, 1200, 37, True, 0),              # window over several tiles, split
    ([64, 200], 2, 64, 1, 64, 16, -1, 0, False, 0),                  # one key head for 64
    ([300, 70], 1, 4, 4, 64, 16, 50, 1000, False, 0),                # more sinks than keys
    ([60001], 1, 2, 1, 64, 64, -1, 0, False, 0),                     # hundreds of parts of one pair
    ([70003, 5], 3, 4, 1, 128, 256, -1, 0, True, 0),
]


@pytest.mark.parametrize("lens,n_q,h_q,h_kv,d,page,window,sinks,e4m3,max_pages", CASES)
def test_decode(lens, n_q, h_q, h_kv, d, page, window, sinks, e4m3, max_pages):
    q, kp, vp, table, ln, sc = make(21, lens, n_q, h_q, h_kv, d, page, e4m3, max_pages)
    scale = 1 / math.sqrt(d)
    got = run(q, kp, vp, table, ln, sc, None, window, sinks)
    check(*got, *ref.paged_decode(q, kp, vp, table, ln, scale, window, sinks, *sc))
    again = run(q, kp, vp, table, ln, sc, None, window, sinks, fill=0)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


def test_many_sequences():
    """More sequences than a CTA has threads, most of them empty: the list of parts."""
    g = torch.Generator().manual_seed(4)
    lens = [int(x) if keep else 0 for x, keep in zip(torch.randint(1, 90, (300,), generator=g),
                                                     torch.rand(300, generator=g) < 0.4)]
    lens[17] = 1700
    q, kp, vp, table, ln, sc = make(22, lens, 1, 2, 2, 64, 16)
    check(*run(q, kp, vp, table, ln, sc), *ref.paged_decode(q, kp, vp, table, ln, 0.125))


@pytest.mark.parametrize("B,n_q,h_q,h_kv,d,window", [
    (400, 1, 8, 8, 64, -1),    # more pairs than parts of the list
    (130, 1, 32, 8, 128, -1),  # four rows a pair
    (260, 4, 16, 4, 64, 70),   # two row tiles' worth of rows, short windows
])
def test_large_batches_of_short_sequences(B, n_q, h_q, h_kv, d, window):
    """A capacity far above the lengths: the device cuts up the list, whatever its shape."""
    g = torch.Generator().manual_seed(B)
    lens = torch.randint(0, 60, (B,), generator=g).tolist()
    lens[3], lens[B // 2] = 333, 0
    q, kp, vp, table, ln, sc = make(B, lens, n_q, h_q, h_kv, d, 16, max_pages=100)
    check(*run(q, kp, vp, table, ln, sc, None, window),
          *ref.paged_decode(q, kp, vp, table, ln, 1 / math.sqrt(d), window))


def test_two_streams_at_once():
    """Calls on two streams, each with its own workspace, do not touch each other."""
    cases = [make(61 + i, [700 + 90 * i, 1200, 3], 1, 8, 2, 64, 16) for i in range(2)]
    want = [run(*c) for c in cases]
    dev = [[x.cuda() if torch.is_tensor(x) else x for x in c] for c in cases]
    outs = [[torch.empty_like(c[0]) for _ in range(20)] for c in dev]
    size = attn.attn_paged_decode_workspace_size(3, 1, 8, 2, 64)
    ws = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for i in range(20):
        for (q, kp, vp, table, ln, _), out, w, st in zip(dev, outs, ws, streams):
            attn.attn_paged_decode(q, kp, vp, out[i], table, ln, w, stream=st)
    torch.cuda.synchronize()
    for (out, _), got in zip(want, outs):
        assert all(torch.equal(out, x.cpu()) for x in got)


def test_lengths_are_clamped_and_scale_used_as_given():
    q, kp, vp, table, _, sc = make(23, [64, 64, 64], 1, 2, 2, 64, 16)
    ln = torch.tensor([-5, 64, 1 << 30], dtype=torch.int32)
    for scale in (-0.3, 0.0, 0.7):
        check(*run(q, kp, vp, table, ln, sc, scale), *ref.paged_decode(q, kp, vp, table, ln, scale))


@pytest.mark.parametrize("e4m3", [False, True])
def test_missing_pages_inside_the_length(e4m3):
    """Keys of a table entry that names no page are illegal; all of them: an empty row."""
    q, kp, vp, table, ln, sc = make(24, [100, 80, 1300], 2, 4, 2, 64, 16, e4m3)
    table[0, 2], table[0, 6] = -7, kp.shape[0]
    table[1, :] = -1
    table[2, 5:40] = 1 << 29
    check(*run(q, kp, vp, table, ln, sc), *ref.paged_decode(q, kp, vp, table, ln, 0.125, -1, 0, *sc))


@pytest.mark.parametrize("d,e4m3", [(64, False), (128, False), (64, True), (128, True)])
def test_specials_reach_only_the_rows_that_see_them(d, e4m3):
    """inf or NaN in the newest key's value (and key) belongs to the newest query alone; in a
    key that has left some rows' windows, to the others."""
    lens, n_q, page, window = [40, 90], 4, 16, 30
    q, kp, vp, table, ln, sc = make(25, lens, n_q, 4, 2, d, page, e4m3)
    bad = NAN if e4m3 else INF
    raw = [x.float() for x in (kp, vp)]
    for b, length in enumerate(lens):
        at = length - 1
        raw[1][table[b, at // page], 0, at % page, 3] = bad
        raw[0][table[b, at // page], 1, at % page, 5] = NAN
        at = length - n_q - window + 1  # seen by the first two queries only
        raw[1][table[b, at // page], 1, at % page, d - 1] = bad
    kp, vp = (x.to(y.dtype) for x, y in zip(raw, (kp, vp)))
    out, lse = run(q, kp, vp, table, ln, sc, None, window)
    want, want_lse, qb, lb = ref.paged_decode(q, kp, vp, table, ln, 1 / math.sqrt(d), window, 0, *sc)
    assert torch.equal(torch.isfinite(out), torch.isfinite(want))
    fin = torch.isfinite(want)
    err = (out.double() - want).abs()[fin]
    assert torch.all(err <= 6 * qb[fin]) and torch.isfinite(out[:, 0, 0, :3]).all()
    assert torch.isfinite(want[:, :3, :2]).all()  # key head 0: the first three queries are clean
    ok = torch.isfinite(want_lse)
    assert torch.equal(ok, torch.isfinite(lse)) and torch.all((lse.double() - want_lse)[ok].abs() <= lb[ok])


def test_row_of_another_head_is_not_touched_by_special_queries():
    q, kp, vp, table, ln, sc = make(26, [70], 1, 4, 1, 64, 16)
    q[0, 0, 1, 7] = NAN
    q[0, 0, 2] = 0
    out, _ = run(q, kp, vp, table, ln, sc)
    want, _, qb, _ = ref.paged_decode(q, kp, vp, table, ln, 0.125)
    assert torch.isnan(out[0, 0, 1]).all()
    for h in (0, 2, 3):
        assert torch.all((out[0, 0, h].double() - want[0, 0, h]).abs() <= 6 * qb[0, 0, h])


def test_e4m3_query_ranges():
    """Queries of very large and very small rows keep their precision (they are scaled to
    f16's range by powers of two)."""
    q, kp, vp, table, ln, sc = make(27, [60], 1, 4, 2, 128, 16, True)
    for h, s in enumerate((1e-30, 1e30, 1.0, 3e38)):
        q[0, 0, h] = (q[0, 0, h].float().clamp(-1, 1) * s).bfloat16()
    for scale in (1e-30, 1e-33):
        scale = float(torch.tensor(scale))  # as the float argument has it
        check(*run(q, kp, vp, table, ln, sc, scale), *ref.paged_decode(q, kp, vp, table, ln, scale, -1, 0, *sc))


def test_cache_beyond_four_gigabytes():
    """Byte offsets past 32 bits: the pages used lie at the end of a 5 GB pool."""
    page, h_kv, d = 64, 8, 128
    n_pages = 5 * (1 << 30) // (page * h_kv * d * 2)
    q, kp, vp, table, ln, sc = make(28, [150], 1, 8, h_kv, d, page, poison=False)
    out = torch.empty(q.shape, dtype=torch.bfloat16, device="cuda")
    big = [torch.empty(n_pages, h_kv, page, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    for x, y in zip(big, (kp, vp)):
        x[-len(y):] = y.cuda()
    far = torch.where(table >= 0, table + (n_pages - len(kp)), table).int()
    ws = torch.empty(attn.attn_paged_decode_workspace_size(1, 1, 8, h_kv, d), dtype=torch.uint8, device="cuda")
    attn.attn_paged_decode(q.cuda(), *big, out, far.cuda(), ln.cuda(), ws)
    # and the append: one more token in the last page's free rows
    k = torch.randn(1, h_kv, d, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    pos = torch.tensor([150], dtype=torch.int32, device="cuda")
    attn.attn_paged_append(k, k, *big, pos, far.cuda())
    torch.cuda.synchronize()
    want, _, qb, _ = ref.paged_decode(q, kp, vp, table, ln, 1 / math.sqrt(d))
    assert torch.all((out.cpu().double() - want).abs() <= 6 * qb)
    for x in big:
        assert torch.equal(x[far[0, 2], :, 150 - 128], k[0])


# ---------------------------------------------------------------- together
def full_attention(q, k, v, window, sinks, scale):
    """Float64 causal attention of [n, h, d] rows with shared heads."""
    n, h, d = q.shape
    group = h // k.shape[1]
    out = torch.zeros(n, h, d, dtype=torch.float64)
    for i in range(n):
        keys = ref.legal_keys(i + 1, 1, 0, window, sinks)
        for z in range(h):
            s = scale * (k[keys, z // group] @ q[i, z])
            out[i, z] = torch.softmax(s, 0) @ v[keys, z // group]
    return out


@pytest.mark.parametrize("window,sinks,e4m3,captured",
                         [(-1, 0, False, False), (20, 3, False, True), (-1, 0, True, True)])
def test_generation(window, sinks, e4m3, captured):
    """Two prompts appended in one packed call, then tokens one at a time (append + decode,
    also as a captured graph replayed with new inputs), on a side stream. Against the
    float64 attention of the whole sequences over the float64 q, k, v rounded to their stored
    types. Then the weights' and the output's rounding remain (u / 2 each in root mean square,
    0.7 x 2^-8 in quadrature), and the few stored values that lie so near a rounding border
    that fp32 takes the other side (2^-12 of the bf16 ones): within 2 x 2^-8 in norm."""
    B, h_q, h_kv, d, page, steps, prompt = 2, 4, 2, 64, 16, 12, [21, 34]
    g = torch.Generator().manual_seed(31)
    total = [p + steps for p in prompt]
    x = [torch.randn(n, h_q + 2 * h_kv, d, generator=g).bfloat16() for n in total]
    w = [(1 + 0.2 * torch.randn(d, generator=g)).bfloat16() for _ in range(2)]
    rot = ref.rotation_table(64, d)
    table = torch.randperm(8, generator=g).int().view(2, 4)
    kind = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    kp, vp = (torch.full((8, h_kv, page, d), NAN, device="cuda").to(kind) for _ in range(2))
    scales = dict(k_scale=torch.full((h_kv,), 2.0 ** -5, device="cuda"),
                  v_scale=torch.full((h_kv,), 2.0 ** -6, device="cuda")) if e4m3 else {}
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        common = dict(cos_sin=rot.cuda(), q_weight=w[0].cuda(), k_weight=w[1].cuda(), **scales)
        dtable = table.cuda()
        packed = torch.cat([x[0][:prompt[0]], x[1][:prompt[1]]]).cuda()
        pos = torch.cat([torch.arange(n) for n in prompt]).int().cuda()
        seq = torch.repeat_interleave(torch.arange(2), torch.tensor(prompt)).int().cuda()
        q_out = torch.empty(len(pos), h_q, d, dtype=torch.bfloat16, device="cuda")
        split = lambda t: (t[:, h_q:h_q + h_kv], t[:, h_q + h_kv:])  # noqa: E731
        attn.attn_paged_append(*split(packed), kp, vp, pos, dtable, seq_ids=seq, q=packed[:, :h_q], q_out=q_out,
                               **common)
        token = torch.empty(B, h_q + 2 * h_kv, d, dtype=torch.bfloat16, device="cuda")
        lens = torch.tensor(prompt, dtype=torch.int32, device="cuda")
        at = torch.empty_like(lens)
        q1, out = (torch.empty(B, 1, h_q, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        ws = torch.empty(attn.attn_paged_decode_workspace_size(B, 1, h_q, h_kv, d), dtype=torch.uint8, device="cuda")

        def step():
            at.copy_(lens)
            lens.add_(1)
            attn.attn_paged_append(*split(token), kp, vp, at, dtable, q=token[:, :h_q], q_out=q1.view(B, h_q, d),
                                   **common)
            attn.attn_paged_decode(q1, kp, vp, out, dtable, lens, ws, window=window, sinks=sinks, **scales)

        got, graph = [], None
        if captured:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=stream):
                step()
        for i in range(steps):
            token.copy_(torch.stack([x[b][prompt[b] + i] for b in range(B)]))
            graph.replay() if graph else step()
            got.append(out[:, 0].clone())
    stream.synchronize()
    for b in range(B):
        q, k = (torch.stack([ref.norm_rope(x[b][i, lo:hi], wt, rot[i], 1e-6, False)[0] for i in range(total[b])])
                for lo, hi, wt in ((0, h_q, w[0]), (h_q, h_q + h_kv, w[1])))
        v = x[b][:, h_q + h_kv:].double()
        step_k, step_v = (2.0 ** -5, 2.0 ** -6) if e4m3 else (1, 1)  # the scales: powers of two
        q = q.bfloat16().double()
        k, v = ((y / step).to(kind).double() * step for y, step in ((k, step_k), (v, step_v)))
        want = full_attention(q, k, v, window, sinks, 0.125)[prompt[b]:]
        err = torch.stack([o[b].double().cpu() for o in got]) - want
        assert err.norm() <= 2 * ref.U_BF16 * want.norm()


def test_training_form_feeds_attention():
    """attn_norm_rope -> attn_fwd -> attn_bwd -> attn_norm_rope_bwd, against float64 autograd
    of the same chain in norm: bf16 roundings of q, k, the weights, dS and the gradients on
    the way are some ten steps of relative 2^-8 each, in quadrature 3.2 x 2^-8 = 1.3e-2; twice that."""
    B, n, h, d = 1, 130, 2, 64
    g = torch.Generator().manual_seed(41)
    qkv = torch.randn(B, n, 3 * h, d, generator=g).bfloat16()
    w = [(1 + 0.2 * torch.randn(d, generator=g)).bfloat16() for _ in range(2)]
    rot, go = ref.rotation_table(n, d), torch.randn(B, h, n, d, generator=g).bfloat16()
    dq_in = qkv.cuda()
    q, k, v = dq_in[:, :, :h], dq_in[:, :, h:2 * h], dq_in[:, :, 2 * h:].transpose(1, 2).contiguous()
    qo, ko, out = (torch.empty(B, h, n, d, dtype=torch.bfloat16, device="cuda") for _ in range(3))
    lse = torch.empty(B, h, n, device="cuda")
    attn.attn_norm_rope(q, k, qo, ko, rot.cuda(), w[0].cuda(), w[1].cuda())
    attn.attn_fwd(qo, ko, v, out, lse, mask_mode=attn.MASK_CAUSAL)
    grads = [torch.empty_like(qo) for _ in range(3)]
    ws = torch.empty(attn.attn_bwd_workspace_size(B, h, n, d), dtype=torch.uint8, device="cuda")
    attn.attn_bwd(qo, ko, v, out, go.cuda(), lse, *grads, ws, mask_mode=attn.MASK_CAUSAL)
    dqkv = torch.zeros_like(dq_in)
    dw = [torch.empty(d, device="cuda") for _ in range(2)]
    ws = torch.empty(attn.attn_norm_rope_bwd_workspace_size(B, n, h, h, d), dtype=torch.uint8, device="cuda")
    attn.attn_norm_rope_bwd(q, k, grads[0], grads[1], dqkv[:, :, :h], dqkv[:, :, h:2 * h], ws, rot.cuda(), w[0].cuda(),
                            w[1].cuda(), *dw)
    dqkv[:, :, 2 * h:] = grads[2].transpose(1, 2)
    torch.cuda.synchronize()
    leaf = qkv.double().requires_grad_()
    lw = [t.double().requires_grad_() for t in w]

    def nr(x, weight):
        y = x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt() * weight
        c, s = (t.double()[None, :, None] for t in rot.split(d // 2, 1))
        a, b = y.split(d // 2, -1)
        return torch.cat([a * c - b * s, b * c + a * s], -1).transpose(1, 2)

    s = nr(leaf[:, :, :h], lw[0]) @ nr(leaf[:, :, h:2 * h], lw[1]).transpose(2, 3) / math.sqrt(d)
    s = s.masked_fill(torch.ones(n, n).triu(1).bool(), -INF)
    o = torch.softmax(s, -1) @ leaf[:, :, 2 * h:].transpose(1, 2)
    o.backward(go.double())
    rel = lambda a, b: ((a.double().cpu() - b).norm() / b.norm()).item()  # noqa: E731
    assert rel(out, o.detach()) <= 2.6e-2
    for part in (slice(0, h), slice(h, 2 * h), slice(2 * h, 3 * h)):
        assert rel(dqkv[:, :, part], leaf.grad[:, :, part]) <= 2.6e-2
    assert rel(dw[0], lw[0].grad) <= 2.6e-2 and rel(dw[1], lw[1].grad) <= 2.6e-2


def test_refusals():
    q, kp, vp, table, ln, sc = (x.cuda() if torch.is_tensor(x) else x for x in make(51, [20, 30], 1, 4, 2, 64, 16))
    ws = torch.empty(attn.attn_paged_decode_workspace_size(2, 1, 4, 2, 64), dtype=torch.uint8, device="cuda")
    ok = dict(q=q, k_pages=kp, v_pages=vp, out=torch.empty_like(q), page_table=table, cache_lens=ln, workspace=ws)
    attn.attn_paged_decode(**ok)
    one = torch.ones(2, device="cuda")
    for bad in (dict(q=q.float()), dict(v_pages=vp[1:]), dict(k_pages=kp[..., :32]), dict(page_table=table[:1]),
                dict(cache_lens=ln.long()), dict(k_scale=one), dict(lse=torch.empty(2, 4, device="cuda")),
                dict(k_pages=kp.to(torch.float8_e4m3fn)),
                dict(k_pages=kp.to(torch.float8_e4m3fn), v_pages=vp.to(torch.float8_e4m3fn), k_scale=one),
                dict(workspace=ws.cpu()), dict(page_table=table.cpu())):
        with pytest.raises(ValueError):
            attn.attn_paged_decode(**(ok | bad))
    for bad in (dict(workspace=ws[:-1]), dict(window=-2), dict(sinks=-1), dict(scale=NAN)):
        with pytest.raises(attn.AttnError):
            attn.attn_paged_decode(**(ok | bad))
    torch.cuda.synchronize()
