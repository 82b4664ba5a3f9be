"""attn_norm_rope, its gradients and attn_paged_append at sizes where a lane group walks over
several heads and a warp over several items: whole-tensor float64 forms on the CPU, the
tolerances of test_rope_gpu.py. A lane group takes as many heads, up to 8, as leave 304 CTAs
(a CTA has 32 tokens of 64 columns, or 16 of 128, side by side), and the gradients' items (8
or 4 tokens of one head) are cut into equal runs for the warps of 456 CTAs, shared out by the
kinds' heads: the tests state which of these they reach."""
import pytest
import torch

import paged_reference as ref
from test_rope_gpu import EPS, NAN, check, dev, rand
from transformer_scaled_dot_mha_gb300 import attn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    attn.lib()


def heads_per_group(tokens, d, heads):
    tiles = -(-tokens // (2048 // d))
    return next((hp for hp in (8, 4, 2) if tiles * sum(-(-h // hp) for h in heads) >= 304), 1)


def items_per_warp(tokens, d, h_q, h_kv):
    share = min(max((456 * h_q + (h_q + h_kv) // 2) // (h_q + h_kv), 1), 455)
    total = [-(-tokens // (512 // d)) * h for h in (h_q, h_kv)]
    return [-(-t // (4 * min(-(-t // 4), s))) for t, s in zip(total, (share, 456 - share))]


def turn(y, rows, interleaved, back=False):
    """y [tokens, h, d] float64, rows [tokens, d_rot]: (turned, sizes of the terms)."""
    m = rows.shape[1] // 2
    a, b = ref.pair_columns(2 * m, interleaved)
    c, s = rows[:, None, :m].double(), rows[:, None, m:].double() * (-1 if back else 1)
    o, size = y.clone(), y.abs()
    o[..., a], o[..., b] = y[..., a] * c - y[..., b] * s, y[..., b] * c + y[..., a] * s
    size[..., a] = (y[..., a] * c).abs() + (y[..., b] * s).abs()
    size[..., b] = (y[..., b] * c).abs() + (y[..., a] * s).abs()
    return o, size


def forward(x, weight, rows, inter):
    y = x.double()
    if weight is not None:
        y = y / (y.square().mean(-1, keepdim=True) + EPS).sqrt() * weight.double()
    return turn(y, rows, inter)


def inputs(seed, B, n, h_q, h_kv, d, d_rot, norm, given):
    g = torch.Generator().manual_seed(seed)
    qkv = rand(g, B, n, (h_q + 2 * h_kv) * d + 8, scale=1.7)
    w = [(1 + 0.2 * torch.randn(d, generator=g)).to(torch.bfloat16) if norm else None for _ in range(2)]
    table = ref.rotation_table(n + 5, d_rot)
    pos = torch.arange(n).repeat(B, 1)
    if given:
        pos = torch.randint(-1, n + 7, (B, n), generator=g)
    real = ((pos >= 0) & (pos < n + 5)).view(-1)
    return g, qkv, w, table, pos, real, table[pos.view(-1).clamp(0, n + 4)]


def split(t, h_q, h_kv, d):
    return [x.unflatten(-1, (-1, d)) for x in (t[..., :h_q * d], t[..., h_q * d:(h_q + h_kv) * d])]


SIZES = [  # B, n, h_q, h_kv, d, d_rot, norm, interleaved, positions given, heads per lane group
    (3, 1100, 9, 7, 64, 64, True, False, True, 8),     # a second unit of one head, one of seven
    (1, 557, 64, 8, 128, 128, True, True, False, 8),
    (1, 1637, 5, 1, 128, 48, True, False, True, 4),    # four heads and one
    (1, 1289, 7, 7, 64, 16, False, True, False, 2),
    (2, 811, 7, 3, 64, 64, True, True, True, 2),       # a ragged last tile
]


@pytest.mark.parametrize("B,n,h_q,h_kv,d,d_rot,norm,inter,given,hp", SIZES)
def test_forward_walks_over_heads(B, n, h_q, h_kv, d, d_rot, norm, inter, given, hp):
    assert heads_per_group(B * n, d, (h_q, h_kv)) == hp
    _, qkv, w, table, pos, real, rows = inputs(81, B, n, h_q, h_kv, d, d_rot, norm, given)
    q, k = split(qkv.cuda(), h_q, h_kv, d)
    outs = [torch.full((B, h, n, d), NAN, dtype=torch.bfloat16, device="cuda") for h in (h_q, h_kv)]
    attn.attn_norm_rope(q, k, *outs, dev(table), *map(dev, w), positions=pos.int().cuda() if given else None, eps=EPS,
                        interleaved=inter)
    torch.cuda.synchronize()
    for x, weight, got in ((q, w[0], outs[0]), (k, w[1], outs[1])):
        want, size = forward(x.cpu().flatten(0, 1), weight, rows, inter)
        want[~real], size[~real] = 0, 0
        check(got.transpose(1, 2).flatten(0, 1), want, size)


GRADS = [  # B, n, h_q, h_kv, d, d_rot, norm, interleaved, positions given, items per warp (queries, keys)
    (1, 1500, 12, 5, 64, 64, True, False, False, (2, 2)),
    (1, 2100, 12, 5, 64, 64, True, True, True, (3, 3)),
    (3, 1100, 12, 5, 64, 48, True, False, True, (4, 4)),     # the ring of three items is reused
    (1, 4001, 9, 7, 128, 128, True, False, False, (9, 9)),   # the keys' runs cross token groups
    (2, 4999, 1, 1, 128, 64, True, True, True, (3, 3)),      # other tokens in every item
    (1, 4001, 9, 7, 128, 128, False, True, True, (9, 9)),    # without a norm six items are in flight
    (2, 1999, 8, 1, 64, 64, True, False, True, (3, 3)),
]


@pytest.mark.parametrize("B,n,h_q,h_kv,d,d_rot,norm,inter,given,items", GRADS)
def test_gradients_of_many_items(B, n, h_q, h_kv, d, d_rot, norm, inter, given, items):
    assert tuple(items_per_warp(B * n, d, h_q, h_kv)) == items
    gen, qkv, w, table, pos, real, rows = inputs(82, B, n, h_q, h_kv, d, d_rot, norm, given)
    grads = [rand(gen, B, h, n, d) for h in (h_q, h_kv)]
    gq = qkv.cuda()
    spare = torch.full_like(gq, 7.0)
    q, k, dq, dk = *split(gq, h_q, h_kv, d), *split(spare, h_q, h_kv, d)
    dw = [torch.full((d,), NAN, device="cuda") if norm else None for _ in range(2)]
    ws = None
    if norm:
        ws = torch.full((attn.attn_norm_rope_bwd_workspace_size(B, n, h_q, h_kv, d),), 255, dtype=torch.uint8,
                        device="cuda")
    for again in range(2):
        attn.attn_norm_rope_bwd(q, k, grads[0].cuda(), grads[1].cuda(), dq, dk, ws, dev(table), *map(dev, w), *dw,
                                positions=pos.int().cuda() if given else None, eps=EPS, interleaved=inter)
        torch.cuda.synchronize()
        got = [spare.clone()] + [x.clone() for x in dw if x is not None]
        if again:
            assert all(torch.equal(a, b) for a, b in zip(first, got))
        first = got
    for x, weight, gr, got, got_w in ((q, w[0], grads[0], dq, dw[0]), (k, w[1], grads[1], dk, dw[1])):
        gy, gsize = turn(gr.transpose(1, 2).flatten(0, 1).double(), rows, inter, back=True)
        want, size = gy, gsize
        if norm:
            x = x.cpu().flatten(0, 1).double()
            r = 1 / (x.square().mean(-1, keepdim=True) + EPS).sqrt()
            u, usize = gy * weight.double(), gsize * weight.double().abs()
            want = r * (u - x * r ** 2 * (u * x).mean(-1, keepdim=True))
            size = r * (usize + x.abs() * r ** 2 * (usize * x.abs()).mean(-1, keepdim=True))
            want_w, size_w = (gy * x * r)[real].sum((0, 1)), (gsize * x.abs() * r)[real].sum((0, 1))
            err = (got_w.double().cpu() - want_w).abs()
            assert torch.all(err <= (real.sum() * x.shape[1] * 2.0 ** -24 + 2.0 ** -18) * size_w)
        want[~real], size[~real] = 0, 0
        check(got.flatten(0, 1), want, size)
    assert torch.all(spare[..., (h_q + h_kv) * d:] == 7.0)


@pytest.mark.parametrize("toks,h_q,h_kv,d,d_rot,norm,inter,page,e4m3,hp", [
    ([900, 1, 1283, 301], 9, 7, 64, 64, True, False, 20, False, 8),
    ([600, 333, 511], 5, 1, 128, 48, False, True, 64, True, 4),
    ([940, 79], 7, 5, 64, 32, True, False, 16, True, 2),
    ([1500, 777, 1111], 0, 11, 64, 64, True, True, 7, False, 8),
])
def test_append_walks_over_heads(toks, h_q, h_kv, d, d_rot, norm, inter, page, e4m3, hp):
    T = sum(toks) + 3
    assert heads_per_group(T, d, (h_q, h_kv, h_kv)) == hp
    g = torch.Generator().manual_seed(83)
    need = [-(-t // page) for t in toks]
    order, at = torch.randperm(sum(need) + 2, generator=g), 0
    table = torch.full((len(toks), max(need)), -1, dtype=torch.int32)
    for s, n in enumerate(need):
        table[s, :n], at = order[at:at + n].int(), at + n
    kind = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    before = torch.randn(len(order), h_kv, page, d, generator=g).to(kind)
    gk, gv = before.cuda(), before.cuda()
    seq = torch.repeat_interleave(torch.arange(len(toks)), torch.tensor(toks))
    pos = torch.cat([torch.arange(t) for t in toks])
    mix = torch.randperm(len(seq), generator=g)  # tokens in any order
    seq, pos = torch.cat([seq[mix], torch.zeros(3).long()]), torch.cat([pos[mix], torch.full((3,), -1)])
    qkv = rand(g, T, (h_q + 2 * h_kv) * d + 8, scale=1.7)
    parts = [x.unflatten(-1, (-1, d)) if x.shape[-1] else None for x in
             qkv.cuda().split([h_q * d, h_kv * d, h_kv * d, 8], -1)[:3]]
    w = [(1 + 0.2 * torch.randn(d, generator=g)).to(torch.bfloat16) if norm else None for _ in range(2)]
    rot = ref.rotation_table(max(toks), d_rot)
    scale = [0.01 + 0.05 * torch.rand(h_kv, generator=g) if e4m3 else None for _ in range(2)]
    q_out = torch.full((T, h_q, d), 5.0, dtype=torch.bfloat16, device="cuda") if h_q else None
    attn.attn_paged_append(parts[1], parts[2], gk, gv, pos.int().cuda(), table.cuda(), seq_ids=seq.int().cuda(),
                           q=parts[0], q_out=q_out, cos_sin=rot.cuda(), q_weight=dev(w[0]) if h_q else None,
                           k_weight=dev(w[1]), k_scale=dev(scale[0]), v_scale=dev(scale[1]), eps=EPS, interleaved=inter)
    torch.cuda.synchronize()
    parts = [None if x is None else x[:-3].cpu() for x in parts]
    seq, pos = seq[:-3], pos[:-3]
    page_of, rows = table[seq, pos // page].long(), rot[pos]
    if h_q:
        check(q_out[:-3], *forward(parts[0], w[0], rows, inter))
        assert torch.all(q_out[-3:] == 5.0)
    want, size = forward(parts[1], w[1], rows, inter)
    got_k, got_v = (x.cpu()[page_of, :, pos % page] if not e4m3 else
                    x.cpu().view(torch.int8)[page_of, :, pos % page].view(kind) for x in (gk, gv))
    if e4m3:
        s = scale[0].double()[:, None]
        y = (want / s).clamp(-448, 448)
        step = torch.maximum(2.0 ** -4 * y.abs(), torch.tensor(2.0 ** -10))
        assert torch.all((got_k.double() - y).abs() <= step + 2 * ref.U_ROPE * size / s)
        exact_v = (parts[2].float() / scale[1][:, None]).clamp(-448, 448).to(kind)
        assert torch.equal(got_v.view(torch.int8), exact_v.view(torch.int8))
    else:
        check(got_k, want, size)
        assert torch.equal(got_v, parts[2])
    touched = torch.zeros(len(order), page, dtype=torch.bool)
    touched[page_of, pos % page] = True
    raw = torch.int8 if e4m3 else torch.int16
    for got in (gk, gv):
        assert torch.all((got.cpu().view(raw) == before.view(raw)).all(-1).all(1) | touched)


@pytest.mark.parametrize("d", [64, 128])
def test_padding_tokens_may_hold_anything(d):
    """Infinities and NaN in padding tokens reach nothing: zeros there, all else bit for bit as with
    zeros in their place."""
    B, n, h_q, h_kv = 2, 700, 3, 2
    gen, qkv, w, table, pos, real, _ = inputs(84, B, n, h_q, h_kv, d, d, True, True)
    grads = [rand(gen, B, h, n, d) for h in (h_q, h_kv)]
    assert 0 < (~real).sum() < B * n
    got = []
    for fill in (0.0, NAN, float("inf")):
        x, gr = qkv.clone(), [t.clone() for t in grads]
        x.view(B * n, -1)[~real] = fill
        for t in gr:
            t.transpose(1, 2)[~real.view(B, n)] = fill
        q, k = split(x.cuda(), h_q, h_kv, d)
        outs = [torch.full((B, h, n, d), NAN, dtype=torch.bfloat16, device="cuda") for h in (h_q, h_kv)]
        back = [torch.full((B, n, h, d), NAN, dtype=torch.bfloat16, device="cuda") for h in (h_q, h_kv)]
        dw = [torch.full((d,), NAN, device="cuda") for _ in range(2)]
        ws = torch.empty(attn.attn_norm_rope_bwd_workspace_size(B, n, h_q, h_kv, d), dtype=torch.uint8, device="cuda")
        at = pos.int().cuda()
        attn.attn_norm_rope(q, k, *outs, dev(table), *map(dev, w), positions=at, eps=EPS)
        attn.attn_norm_rope_bwd(q, k, *map(dev, gr), *back, ws, dev(table), *map(dev, w), *dw, positions=at, eps=EPS)
        torch.cuda.synchronize()
        got.append([t.cpu() for t in outs + back + dw])
        for t in got[-1][:2]:
            assert torch.all(t.transpose(1, 2)[~real.view(B, n)] == 0)
        for t in got[-1][2:4]:
            assert torch.all(t[~real.view(B, n)] == 0)
    for other in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(got[0], other))
    assert all(torch.isfinite(t).all() for t in got[0])
