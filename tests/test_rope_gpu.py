"""attn_norm_rope, its gradients and attn_paged_append against the plain float64 forms.

Tolerance per output element: one rounding to the stored type (bf16: 2^-8 of the value;
e4m3: 2^-4 of it, or half a step of 2^-9 below the normal range) plus U_ROPE of the sizes
of the terms it is made of (paged_reference.py counts the fp32 roundings). Gradients of the
weights are fp32 sums over R rows: any order of summation is within R 2^-24 of the terms'
sizes, plus 2^-18 for the terms. Copied and untouched values have to be equal bit for bit.
"""
import pytest
import torch

import paged_reference as ref
from transformer_scaled_dot_mha_gb300 import attn

pytestmark = pytest.mark.gpu
EPS = 1e-6
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    attn.lib()


def rand(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g) * scale).to(torch.bfloat16)


def dev(t):
    return None if t is None else t.cuda()


def check(got, want, size, u=ref.U_BF16):
    err = (got.double().cpu() - want).abs()
    bound = u * want.abs() + (1 + u) * ref.U_ROPE * size
    assert torch.all(err <= bound), f"off by {(err / bound.clamp_min(1e-300)).max():.3f} of the bound"


def setup(seed, B, n, h_q, h_kv, d, d_rot, norm, positions):
    """Views q, k of a fused projection with 8 spare columns, weights, table, positions."""
    g = torch.Generator().manual_seed(seed)
    wide = (h_q + 2 * h_kv) * d + 8
    qkv = rand(g, B, n, wide, scale=1.7)
    w = [(1 + 0.2 * torch.randn(d, generator=g)).to(torch.bfloat16) if norm else None for _ in range(2)]
    n_pos = n + 5
    table = ref.rotation_table(n_pos, d_rot) if d_rot else None
    pos = None
    if positions:
        pos = torch.randint(-1, n_pos + 2, (B, n), generator=g, dtype=torch.int32)  # some before, some behind the table
    return qkv, w, table, pos




CASES = [  # B, n, h_q, h_kv, d, d_rot, norm, interleaved, positions given
    (1, 1, 1, 1, 64, 64, True, False, False),
    (2, 33, 8, 8, 64, 64, True, False, False),
    (3, 7, 5, 1, 64, 64, True, True, True),
    (2, 40, 8, 2, 128, 128, True, False, True),
    (1, 77, 4, 4, 128, 128, False, True, False),
    (2, 9, 3, 3, 128, 64, True, False, False),
    (2, 9, 3, 3, 128, 48, False, False, True),
    (2, 19, 6, 2, 64, 16, True, True, False),
    (2, 18, 6, 2, 64, 48, True, False, True),
    (1, 65, 9, 7, 64, 0, True, False, False),
    (1, 600, 16, 4, 64, 64, True, False, False),
]


@pytest.mark.parametrize("B,n,h_q,h_kv,d,d_rot,norm,inter,given", CASES)
def test_forward(B, n, h_q, h_kv, d, d_rot, norm, inter, given):
    qkv, w, table, pos = setup(1, B, n, h_q, h_kv, d, d_rot, norm, given)
    gq = qkv.cuda()
    q, k = (x.unflatten(-1, (-1, d)) for x in (gq[..., :h_q * d], gq[..., h_q * d:(h_q + h_kv) * d]))
    outs = [torch.full((B, h, n, d), NAN, dtype=torch.bfloat16, device="cuda") for h in (h_q, h_kv)]
    attn.attn_norm_rope(q, k, *outs, dev(table), *map(dev, w), positions=dev(pos), eps=EPS, interleaved=inter)
    torch.cuda.synchronize()
    for x, weight, got in ((q, w[0], outs[0]), (k, w[1], outs[1])):
        x = x.cpu()
        want = torch.zeros(got.shape, dtype=torch.float64)
        size = torch.zeros_like(want)
        for b in range(B):
            for i in range(n):
                at = i if pos is None else int(pos[b, i])
                if at < 0 or (table is not None and at >= table.shape[0]):
                    continue  # padding: zeros
                row = None if table is None else table[at]
                want[b, :, i], size[b, :, i] = ref.norm_rope(x[b, i], weight, row, EPS, inter)
        check(got, want, size)


@pytest.mark.parametrize("B,n,h_q,h_kv,d,d_rot,norm,inter,given", CASES)
def test_gradients(B, n, h_q, h_kv, d, d_rot, norm, inter, given):
    qkv, w, table, pos = setup(2, B, n, h_q, h_kv, d, d_rot, norm, given)
    gen = torch.Generator().manual_seed(3)
    g = [rand(gen, B, h, n, d) for h in (h_q, h_kv)]
    gq = qkv.cuda()

    def split(t):
        return [x.unflatten(-1, (-1, d)) for x in (t[..., :h_q * d], t[..., h_q * d:(h_q + h_kv) * d])]

    q, k = split(gq)
    spare = torch.full_like(gq, 7.0)
    dq, dk = split(spare)
    dw = [torch.full((d,), NAN, device="cuda") if norm else None for _ in range(2)]
    ws = None
    if norm:
        ws = torch.full((attn.attn_norm_rope_bwd_workspace_size(B, n, h_q, h_kv, d),), 255, dtype=torch.uint8,
                        device="cuda")
    call = lambda: attn.attn_norm_rope_bwd(  # noqa: E731
        q, k, g[0].cuda(), g[1].cuda(), dq, dk, ws, dev(table), *map(dev, w), *dw, positions=dev(pos), eps=EPS,
        interleaved=inter)
    call()
    torch.cuda.synchronize()
    first = [t.clone() for t in [spare] + [x for x in dw if x is not None]]
    for x, weight, gr, got, got_w, h in ((q, w[0], g[0], dq, dw[0], h_q), (k, w[1], g[1], dk, dw[1], h_kv)):
        x = x.cpu()
        want = torch.zeros(B, n, h, d, dtype=torch.float64)
        size = torch.zeros_like(want)
        want_w, size_w = torch.zeros(d, dtype=torch.float64), torch.zeros(d, dtype=torch.float64)
        for b in range(B):
            for i in range(n):
                at = i if pos is None else int(pos[b, i])
                if at < 0 or (table is not None and at >= table.shape[0]):
                    continue
                row = None if table is None else table[at]
                want[b, i], size[b, i], a, c = ref.norm_rope_bwd(x[b, i], gr[b, :, i], weight, row, EPS, inter)
                if norm:
                    want_w, size_w = want_w + a, size_w + c
        check(got, want, size)
        if norm:
            err = (got_w.double().cpu() - want_w).abs()
            assert torch.all(err <= (B * n * h * 2.0 ** -24 + 2.0 ** -18) * size_w)
    assert torch.all(spare[..., (h_q + h_kv) * d:] == 7.0)  # what lies between the heads and the stride
    call()  # the same bits again
    torch.cuda.synchronize()
    for a, b in zip(first, [spare] + [x for x in dw if x is not None]):
        assert torch.equal(a, b)


def test_gradients_against_differences():
    """sum(g . o) moves by dx . e along a direction e, and by dw . e: central differences of
    the float64 form, checked against the library's gradients in norm (bf16 rounding of dx:
    2^-8 relative per element, so 2^-8 |dx| |e| in all)."""
    B, n, h, d, step = 1, 12, 3, 64, 1e-4
    qkv, w, table, _ = setup(5, B, n, h, h, d, 64, True, False)
    g = torch.Generator().manual_seed(6)
    x, gr = qkv[..., :h * d].unflatten(-1, (h, d)), rand(g, B, h, n, d)
    direction = torch.randn(B, n, h, d, generator=g, dtype=torch.float64)
    dir_w = torch.randn(d, generator=g, dtype=torch.float64)

    def value(xx, ww):
        rows = [ref.norm_rope(xx[0, i], ww, table[i], EPS, False)[0] * gr[0, :, i].double() for i in range(n)]
        return torch.stack(rows).sum()

    fx = (value(x.double() + step * direction, w[0]) - value(x.double() - step * direction, w[0])) / (2 * step)
    fw = (value(x, w[0].double() + step * dir_w) - value(x, w[0].double() - step * dir_w)) / (2 * step)
    gq = x.contiguous().cuda()
    dq, dk = torch.empty_like(gq), torch.empty_like(gq)
    dw = [torch.empty(d, device="cuda") for _ in range(2)]
    ws = torch.empty(attn.attn_norm_rope_bwd_workspace_size(B, n, h, h, d), dtype=torch.uint8, device="cuda")
    attn.attn_norm_rope_bwd(gq, gq, gr.cuda(), gr.cuda(), dq, dk, ws, table.cuda(), dev(w[0]), dev(w[1]), *dw, eps=EPS)
    torch.cuda.synchronize()
    dx = dq.double().cpu()
    assert abs((dx * direction).sum() - fx) <= 2.0 ** -8 * dx.norm() * direction.norm() + 1e-6 * abs(fx)
    got = (dw[0].double().cpu() * dir_w).sum()
    assert abs(got - fw) <= 1e-5 * dw[0].double().cpu().norm() * dir_w.norm()


def test_zero_rows_and_large_values():
    """A zero row stays zero (eps keeps the root finite), and entries of 2^40, whose squares
    stay within fp32, come out as one."""
    x = torch.zeros(1, 2, 1, 64, dtype=torch.bfloat16, device="cuda")
    x[0, 1] = 2.0 ** 40
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    out = [torch.full((1, 1, 2, 64), NAN, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    attn.attn_norm_rope(x, x, *out, None, w, w)
    torch.cuda.synchronize()
    assert torch.all(out[0][0, 0, 0] == 0) and torch.all(out[0][0, 0, 1] == 1)


# ---------------------------------------------------------------- append
APPEND = [  # tokens per sequence, starts, h_q, h_kv, d, d_rot, norm, interleaved, page, e4m3
    ([1], [0], 1, 1, 64, 64, True, False, 16, False),
    ([1, 1, 1], [0, 15, 16], 8, 8, 64, 64, True, False, 16, False),
    ([5, 1, 37, 64], [0, 63, 3, 64], 8, 2, 128, 128, True, True, 64, False),
    ([9, 30], [2, 0], 4, 4, 64, 32, False, False, 20, True),
    ([17, 3, 50], [0, 100, 31], 16, 2, 128, 64, True, False, 32, True),
    ([4, 2], [0, 5], 6, 3, 128, 0, True, False, 1, False),
    ([40], [7], 0, 5, 64, 64, True, False, 7, True),
]


def pool(g, need, page, h_kv, d, e4m3):
    """A page table over a shuffled pool, and the pool filled with finite bit patterns."""
    total = sum(need) + 2
    order = torch.randperm(total, generator=g)
    table = torch.full((len(need), max(need) + 1), -1, dtype=torch.int32)
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = order[at:at + n].int()
        at += n
    x = torch.randn(total, h_kv, page, d, generator=g)
    return table, x.to(torch.float8_e4m3fn) if e4m3 else x.to(torch.bfloat16)


@pytest.mark.parametrize("toks,starts,h_q,h_kv,d,d_rot,norm,inter,page,e4m3", APPEND)
def test_append(toks, starts, h_q, h_kv, d, d_rot, norm, inter, page, e4m3):
    g = torch.Generator().manual_seed(11)
    need = [-(-(a + b) // page) for a, b in zip(toks, starts)]
    table, kp = pool(g, need, page, h_kv, d, e4m3)
    vp = kp.flip(0).contiguous()
    seq = torch.repeat_interleave(torch.arange(len(toks)), torch.tensor(toks)).int()
    pos = torch.cat([torch.arange(a, a + b) for a, b in zip(starts, toks)]).int()
    # padding tokens and tokens whose place does not exist are skipped whole
    bad_seq = torch.tensor([0, -1, len(toks), 0, len(toks) - 1], dtype=torch.int32)
    bad_pos = torch.tensor([-1, 0, 0, table.shape[1] * page, max(need) * page], dtype=torch.int32)
    seq, pos = torch.cat([seq, bad_seq]), torch.cat([pos, bad_pos])
    T = len(seq)
    qkv = rand(g, T, (h_q + 2 * h_kv) * d + 8, scale=1.7)
    w = [(1 + 0.2 * torch.randn(d, generator=g)).to(torch.bfloat16) if norm else None for _ in range(2)]
    rot = ref.rotation_table(int(pos.max()) + 1, d_rot) if d_rot else None
    scale = [0.01 + 0.05 * torch.rand(h_kv, generator=g) if e4m3 else None for _ in range(2)]
    gq = qkv.cuda()
    parts = gq.split([h_q * d, h_kv * d, h_kv * d, 8], -1)[:3]
    parts = [x.unflatten(-1, (-1, d)) if x.shape[-1] else None for x in parts]
    q_out = torch.full((T, h_q, d), 5.0, dtype=torch.bfloat16, device="cuda") if h_q else None
    gk, gv = kp.cuda(), vp.cuda()
    attn.attn_paged_append(parts[1], parts[2], gk, gv, pos.cuda(), table.cuda(), seq_ids=seq.cuda(), q=parts[0],
                           q_out=q_out, cos_sin=dev(rot), q_weight=dev(w[0]) if h_q else None, k_weight=dev(w[1]),
                           k_scale=dev(scale[0]), v_scale=dev(scale[1]), eps=EPS, interleaved=inter)
    torch.cuda.synchronize()
    parts = [None if x is None else x.cpu() for x in parts]
    touched = torch.zeros(kp.shape[0], page, dtype=torch.bool)
    for x in range(T - len(bad_seq)):
        at, page_id = int(pos[x]), int(table[seq[x], pos[x] // page])
        touched[page_id, at % page] = True
        row = None if rot is None else rot[at]
        if h_q:
            want, size = ref.norm_rope(parts[0][x], w[0], row, EPS, inter)
            check(q_out[x], want, size)
        want, size = ref.norm_rope(parts[1][x], w[1], row, EPS, inter)
        got_k, got_v = gk[page_id, :, at % page].cpu(), gv[page_id, :, at % page].cpu()
        if not e4m3:
            check(got_k, want, size)
            assert torch.equal(got_v, parts[2][x])
        else:
            s = scale[0].double()[:, None]
            y = (want / s).clamp(-448, 448)
            err = (got_k.double() - y).abs()
            step = torch.maximum(2.0 ** -4 * y.abs(), torch.tensor(2.0 ** -10))
            assert torch.all(err <= step + 2 * ref.U_ROPE * size / s)
            exact_v = (parts[2][x].float() / scale[1][:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
            assert torch.equal(got_v.view(torch.int8), exact_v.view(torch.int8))
    if h_q:
        assert torch.all(q_out[T - len(bad_seq):] == 5.0)
    raw = torch.int8 if e4m3 else torch.int16
    for got, before in ((gk, kp), (gv, vp)):
        same = (got.cpu().view(raw) == before.view(raw)).all(-1).all(1)
        assert torch.all(same | touched)


def test_append_keeps_saturation_and_specials():
    """8-bit values saturate at 448 and infinities with them; NaN stays NaN."""
    v = torch.tensor([1e9, -1e9, float("inf"), -float("inf"), NAN, 0.0, -0.0, 448.0] * 8, dtype=torch.bfloat16)
    x = v.view(1, 1, 64).cuda()
    kp = torch.zeros(1, 1, 4, 64, device="cuda").to(torch.float8_e4m3fn)
    vp, one = kp.clone(), torch.ones(1, device="cuda")
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    attn.attn_paged_append(x, x, kp, vp, zero, zero.view(1, 1), k_scale=one, v_scale=one)
    torch.cuda.synchronize()
    want = torch.tensor([448.0, -448.0, 448.0, -448.0, NAN, 0.0, -0.0, 448.0] * 8)
    for got in (kp, vp):
        got = got[0, 0, 0].float().cpu()
        assert torch.equal(got.nan_to_num(7.0), want.nan_to_num(7.0))
        assert torch.equal(torch.signbit(got[::8]), torch.signbit(want[::8]))


def test_refusals():
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
    q, out, rot = z(2, 3, 4, 64), z(2, 4, 3, 64), z(3, 64, dtype=torch.float32)
    attn.attn_norm_rope(q, q, out, out.clone(), rot)
    for bad in (dict(q=q.float()), dict(q=z(2, 3, 4, 96)), dict(q_out=z(2, 3, 4, 64)), dict(cos_sin=rot.double()),
                dict(q_weight=z(32), k_weight=z(64)), dict(positions=z(2, 4, dtype=torch.int32)),
                dict(q=z(2, 3, 4, 128)[..., ::2]), dict(q=z(2, 4, 3, 64).transpose(1, 2))):
        a = dict(q=q, k=q, q_out=out, k_out=out.clone(), cos_sin=rot) | bad
        with pytest.raises(ValueError):
            attn.attn_norm_rope(**a)
    for bad in (dict(cos_sin=z(2, 64, dtype=torch.float32)), dict(q_weight=z(64)), dict(eps=-1.0),
                dict(cos_sin=z(3, 24, dtype=torch.float32))):
        a = dict(q=q, k=q, q_out=out, k_out=out.clone(), cos_sin=rot) | bad
        with pytest.raises(attn.AttnError):
            attn.attn_norm_rope(**a)
