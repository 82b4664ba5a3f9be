"""attn_paged_decode where the weights' precision shows: a dominant first token without a value
(the output is the sum of many tiny weights), and values that cancel. Against the plain
float64 form, in both forms of the work split."""
import math

import pytest
import torch

import paged_reference as ref
from test_paged_gpu import check, make, run
from transformer_scaled_dot_mha_gb300 import attn

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    attn.lib()


# 60 x 16 pairs of up to 750 keys: more than half as many pairs as resident warps, up to 24
# tiles each, so that a pair is one warp's from its first key to its last
WHOLE = torch.randint(400, 750, (60,), generator=torch.Generator().manual_seed(70)).tolist()


@pytest.mark.parametrize("lens,h_kv,d,group,e4m3", [
    (WHOLE, 16, 64, 1, True), (WHOLE, 16, 64, 1, False), ([700, 64, 33], 2, 128, 1, True),
    ([700, 64], 2, 128, 12, True)])
@pytest.mark.parametrize("first", [1.5, 2.0, 2.25])
def test_dominant_first_token_without_a_value(lens, h_kv, d, group, e4m3, first):
    """The first key scores 12, 16 or 18 above the others' mean and its value is zero: the other
    weights are 2^-16 to 2^-26 of it (the others' scores spread by 0.6), and the output is
    their sum alone."""
    q, kp, vp, table, ln, _ = make(71, lens, 1, group * h_kv, h_kv, d, 64, False)
    one = torch.ones(h_kv) if e4m3 else None
    q.fill_(1.0)
    raw_k, raw_v = kp.float() * (0.577 * (64 / d) ** 0.5), vp.float()
    for b in range(len(lens)):
        raw_k[table[b, 0], :, 0] = first * 64 / d  # the score: first * 64 / 8
        raw_v[table[b, 0], :, 0] = 0
    kind = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    kp, vp = raw_k.to(kind), raw_v.to(kind)
    got = run(q, kp, vp, table, ln, [one, one], 0.125)
    check(*got, *ref.paged_decode(q, kp, vp, table, ln, 0.125, -1, 0, one, one))


@pytest.mark.parametrize("lens,h_kv,d,group,e4m3", [
    ([300, 17, 700], 2, 64, 1, False), ([300, 700], 2, 128, 1, False), ([300, 700], 2, 64, 16, False),
    ([300, 700], 2, 128, 16, False), (WHOLE, 16, 64, 1, False), ([300, 17, 700], 2, 64, 1, True),
    ([300, 700], 2, 128, 1, True), ([300, 700], 2, 64, 16, True), ([300, 700], 2, 128, 16, True)])
def test_weights_keep_their_precision(lens, h_kv, d, group, e4m3):
    """Value j is +-1 / (n p_j), rounded to its type: the terms p_j v_j cancel up to that
    rounding, so an error of the weights is as large as the output itself (bf16 pages) or
    a good part of it (e4m3).

    Queries are 0, +-1/2 and keys multiples of 1/8 below 2: products and sums of a score are
    exact in fp32. What remains: the factor scale log2(e) and its product (2^-23 of the score,
    in log2 units below 7, eight standard deviations: 2^-20), the exponential, its argument and
    the sums (2^-20 together): weights within 2^-18 of themselves, one way for all at the
    worst; the second product takes them in two bf16 parts (2^-15; e4m3 pages: rounded to f16,
    2^-11), independently; the output is rounded once (u / 2 in root mean square)."""
    g = torch.Generator().manual_seed(72)
    q, kp, vp, table, ln, _ = make(73, lens, 1, group * h_kv, h_kv, d, 64, False)
    B, one = len(lens), torch.ones(h_kv) if e4m3 else None
    scale = 0.125
    per_head = torch.randint(-1, 2, (B, 1, h_kv, 1, d), generator=g).float() / 2
    q = per_head.expand(B, 1, h_kv, group, d).reshape(q.shape).bfloat16()
    kind = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    raw_k, raw_v = (kp.float() * 8).round().clamp(-15, 15) / 8, vp.float()
    for b, n in enumerate(lens):
        keys = torch.arange(n)
        pages = table[b].long()[keys // 64]
        s = scale * torch.einsum("nhd,hd->nh", raw_k[pages, :, keys % 64].double(), per_head[b, 0, :, 0].double())
        p = torch.softmax(s, 0)
        sign = torch.where(torch.rand(n, h_kv, d, generator=g) < 0.5, -1.0, 1.0)
        sign[1::2] = -sign[:n // 2 * 2:2]  # in pairs
        raw_v[pages, :, keys % 64] = (sign / (n * p[..., None])).float()
    kp, vp = raw_k.to(kind), raw_v.to(kind)
    assert torch.equal(kp.float().nan_to_num(0), raw_k.nan_to_num(0))
    out, lse = run(q, kp, vp, table, ln, [one, one], scale)
    want, want_lse, _, lb = ref.paged_decode(q, kp, vp, table, ln, scale, -1, 0, one, one)
    assert torch.all((lse.double() - want_lse).abs() <= lb)
    for b, n in enumerate(lens):
        keys = torch.arange(n)
        pages = table[b].long()[keys // 64]
        k, v = (x.float()[pages, :, keys % 64].double() for x in (kp, vp))
        p = torch.softmax(scale * torch.einsum("nhd,hd->nh", k, per_head[b, 0, :, 0].double()), 0)[..., None]
        all_ways, each_way = (p * v.abs()).sum(0), (p * v).square().sum(0).sqrt()
        w = want[b, 0].view(h_kv, group, d)
        fixed = (2.0 ** -18 * all_ways) ** 2 + ((ref.U_F16 if e4m3 else 2.0 ** -15) * each_way) ** 2
        bound = ((ref.U_BF16 / 2 * w) ** 2 + fixed[:, None]).sqrt()
        err = (out[b, 0].double().view(h_kv, group, d) - w).abs()
        assert err.norm() <= bound.norm(), f"{(err.norm() / bound.norm()).item():.2f} of the bound"


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens", [[1, 40, 70], [900, 1300]])
def test_infinite_values_stay_infinite(d, lens):
    """A visible infinity, among weights of exactly one too, gives an infinity of its sign, and
    NaN only where both signs meet; the other columns stay as they are."""
    q, kp, vp, table, ln, sc = make(74, lens, 1, 4, 2, d, 16)
    for b, n in enumerate(lens):
        for at in {0, n // 2, n - 1}:
            vp[table[b, at // 16], 0, at % 16, 3] = INF
            vp[table[b, at // 16], 1, at % 16, 5] = -INF
        vp[table[b, 0], 0, 0, d - 1] = INF
        vp[table[b, (n - 1) // 16], 0, (n - 1) % 16, d - 1] = -INF
    got = run(q, kp, vp, table, ln, sc)
    want = ref.paged_decode(q, kp, vp, table, ln, 1 / math.sqrt(d))
    inf = torch.isinf(want[0])
    assert inf.any() and torch.equal(got[0].double()[inf], want[0][inf])
    check(*got, *want)
