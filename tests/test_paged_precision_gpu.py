"""attn_paged_decode where the weights' precision shows: a dominant first token without a value
(the output is the sum of many tiny weights). Against the plain float64 form, in both forms
of the work split."""
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


# 60 x 16 pairs of up to 750 keys: more than half as many pairs as resident warps, up to 24
# tiles each, so that a pair is one warp's from its first key to its last
WHOLE = torch.randint(400, 750, (60,), generator=torch.Generator().manual_seed(70)).tolist()


@pytest.mark.parametrize("lens,h_kv,d,group,e4m3", [
    (WHOLE, 16, 64, 1, True), (WHOLE, 16, 64, 1, False), ([700, 64, 33], 2, 128, 1, True), ([700, 64], 2, 128, 12, True)])
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
