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
