"""The binding's argument handling for norm + rotation and the paged cache, as far as it goes
without a GPU."""
import pytest
import torch

from transformer_scaled_dot_mha_gb300 import attn


def zeros(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


def test_host_tensors_are_refused_as_values():
    """As by every other entry point: a ValueError, with or without a GPU in the machine."""
    i32 = torch.int32
    x, out, rows, pages = zeros(1, 2, 1, 64), zeros(1, 1, 2, 64), zeros(2, 1, 64), zeros(1, 1, 16, 64)
    calls = [
        lambda: attn.attn_norm_rope(x, x, out, out, None),
        lambda: attn.attn_norm_rope_bwd(x, x, out, out, x, x, None, None),
        lambda: attn.attn_paged_append(rows, rows, pages, pages, zeros(2, dtype=i32), zeros(2, 1, dtype=i32)),
        lambda: attn.attn_paged_decode(x, pages, pages, x, zeros(1, 1, dtype=i32), zeros(1, dtype=i32), x),
    ]
    for call in calls:
        with pytest.raises(ValueError, match="CUDA"):
            call()


@pytest.mark.parametrize("short_ways", [True, False])
def test_current_device_and_stream_with_and_without_private_names(monkeypatch, short_ways):
    """Every entry point asks for the current stream: it has to be found by public names too."""
    for name, short in (("_cuda_getDevice", lambda: 3), ("_cuda_getCurrentRawStream", lambda dev: 70 + dev)):
        if short_ways:
            monkeypatch.setattr(torch._C, name, short, raising=False)
        else:
            monkeypatch.delattr(torch._C, name, raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev=None: type("S", (), {"cuda_stream": 70 + dev}))
    device, stream = attn._short_ways()
    assert device() == 3 and stream(2) == 72
    monkeypatch.setattr(attn, "_current_device", device)
    monkeypatch.setattr(attn, "_current_stream", stream)
    assert attn._stream_handle(None) == 73
    assert attn._raw_stream(None, 2) == 72
    assert attn._raw_stream(5, 2) == attn._stream_handle(5) == 5


def test_numbers_beyond_a_c_int_keep_their_side():
    """A window of 2^32 + 1 once became 1, one of 2^32 0, and -2^32 - 1 became -1 (no window)."""
    for x, want in ((2 ** 32 + 1, 2 ** 31 - 1), (2 ** 63, 2 ** 31 - 1), (2 ** 31 - 1, 2 ** 31 - 1),
                    (-2 ** 32 - 1, 1 - 2 ** 31), (-1, -1), (0, 0), (1023, 1023)):
        assert attn._int32(x) == want
