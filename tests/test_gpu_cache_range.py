"""The largest values of the 4-bit cache, written and read back."""
import numpy as np
import pytest

from helpers import bits, dev_bf16

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hs2():
    import torch
    assert torch.cuda.is_available()
    import long_context_bridge_b200 as m
    return m


def test_largest_values_read_back(hs2):
    """Groups whose largest |x| runs over bf16's last 300 finite values: finite,
    and within half a step of the input, but for 0x7F7F, whose code 7 means
    7 * 146/128 * 2^125 = 1.99609375 * 2^127, half way from 0x7F7F (1.9921875 *
    2^127) to 2^128: infinite to nearest even, by the format's definition."""
    import torch
    top = np.arange(0x7F80 - 300, 0x7F80)
    n = len(top)
    x = np.zeros((n, 1, 128), np.uint16)
    x[:, 0, ::32] = top[:, None]
    x[:, 0, 1::32] = top[:, None] | 0x8000
    x[:, 0, 2::32] = 0x7E00
    shape = hs2.Shape.make(n, 1, 1)
    cache = torch.zeros(1, 1, n, 144, dtype=torch.uint8, device="cuda")
    hs2.hs2_cache_write_q4(dev_bf16(x), dev_bf16(x), None, cache, shape)
    K = torch.zeros(n, 1, 128, dtype=torch.bfloat16, device="cuda")
    V = torch.zeros_like(K)
    hs2.hs2_cache_read_q4(cache, None, K, V, shape)
    value = lambda b: (b.astype(np.uint32) << 16).view(np.float32).astype(np.float64)  # noqa: E731
    want = value(x)
    for got in (bits(K), bits(V)):
        assert np.array_equal(bits(K), got)
        finite = np.isfinite(value(got))
        assert finite[:-1].all()
        # half a step of the codes (amax / 7, its rounding to bf16) and half one of bf16
        step = np.abs(want).max(-1, keepdims=True) / 7 * (1 + 2.0 ** -8)
        assert np.all(np.abs(value(got) - want)[:-1] <= (step / 2 + 2.0 ** -8 * np.abs(want))[:-1])
        assert np.array_equal(~finite[-1, 0], np.isin(np.arange(128) % 32, [0, 1]))
        assert (got[-1, 0, ::32] == 0x7F80).all() and (got[-1, 0, 1::32] == 0xFF80).all()
    assert hs2.hs2_get_device_status() == hs2.OK
