"""The decode step's selection where scores do not spread: ties of more
candidates than a scoring CTA's list holds (1024), within and past the capacity
of the list in memory (8192), and no selection at all."""
import numpy as np
import pytest

import q4_reference as ref
from helpers import dev
from test_gpu_q4 import rand_q

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hs2():
    import torch
    assert torch.cuda.is_available()
    import long_context_bridge_b200 as m
    return m


def step(hs2, fmt, B, H, Hq, n, lens, k, w):
    """One block step over a cache whose records are all the same: idx, o, V row."""
    import torch
    shape = hs2.Shape.make(n, Hq, H, k_global=k, window=w)
    rng = np.random.default_rng(k + n)
    q = rand_q(B, Hq, 3)
    o, lse = torch.empty_like(q), torch.empty(B, Hq, device="cuda")
    idx = torch.full((B, H, k + w), -9, dtype=torch.int32, device="cuda")
    os_ = torch.empty_like(q)
    op = hs2.OP_BLOCK_DECODE if fmt == "fp8" else hs2.OP_BLOCK_DECODE_Q4
    ws = torch.full((hs2.workspace_size(op, shape, B),), 0xFF, dtype=torch.uint8, device="cuda")
    if fmt == "fp8":
        codes = dev(rng.integers(0, 0x60, (2, 128)).astype(np.uint8))
        Kc, Vc = (codes[i].expand(B, n, H, 128).contiguous() for i in range(2))
        S = torch.full((B, n, H), 1 / 64.0, device="cuda")
        v = Vc[0, 0, 0].view(torch.float8_e4m3fn).double() / 64
        hs2.hs2_block_decode(lens, q, Kc, Vc, S, S, o, lse, idx, [q], [os_], shape, ws)
    else:
        rec = ref.records(*(ref.to_bf16_bits(rng.standard_normal((1, 128))) for _ in range(2)))
        cache = dev(rec[0]).expand(B, H, n, 144).contiguous()
        v = dev(ref.values(rec)[1][0])
        hs2.hs2_block_decode_q4(lens, q, cache, o, lse, idx, [q], [os_], shape, ws)
    assert hs2.hs2_get_device_status() == hs2.OK
    # every weight multiplies the same row: half a bf16 step, a rounding of P to
    # f16 and the sums' roundings (n / 16 + 64 of 2^-23) of it
    tol = (2.0 ** -8 + 2.0 ** -11 + (n / 16 + 64) * 2.0 ** -23) * v.abs() + 1e-30
    for x in (o, os_):
        assert ((x.double() - v).abs() <= tol).all()
    return idx.cpu().numpy()


@pytest.mark.parametrize("fmt", ["fp8", "q4"])
@pytest.mark.parametrize("B,H,n,k", [(40, 15, 3000, 100), (64, 10, 1100, 1000), (60, 10, 8100, 7), (60, 10, 9000, 500),
                                     (2, 2, 40000, 64)])
def test_ties_past_a_list(hs2, fmt, B, H, n, k):
    w = 16
    lens = [n - (b % 5) for b in range(B)]
    idx = step(hs2, fmt, B, H, H * 2, n, lens, k, w)
    for b in range(B):
        want = np.r_[np.arange(k), np.arange(lens[b] - w, lens[b])]
        assert np.array_equal(idx[b], np.broadcast_to(want, (H, k + w)))


@pytest.mark.parametrize("fmt", ["fp8", "q4"])
@pytest.mark.parametrize("B,H,n", [(1, 2, 20000), (3, 1, 500), (64, 10, 2000)])
def test_no_selection(hs2, fmt, B, H, n):
    w = 8
    lens = [n - 3 * (b % 7) for b in range(B)]
    idx = step(hs2, fmt, B, H, H * 2, n, lens, 0, w)
    for b in range(B):
        assert np.array_equal(idx[b], np.broadcast_to(np.arange(lens[b] - w, lens[b]), (H, w)))
