"""The merge of the ranks' selection records (hs2_decode_cp_sparse) when the
records repeat: a caller that gathers one rank's records twice, or records that
were never filled."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hs2():
    import torch
    assert torch.cuda.is_available()
    import long_context_bridge_b200 as m
    return m


@pytest.mark.parametrize("R,k", [(2, 7), (4, 2048), (8, 1000), (2, 1), (1, 300)])
@pytest.mark.parametrize("same", ["all one entry", "zeros", "a rank's records twice"])
def test_repeated_records_stay_in_bounds(hs2, R, k, same):
    """The k best records come out, repeats among them, ascending, then the window."""
    import torch
    B, H, Hq, w, n = 2, 2, 4, 5, 4000
    rng = np.random.default_rng(k)
    rec = np.zeros((R, B, H, k, 2), np.uint32)
    if same == "all one entry":
        rec[..., 0], rec[..., 1] = np.float32(0.25).view(np.uint32), 5
    elif same != "zeros":
        for b in range(B):
            for g in range(H):
                at = rng.permutation(n - w)[:k]
                rec[:, b, g, :, 0] = rng.random(k).astype(np.float32).view(np.uint32)
                rec[:, b, g, :, 1] = at
    shape = hs2.Shape.make(n, Hq, H, k_global=k, window=w)
    Kc = torch.zeros(B, n, H, 128, dtype=torch.uint8, device="cuda")
    S = torch.ones(B, n, H, device="cuda")
    # idx between guards
    buf = torch.full((B * H * (k + w) + 64,), -77, dtype=torch.int32, device="cuda")
    idx = buf[32:-32].view(B, H, k + w)
    recs = torch.from_numpy(rec.view(np.int32)).cuda()
    hs2.hs2_decode_cp_sparse([n] * B, [0] * B, [n] * B, R, recs, idx, Kc, Kc, S, S, [], None, shape)
    assert hs2.hs2_get_device_status() == hs2.OK
    got = idx.cpu().numpy()
    assert (buf[:32] == -77).all() and (buf[-32:] == -77).all()
    for b in range(B):
        for g in range(H):
            assert np.array_equal(got[b, g, k:], np.arange(n - w, n))
            # the k best of all records, the higher score first, then the smaller position
            r = rec[:, b, g].reshape(-1, 2).astype(np.int64)
            best = r[np.lexsort((r[:, 1], -r[:, 0]))][:k, 1]
            assert np.array_equal(got[b, g, :k], np.sort(best))
