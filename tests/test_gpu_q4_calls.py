"""Calls over the 4-bit cache that the interface allows beyond the plain ones:
buffers that layers share, other argument types, other launch shapes."""
import pytest

from helpers import dev
from test_gpu_q4 import make_cache, rand_q

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hs2():
    import torch
    assert torch.cuda.is_available()
    import long_context_bridge_b200 as m
    return m


@pytest.mark.parametrize("B,Hq,H,k", [(2, 8, 1, 200), (6, 32, 4, 200), (40, 16, 1, 200), (2, 8, 1, 1100)])
def test_block_layers_that_share_buffers(hs2, B, Hq, H, k):
    """Layers chained through their buffers, and buffers written again, give
    what one call per layer in order gives."""
    import torch
    w, n = 30, k + 700
    lens = [n - 7 * b for b in range(B)]
    shape = hs2.Shape.make(n, Hq, H, k_global=k, window=w)
    cache, q = dev(make_cache(lens, n, H, 1)), rand_q(B, Hq, 2)
    ws = torch.empty(hs2.workspace_size(hs2.OP_BLOCK_DECODE_Q4, shape, B), dtype=torch.uint8, device="cuda")
    idx = torch.empty(B, H, k + w, dtype=torch.int32, device="cuda")
    o, lse = torch.empty_like(q), torch.empty(B, Hq, device="cuda")
    # names of the layers' queries and outputs; buffers a .. e, f holds o_full's values
    runs = {"chain": ["ab", "bc", "cd", "de"], "same output": ["ab", "cb", "db"],
            "overwritten queries": ["ab", "ca", "db"], "in place": ["aa", "aa", "aa"],
            "queries from o_full": ["fa", "ab"], "apart": ["ab", "cd"],
            "chain of ten": ["ab", "ba"] * 5}
    for what, layers in runs.items():
        outs = []
        for alone in (False, True):
            buf = {c: rand_q(B, Hq, 10 + i) for i, c in enumerate("abcde")} | {"f": o}
            if not alone:
                hs2.hs2_block_decode_q4(lens, q, cache, o, lse, idx, [buf[x[0]] for x in layers],
                                        [buf[x[1]] for x in layers], shape, ws)
            else:
                for x in layers:
                    hs2.hs2_sparse_attn_q4(buf[x[0]], cache, idx, buf[x[1]], None, shape)
            outs.append({c: t.clone() for c, t in buf.items()})
        for c in outs[0]:
            assert torch.equal(outs[0][c], outs[1][c]), f"{what}: buffer {c}"
    # queries that begin in the middle of the layer before's output
    buf, want = (torch.cat([rand_q(B, Hq, 20), rand_q(B, Hq, 21)]) for _ in range(2))
    half, q0, last, o1 = B // 2, rand_q(B, Hq, 22), torch.empty_like(o), torch.empty_like(o)
    hs2.hs2_block_decode_q4(lens, q, cache, o, lse, idx, [q0, buf[half:half + B]], [buf[:B], last], shape, ws)
    hs2.hs2_sparse_attn_q4(q0, cache, idx, want[:B], None, shape)
    hs2.hs2_sparse_attn_q4(want[half:half + B], cache, idx, o1, None, shape)
    assert torch.equal(buf, want) and torch.equal(last, o1)
    assert hs2.hs2_get_device_status() == hs2.OK
