"""Calls over the 4-bit cache that the interface allows beyond the plain ones:
buffers that layers share, other argument types, other launch shapes."""
import numpy as np
import pytest

import q4_reference as ref
from helpers import dev, host_f64
from test_gpu_q4 import SC, make_cache, rand_q

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


def test_block_with_a_million_heads(hs2):
    """2^20 (sequence, KV head) pairs, whose counters pass 2^31 words (the
    workspace is 77 GB): every list holds its one best candidate, whatever the
    workspace held."""
    import torch
    B, H, n, k, w = 64, 1 << 14, 3, 1, 1
    shape = hs2.Shape.make(n, H, H, k_global=k, window=w)
    need = hs2.workspace_size(hs2.OP_BLOCK_DECODE_Q4, shape, B)
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < need + (8 << 30):
        pytest.skip("needs 86 GB of free device memory")
    ws = torch.empty(need // 4, dtype=torch.int32, device="cuda").fill_(100)
    rng = np.random.default_rng(3)
    K, V = np.zeros((2, 128)), rng.standard_normal((2, 128))
    K[0, 0], K[1, 0] = 2.0, -2.0                # the best candidate, every other key
    rec = ref.records(ref.to_bf16_bits(K), ref.to_bf16_bits(V))
    best = torch.randint(0, 2, (B, H), device="cuda", generator=torch.Generator("cuda").manual_seed(4))
    mine = best[..., None] == torch.arange(n, device="cuda")
    cache = torch.where(mine[..., None], dev(rec[0]), dev(rec[1]))
    q = torch.zeros(B, H, 128, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1.0
    o, os_, lse = torch.empty_like(q), torch.empty_like(q), torch.empty(B, H, device="cuda")
    idx = torch.empty(B, H, k + w, dtype=torch.int32, device="cuda")
    hs2.hs2_block_decode_q4([n] * B, q, cache, o, lse, idx, [q], [os_], shape, ws.view(torch.uint8))
    assert hs2.hs2_get_device_status() == hs2.OK
    assert torch.equal(idx[..., 0].long(), best) and (idx[..., 1] == n - 1).all()
    for c in range(2):      # all heads of one order of keys alike, the first one right
        x, xs, l = o[best == c], os_[best == c], lse[best == c]
        assert (x == x[0]).all() and (xs == xs[0]).all() and (l == l[0]).all()
        qh, keys = host_f64(q[0, :1]), rec[[int(t != c) for t in range(n)]]
        ref.check(host_f64(x[:1]), l[:1].double().cpu().numpy(), qh, keys, SC)
        ref.check(host_f64(xs[:1]), ref.attend(qh, keys[[c, 2]], SC)[1], qh, keys[[c, 2]], SC)
    del ws
    torch.cuda.empty_cache()


def test_binding_takes_whole_numbers_of_any_kind(hs2):
    """Lengths and first slots from numpy and torch as well as ints."""
    import torch
    lens, n, H, Hq, k, w = [120, 77], 120, 2, 8, 30, 8
    shape = hs2.Shape.make(n, Hq, H, k_global=k, window=w)
    cache, q = dev(make_cache(lens, n, H, 1)), rand_q(2, Hq, 2)
    ws = torch.empty(hs2.workspace_size(hs2.OP_BLOCK_DECODE_Q4, shape, 2), dtype=torch.uint8, device="cuda")
    outs = []
    for kind in (list, np.array, torch.tensor, lambda x: np.array(x, np.int32), tuple):
        o, lse, os_ = torch.empty_like(q), torch.empty(2, Hq, device="cuda"), torch.empty_like(q)
        idx = torch.empty(2, H, k + w, dtype=torch.int32, device="cuda")
        hs2.hs2_block_decode_q4(kind(lens), q, cache, o, lse, idx, [q], [os_], shape, ws)
        outs.append((o, lse, idx, os_))
    for x in outs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(x, outs[0]))
    rows = torch.randn(3, H, 128, device="cuda").bfloat16()
    for first in (np.int64(100), np.int32(100), torch.tensor(100)):
        c = [torch.zeros_like(cache) for _ in range(2)]
        hs2.hs2_cache_write_q4(rows, rows, None, c[0], shape, first=100)
        hs2.hs2_cache_write_q4(rows, rows, None, c[1], shape, first=first)
        assert c[0].any() and torch.equal(*c)
        back = [torch.empty_like(rows) for _ in range(3)]
        hs2.hs2_cache_read_q4(c[0], None, back[0], back[1], shape, first=first)
        hs2.hs2_cache_read_q4(c[0], None, back[2], back[1], shape, first=100)
        assert torch.equal(back[0], back[2])


def test_binding_refuses_what_is_no_tensor(hs2):
    """A missing or foreign argument is a ValueError, as everywhere in the binding."""
    import torch
    shape = hs2.Shape.make(16, 8, 2, k_global=3, window=1)
    cache = torch.zeros(2, 2, 16, 144, dtype=torch.uint8, device="cuda")
    Kc, S = torch.zeros(2, 16, 2, 128, dtype=torch.uint8, device="cuda"), torch.zeros(2, 16, 2, device="cuda")
    x = torch.zeros(4, 2, 128, dtype=torch.bfloat16, device="cuda")
    q, lse = torch.zeros(2, 8, 128, dtype=torch.bfloat16, device="cuda"), torch.zeros(2, 8, device="cuda")
    n = torch.zeros(2, dtype=torch.int32, device="cuda")
    idx = torch.zeros(2, 2, 4, dtype=torch.int32, device="cuda")
    ws = torch.zeros(1 << 22, dtype=torch.uint8, device="cuda")
    for bad in (lambda: hs2.hs2_cache_write_q4(None, x, None, cache, shape),
                lambda: hs2.hs2_cache_write_q4(x, None, None, cache, shape),
                lambda: hs2.hs2_cache_write_q4(x[0, 0, 0], x, None, cache, shape),
                lambda: hs2.hs2_cache_write_q4(x, x, [0, 1, 2, 3], cache, shape),
                lambda: hs2.hs2_cache_write_q4(x, x, None, None, shape),
                lambda: hs2.hs2_cache_read_q4(cache, None, x, [x], shape),
                lambda: hs2.hs2_cache_write_fp8(x, x, None, Kc, None, S, shape),
                lambda: hs2.hs2_cache_write_fp8(x, x, None, Kc, Kc, None, shape),
                lambda: hs2.hs2_cache_read_fp8(None, Kc, S, S, None, x, x, shape),
                lambda: hs2.hs2_decode_attn_q4([1, 2], q, cache, q, lse, shape, ws),
                lambda: hs2.hs2_decode_attn_q4(n, None, cache, q, lse, shape, ws),
                lambda: hs2.hs2_decode_attn_q4(n, q, cache, q, None, shape, ws),
                lambda: hs2.hs2_sparse_attn_q4(q, cache, None, q, None, shape),
                lambda: hs2.hs2_block_decode_q4([1, 2], q, cache, q, lse, idx, [None], [q], shape, ws),
                lambda: hs2.hs2_block_decode_q4([1, 2], q, cache, q, lse, None, [], [], shape, ws)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(hs2.HS2Error) as e:
        hs2.hs2_decode_attn_q4(n, q, cache, q, lse, shape, None)
    assert e.value.status == hs2.ERR_WORKSPACE


def test_captured_calls_behind_copies_and_joins(hs2):
    """The dependent launches captured behind a copy, a memset, a join of two
    streams and another call, replayed with new contents."""
    import torch
    B, n, H, Hq, k, w = 3, 500, 2, 16, 200, 30
    shape = hs2.Shape.make(n, Hq, H, k_global=k, window=w)
    cache = torch.zeros(B, H, n, 144, dtype=torch.uint8, device="cuda")
    src, q = torch.zeros_like(cache), torch.zeros(B, Hq, 128, dtype=torch.bfloat16, device="cuda")
    idx = torch.zeros(B, H, k + w, dtype=torch.int32, device="cuda")
    idx_src = torch.zeros_like(idx)
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    o = [torch.zeros_like(q) for _ in range(5)]
    lse = [torch.zeros(B, Hq, device="cuda") for _ in range(5)]
    rows = torch.zeros(B, 2 * H, 128, dtype=torch.bfloat16, device="cuda")
    slot = torch.tensor([b * n + 3 for b in range(B)], dtype=torch.int32, device="cuda")
    ws = torch.empty(hs2.workspace_size(hs2.OP_DECODE_ATTN_Q4, shape, B), dtype=torch.uint8, device="cuda")
    main, side = torch.cuda.Stream(), torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=main):
        cache.copy_(src)                                        # behind a copy
        hs2.hs2_decode_attn_q4(lens, q, cache, o[0], lse[0], shape, ws)
        idx.copy_(idx_src)
        hs2.hs2_sparse_attn_q4(q, cache, idx, o[1], lse[1], shape)
        side.wait_stream(main)                                  # two branches that join
        with torch.cuda.stream(side):
            hs2.hs2_cache_write_q4(rows[:, :H], rows[:, H:], slot, cache, shape)
        hs2.hs2_sparse_attn_q4(o[1], src, idx, o[2], lse[2], shape)
        main.wait_stream(side)
        hs2.hs2_sparse_attn_q4(o[2], cache, idx, o[3], lse[3], shape)
        idx.zero_()                                             # behind a memset
        hs2.hs2_sparse_attn_q4(q, cache, idx, o[4], lse[4], shape)
    for step in range(3):
        rec = make_cache([n] * B, n, H, 30 + step)
        src.copy_(dev(rec))
        q.copy_(rand_q(B, Hq, 40 + step))
        rng = np.random.default_rng(step)
        idx_src.copy_(dev(np.stack([rng.permutation(n)[:k + w] for _ in range(B * H)]).astype(np.int32)).view(B, H, -1))
        rows.copy_(rand_q(B, 2 * H, 50 + step))
        lens.copy_(torch.tensor([n - step, step, 1]))
        g.replay()
        torch.cuda.synchronize()
        full = src.clone()
        x, y = torch.empty_like(q), torch.empty(B, Hq, device="cuda")
        hs2.hs2_decode_attn_q4(lens, q, full, x, y, shape, torch.full_like(ws, 255), stream=0)
        assert torch.equal(x, o[0]) and torch.equal(y, lse[0])
        for i, (a, c, at) in enumerate([(q, src, idx_src), (o[1], src, idx_src), (o[2], cache, idx_src),
                                        (q, cache, idx)], 1):
            hs2.hs2_sparse_attn_q4(a, c, at, x, y, shape, stream=torch.cuda.default_stream())
            torch.cuda.synchronize()
            assert torch.equal(x, o[i]) and torch.equal(y, lse[i]), f"call {i}"
        hs2.hs2_cache_write_q4(rows[:, :H], rows[:, H:], slot, full, shape)
        assert torch.equal(full, cache)
    assert hs2.hs2_get_device_status() == hs2.OK
