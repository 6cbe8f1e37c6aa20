"""Every launch shape of the operators over the 4-bit cache: sixteen heads in one
pair, the merges of few and of many heads, NaN scales in every operator."""
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


def lists_of(rng, B, H, cap, m):
    """Lists of m entries: any order, holes, some full, some empty."""
    idx = np.full((B, H, m), -1, np.int32)
    for b in range(B):
        for g in range(H):
            n = (0, min(cap, m), int(rng.integers(1, min(cap, m) + 1)))[(b + g) % 3]
            idx[b, g, rng.permutation(m)[:n]] = rng.permutation(cap)[:n]
    return idx


def check_lists(o, lse, q, rec, idx, Hq, H):
    oh, qh, G = host_f64(o), host_f64(q), Hq // H
    for b in range(len(oh)):
        for g in range(H):
            h = slice(g * G, g * G + G)
            keys = rec[b, g, idx[b, g][idx[b, g] >= 0]]
            l = ref.attend(qh[b, h], keys, SC)[1] if lse is None else lse[b, h].double().cpu().numpy()
            ref.check(oh[b, h], l, qh[b, h], keys, SC, f"row {b} head {g}, {len(keys)} entries")


# G = 16 splits its heads over two pairs up to 111 lists; from there clusters of
# two up to 148 lists of at least 256 entries, single CTAs beyond; the other G
# take clusters of 8, 4, 2 and 1
@pytest.mark.parametrize("Hq,H,B,m", [(16, 1, 111, 300), (16, 1, 112, 300), (32, 2, 74, 300), (32, 2, 75, 300),
                                      (16, 1, 120, 255), (16, 1, 130, 256), (32, 2, 100, 64), (16, 1, 150, 700),
                                      (8, 1, 37, 1100), (8, 1, 38, 1100), (8, 1, 111, 600), (8, 1, 112, 600),
                                      (8, 1, 222, 300), (8, 1, 223, 300)])
def test_list_launch_shapes(hs2, Hq, H, B, m):
    import torch
    cap = 400
    rng = np.random.default_rng(B + m)
    rec = make_cache([cap] * B, cap, H, B)
    idx, q = lists_of(rng, B, H, cap, m), rand_q(B, Hq, m)
    shape = hs2.Shape.make(cap, Hq, H, k_global=m - 1, window=1)
    o, lse = torch.full_like(q, 3.0), torch.full((B, Hq), 3.0, device="cuda")
    hs2.hs2_sparse_attn_q4(q, dev(rec), dev(idx), o, lse, shape)
    assert hs2.hs2_get_device_status() == hs2.OK
    check_lists(o, lse, q, rec, idx, Hq, H)


@pytest.mark.parametrize("Hq,H,B,L", [(32, 2, 19, 3), (16, 1, 14, 8), (16, 1, 14, 17), (16, 1, 20, 8)])
def test_block_layers_of_sixteen_heads(hs2, Hq, H, B, L):
    """Layers of a block that together pass the 111 lists of the split."""
    import torch
    n, k, w = 500, 260, 40
    lens = [n - 11 * b for b in range(B)]
    rec, q = make_cache(lens, n, H, B), rand_q(B, Hq, 1)
    shape = hs2.Shape.make(n, Hq, H, k_global=k, window=w)
    ws = torch.empty(hs2.workspace_size(hs2.OP_BLOCK_DECODE_Q4, shape, B), dtype=torch.uint8, device="cuda")
    o, lse = torch.empty_like(q), torch.empty(B, Hq, device="cuda")
    idx = torch.empty(B, H, k + w, dtype=torch.int32, device="cuda")
    qs, os_ = [rand_q(B, Hq, 2 + l) for l in range(L)], [torch.empty_like(q) for _ in range(L)]
    hs2.hs2_block_decode_q4(lens, q, dev(rec), o, lse, idx, qs, os_, shape, ws)
    assert hs2.hs2_get_device_status() == hs2.OK
    lists = idx.cpu().numpy()
    for l in range(L):
        check_lists(os_[l], None, qs[l], rec, lists, Hq, H)


# one long context among short ones, so that its heads have tens to hundreds of
# partials: one head per CTA of 16 warps (up to 148 heads) or of four, four heads
# per CTA from 592 on (G >= 4)
@pytest.mark.parametrize("Hq,H,B", [(8, 2, 3), (32, 4, 7), (16, 1, 12), (2, 1, 90), (16, 16, 10), (16, 2, 40),
                                    (16, 4, 38), (32, 2, 19)])
def test_merge_shapes(hs2, Hq, H, B):
    import torch
    cap, G = 40000, Hq // H
    rng = np.random.default_rng(B)
    long = rng.integers(0, B)
    lens = rng.integers(0, 300, B)
    lens[long] = cap - 7
    if B > 5:
        lens[(long + 1) % B] = 0
    cache = torch.full((B, H, cap, 144), 0xFF, dtype=torch.uint8, device="cuda")
    recs = [make_cache([int(n)], max(int(n), 1), H, b)[0, :, :n] for b, n in enumerate(lens)]
    for b, n in enumerate(lens):
        cache[b, :, :n] = dev(recs[b])
    q = rand_q(B, Hq, 5)
    shape = hs2.Shape.make(cap, Hq, H)
    o, lse = torch.empty_like(q), torch.empty(B, Hq, device="cuda")
    ws = torch.full((hs2.workspace_size(hs2.OP_DECODE_ATTN_Q4, shape, B),), 0xFF, dtype=torch.uint8, device="cuda")
    hs2.hs2_decode_attn_q4(dev(lens.astype(np.int32)), q, cache, o, lse, shape, ws)
    assert hs2.hs2_get_device_status() == hs2.OK
    oh, lh, qh = host_f64(o), lse.double().cpu().numpy(), host_f64(q)
    for b in range(B):
        for g in range(H):
            h = slice(g * G, g * G + G)
            ref.check(oh[b, h], lh[b, h], qh[b, h], recs[b][g], SC, f"seq {b} head {g} len {lens[b]}")


def test_bad_entries_before_rows_that_exist(hs2):
    """A list's entries at and behind the capacity are skipped though records
    follow the cache in memory."""
    import torch
    cap, H, Hq, m = 300, 1, 8, 64
    rec = make_cache([cap + 64], cap + 64, H, 5)
    memory = dev(rec)
    cache = memory.view(-1)[:cap * 144].view(1, H, cap, 144)
    rng = np.random.default_rng(6)
    idx = rng.permutation(cap)[:m].astype(np.int32)[None, None]
    bad = idx.copy()
    bad[..., [3, 40, 63]] = [cap, cap + 63, cap + 1]
    shape = hs2.Shape.make(cap, Hq, H, k_global=m - 1, window=1)
    q = rand_q(1, Hq, 7)
    outs = []
    for x in (np.where(bad < cap, bad, -1), bad):
        o, lse = torch.empty_like(q), torch.empty(1, Hq, device="cuda")
        hs2.hs2_sparse_attn_q4(q, cache, dev(x), o, lse, shape)
        assert hs2.hs2_get_device_status() == (hs2.OK if not outs else hs2.ERR_BAD_INDEX)
        outs.append((o, lse))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    check_lists(*outs[1], q, rec[:, :, :cap], np.where(bad < cap, bad, -1), Hq, H)


@pytest.mark.parametrize("Hq,H", [(16, 2), (32, 2)])
def test_nan_scales_in_lists_and_block(hs2, Hq, H):
    """A K group stored with the scale NaN spoils the heads that attend it, a V
    group its own 32 dims of them, and neither anything else; a list that does
    not name the record is clean, and the lists stay in range."""
    import torch
    n, k, w, G = 400, 64, 16, Hq // H
    rec = make_cache([n, n, n], n, H, 3)
    rec[0, 1, 77, 136 + 2:136 + 4] = [0xC0, 0x7F]      # V group 1 of (0, head 1, token 77)
    rec[1, 0, 5, 128:130] = [0xC0, 0x7F]               # K group 0 of (1, head 0, token 5)
    q, cache = rand_q(3, Hq, 4), dev(rec)
    shape = hs2.Shape.make(n, Hq, H, k_global=k, window=w)

    def lists(named):
        idx = np.random.default_rng(8).permutation(n)[:k + w]
        idx = idx[~np.isin(idx, [5, 77])][:k + w - 4]
        idx = np.concatenate([idx, [5, 77] if named else [-1, -1], np.full(k + w - 2 - len(idx), -1)])
        return np.tile(idx.astype(np.int32), (3, H, 1))

    clean = rec.copy()
    clean[0, 1, 77, 138:140] = 0
    for named in (False, True):
        idx = lists(named)
        o, lse = torch.empty_like(q), torch.empty(3, Hq, device="cuda")
        hs2.hs2_sparse_attn_q4(q, cache, dev(idx), o, lse, shape)
        assert hs2.hs2_get_device_status() == hs2.OK
        oh, lh, qh = host_f64(o), lse.double().cpu().numpy(), host_f64(q)
        for b in range(3):
            for g in range(H):
                h = slice(g * G, g * G + G)
                at = idx[b, g][idx[b, g] >= 0]
                if named and (b, g) == (1, 0):
                    assert np.isnan(oh[b, h]).all() and np.isnan(lh[b, h]).all()
                elif named and (b, g) == (0, 1):
                    assert np.isnan(oh[b, h][:, 32:64]).all()
                    want, _, A, _ = ref.attend(qh[b, h], clean[b, g, at], SC)
                    rest = np.r_[0:32, 64:128]
                    tol = 2.0 ** -8 * np.abs(want) + 2.0 ** -9 * A
                    assert np.all(np.abs(oh[b, h] - want)[:, rest] <= tol[:, rest]) and np.isfinite(lh[b, h]).all()
                else:
                    ref.check(oh[b, h], lh[b, h], qh[b, h], rec[b, g, at], SC)
    # the block: attention, lists and sparse layer of the spoilt heads and of the others
    ws = torch.full((hs2.workspace_size(hs2.OP_BLOCK_DECODE_Q4, shape, 3),), 0xFF, dtype=torch.uint8, device="cuda")
    got = []
    for c in (cache, dev(clean_of(rec))):
        o, os_, lse = torch.empty_like(q), torch.empty_like(q), torch.empty(3, Hq, device="cuda")
        idx = torch.empty(3, H, k + w, dtype=torch.int32, device="cuda")
        hs2.hs2_block_decode_q4([n] * 3, q, c, o, lse, idx, [q], [os_], shape, ws)
        assert hs2.hs2_get_device_status() == hs2.OK
        got.append((host_f64(o), lse.cpu().numpy(), idx.cpu().numpy(), host_f64(os_)))
    (o, lse, idx, os_), plain = got
    assert np.all(np.diff(idx[..., :k]) > 0) and idx.min() >= 0 and idx[..., :k].max() < n - w
    assert np.array_equal(idx[..., k:], np.broadcast_to(np.arange(n - w, n), idx[..., k:].shape))
    for b in range(3):
        for g in range(H):
            h = slice(g * G, g * G + G)
            if (b, g) == (1, 0):
                assert np.isnan(o[b, h]).all() and np.isnan(lse[b, h]).all()
                continue
            assert np.array_equal(idx[b, g], plain[2][b, g]) and np.array_equal(lse[b, h], plain[1][b, h])
            spoilt = (b, g) == (0, 1)
            assert np.isnan(o[b, h][:, 32:64]).all() if spoilt else np.array_equal(o[b, h], plain[0][b, h])
            listed = spoilt and 77 in idx[b, g]
            assert np.isnan(os_[b, h][:, 32:64]).all() if listed else np.array_equal(os_[b, h], plain[3][b, h])


def clean_of(rec):
    """The records with every NaN scale replaced by 1."""
    s = rec.copy()
    v = s[..., 128:].view(np.uint16)
    v[v == 0x7FC0] = 0x3F80
    return s
