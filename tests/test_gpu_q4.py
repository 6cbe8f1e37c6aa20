"""The operators over the 4-bit cache on the GPU against numpy in 64 bits
(bounds derived in q4_reference.check): attention of a decode step, sparse
layers over lists, and a run of them together."""
import math

import numpy as np
import pytest

import q4_reference as ref
from helpers import bits, dev, dev_bf16, host_f64

pytestmark = pytest.mark.gpu
SC = 1 / math.sqrt(128)


@pytest.fixture(scope="module")
def hs2():
    import torch
    assert torch.cuda.is_available()
    import long_context_bridge_b200 as m
    return m


def make_cache(lens, cap, H, seed, kmul=1.0, vmul=None):
    """Host records [B, H, cap, 144]; 0xFF (NaN scales) behind each length."""
    rng = np.random.default_rng(seed)
    rec = np.full((len(lens), H, cap, 144), 0xFF, np.uint8)
    for b, n in enumerate(lens):
        K = rng.standard_normal((H, n, 128)) * kmul
        V = rng.standard_normal((H, n, 128))
        if vmul is not None:
            V = V * vmul(rng, (H, n, 1))
        rec[b, :, :n] = ref.records(ref.to_bf16_bits(K), ref.to_bf16_bits(V))
    return rec


def run_attn(hs2, rec, lens, Hq, q, seq_len=None, scale=None, ws=None):
    import torch
    B, H, cap, _ = rec.shape
    shape = hs2.Shape.make(cap, Hq, H, scale=scale)
    o = torch.full((B, Hq, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B, Hq), 3.0, device="cuda")
    if ws is None:  # a workspace full of NaN: nothing in it may be read before it is written
        ws = torch.full((hs2.workspace_size(hs2.OP_DECODE_ATTN_Q4, shape, B),), 0xFF,
                        dtype=torch.uint8, device="cuda")
    n = dev(np.asarray(lens if seq_len is None else seq_len, np.int32))
    hs2.hs2_decode_attn_q4(n, q, dev(rec) if isinstance(rec, np.ndarray) else rec, o, lse, shape, ws)
    return o, lse


def check_attn(o, lse, q, rec, lens, Hq, what="", scale=SC):
    o, lse, qh = host_f64(o), lse.cpu().numpy().astype(np.float64), host_f64(q)
    H = rec.shape[1]
    G = Hq // H
    for b, n in enumerate(lens):
        for g in range(H):
            h = slice(g * G, g * G + G)
            ref.check(o[b, h], lse[b, h], qh[b, h], rec[b, g, :n], scale, f"{what} seq {b} head {g} len {n}")


def rand_q(B, Hq, seed, mul=1.0):
    rng = np.random.default_rng(seed)
    return dev_bf16(ref.to_bf16_bits(rng.standard_normal((B, Hq, 128)) * mul))


LENS = [[1], [0], [5, 0, 1, 16, 17], [31, 32, 33, 64, 65], [127, 128, 129, 0, 255, 256, 257],
        [700, 3, 1000], [4000, 0, 0, 1]]


@pytest.mark.parametrize("Hq,H", [(1, 1), (4, 2), (4, 1), (16, 2), (16, 1), (8, 8)])
@pytest.mark.parametrize("lens", LENS)
def test_attention_lengths(hs2, Hq, H, lens):
    cap = max(max(lens), 1) + (len(lens) % 3)
    rec = make_cache(lens, cap, H, 11)
    q = rand_q(len(lens), Hq, 12)
    o, lse = run_attn(hs2, rec, lens, Hq, q)
    check_attn(o, lse, q, rec, lens, Hq)
    assert hs2.hs2_get_device_status() == hs2.OK


def test_attention_many_ragged_sequences(hs2):
    """More sequences than threads of a CTA, most of them short or idle."""
    rng = np.random.default_rng(3)
    lens = rng.integers(0, 90, 300).tolist()
    lens[7] = 0
    lens[299] = 0
    lens[150] = 90
    rec = make_cache(lens, 90, 2, 21)
    q = rand_q(300, 8, 22)
    o, lse = run_attn(hs2, rec, lens, 8, q)
    check_attn(o, lse, q, rec, lens, 8)


def test_attention_largest_batch_and_workspace_bounds(hs2):
    """512 sequences, a third of them idle, then all of them; nothing is written
    behind a workspace of exactly the size asked for."""
    import torch
    rng = np.random.default_rng(4)
    lens = np.where(rng.random(512) < 0.33, 0, rng.integers(1, 50, 512)).tolist()
    rec = make_cache(lens, 50, 1, 23)
    q = rand_q(512, 4, 24)
    need = hs2.workspace_size(hs2.OP_DECODE_ATTN_Q4, hs2.Shape.make(50, 4, 1), 512)
    buf = torch.full((need + 4096,), 0xAB, dtype=torch.uint8, device="cuda")
    o, lse = run_attn(hs2, rec, lens, 4, q, ws=buf[:need])
    check_attn(o, lse, q, rec, lens, 4)
    o, lse = run_attn(hs2, rec, [0] * 512, 4, q, ws=buf[:need])
    assert not o.any() and torch.isneginf(lse).all()
    assert (buf[need:] == 0xAB).all()
    assert hs2.hs2_get_device_status() == hs2.OK


@pytest.mark.parametrize("Hq,H", [(8, 1), (16, 1)])
def test_attention_long_context(hs2, Hq, H):
    lens = [70001, 333]
    rec = make_cache(lens, 70016, H, 31)
    q = rand_q(2, Hq, 32)
    o, lse = run_attn(hs2, rec, lens, Hq, q)
    check_attn(o, lse, q, rec, lens, Hq)


@pytest.mark.parametrize("qmul,kmul,scale", [(1e-3, 1, None), (30, 3, None), (1e5, 1e-5, None),
                                             (1e-30, 1e28, None), (1, 1, 4.0), (6, 2, 1.0),
                                             (300, 300, 1.0), (1e30, 1e-30, None)])
def test_attention_magnitudes(hs2, qmul, kmul, scale):
    """Flat to one-hot softmax (logits up to thousands), large and small q and K."""
    lens = [515, 40]
    rec = make_cache(lens, 515, 2, 41, kmul=kmul)
    q = rand_q(2, 8, 42, mul=qmul)
    o, lse = run_attn(hs2, rec, lens, 8, q, scale=scale)
    check_attn(o, lse, q, rec, lens, 8, scale=SC if scale is None else np.float64(np.float32(scale)))


def test_attention_rising_logits_and_v_scales(hs2):
    """Keys whose logits grow along the context move the reference again and
    again; V rows of very different magnitude move the scale's reference."""
    n, H, Hq = 900, 1, 8
    rng = np.random.default_rng(51)
    u = rng.standard_normal(128)
    K = np.linspace(0, 6, n)[None, :, None] * u + 0.1 * rng.standard_normal((H, n, 128))
    V = rng.standard_normal((H, n, 128)) * np.exp2(rng.integers(-40, 60, (H, n, 1)))
    rec = ref.records(ref.to_bf16_bits(K), ref.to_bf16_bits(V))[None]
    q = dev_bf16(ref.to_bf16_bits((u + 0.3 * rng.standard_normal((1, Hq, 128)))))
    o, lse = run_attn(hs2, rec, [n], Hq, q)
    check_attn(o, lse, q, rec, [n], Hq)
    # per group of dims: one group 2^20 above the others
    V = rng.standard_normal((H, n, 128))
    V[:, :, 32:64] *= 2.0 ** 20
    rec = ref.records(ref.to_bf16_bits(K), ref.to_bf16_bits(V))[None]
    o, lse = run_attn(hs2, rec, [n], Hq, q)
    check_attn(o, lse, q, rec, [n], Hq)


@pytest.mark.parametrize("mul", [1e-35, 1e30, 2e37])
def test_attention_v_over_the_whole_bf16_range(hs2, mul):
    """V near the ends of bf16: sums of many tokens stay within V's range."""
    lens = [3000, 17]
    rec = make_cache(lens, 3000, 1, 55, vmul=lambda rng, s: mul)
    q = rand_q(2, 8, 56)
    o, lse = run_attn(hs2, rec, lens, 8, q)
    check_attn(o, lse, q, rec, lens, 8)


def test_attention_heads_with_zero_or_mixed_queries(hs2):
    lens = [200]
    rec = make_cache(lens, 200, 1, 61)
    rng = np.random.default_rng(62)
    x = rng.standard_normal((1, 8, 128))
    x[0, 2] = 0
    x[0, 3, 5:] = 0
    x[0, 4] *= np.exp2(rng.integers(-26, 1, 128))     # one head over 26 binades
    q = dev_bf16(ref.to_bf16_bits(x))
    o, lse = run_attn(hs2, rec, lens, 8, q)
    check_attn(o, lse, q, rec, lens, 8)


def test_attention_nan_in_context_stays_in_its_group(hs2):
    """A V group stored with the scale NaN spoils its own 32 dims of that head
    and nothing else; a K group with the scale NaN the whole head."""
    lens, H, Hq = [150, 150], 2, 8
    rec = make_cache(lens, 150, H, 71)
    rec[0, 1, 77, 136 + 2:136 + 4] = [0xC0, 0x7F]      # V group 1 of (0, head 1, token 77)
    rec[1, 0, 3, 128:130] = [0xC0, 0x7F]               # K group 0 of (1, head 0, token 3)
    q = rand_q(2, Hq, 72)
    o, lse = run_attn(hs2, rec, lens, Hq, q)
    o, lse, qh = host_f64(o), lse.cpu().numpy(), host_f64(q)
    assert np.isnan(o[0, 4:, 32:64]).all() and np.isfinite(o[0, 4:, :32]).all()
    assert np.isfinite(o[0, 4:, 64:]).all() and np.isfinite(lse[0]).all()
    assert np.isnan(o[1, :4]).all() and np.isnan(lse[1, :4]).all()
    clean = rec.copy()
    clean[0, 1, 77, 138:140] = 0
    for b, g in ((0, 0), (1, 1)):
        ref.check(o[b, 4 * g:4 * g + 4], lse[b, 4 * g:4 * g + 4], qh[b, 4 * g:4 * g + 4], rec[b, g], SC)
    want = ref.attend(qh[0, 4:], clean[0, 1], SC)[0]
    assert np.abs(o[0, 4:, :32] - want[:, :32]).max() <= 2.0 ** -8 * np.abs(want).max() + 2e-3


def test_attention_bad_lengths_are_clamped_and_reported(hs2):
    lens = [20, 0, 40]
    rec = make_cache([40, 40, 40], 40, 1, 81)
    q = rand_q(3, 8, 82)
    a = run_attn(hs2, rec, lens, 8, q)
    assert hs2.hs2_get_device_status() == hs2.OK
    b = run_attn(hs2, rec, lens, 8, q, seq_len=[20, -3, 41])
    assert hs2.hs2_get_device_status() == hs2.ERR_BAD_INDEX
    assert hs2.hs2_get_device_status() == hs2.OK
    import torch
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_attention_past_four_gigabytes(hs2):
    """Records whose offsets pass 2^32 bytes, in the last sequence."""
    import torch
    B, H, cap, n = 8, 4, 1 << 20, 300
    cache = torch.empty(B, H, cap, 144, dtype=torch.uint8, device="cuda")
    rec = make_cache([n], n, H, 91)
    cache[B - 1, :, :n] = dev(rec[0])
    q = rand_q(B, 16, 92)
    lens = [0] * (B - 1) + [n]
    o, lse = run_attn(hs2, cache, lens, 16, q)
    full = np.zeros((B, H, n, 144), np.uint8)
    full[B - 1] = rec[0]
    check_attn(o, lse, q, full, lens, 16)
    # rows at the far end, written, read back and attended through a list
    shape = hs2.Shape.make(cap, 16, H, k_global=2, window=1)
    rng = np.random.default_rng(93)
    Kb, Vb = (ref.to_bf16_bits(rng.standard_normal((3, H, 128))) for _ in range(2))
    slot = dev(np.array([B * cap - 1, B * cap - 3, 7 * cap - 1], np.int32))
    hs2.hs2_cache_write_q4(dev_bf16(Kb), dev_bf16(Vb), slot, cache, shape)
    Ko = torch.zeros(3, H, 128, dtype=torch.bfloat16, device="cuda")
    Vo = torch.zeros_like(Ko)
    hs2.hs2_cache_read_q4(cache, slot, Ko, Vo, shape)
    r = ref.records(Kb, Vb)
    assert np.array_equal(bits(Ko), ref.to_bf16_bits(ref.values(r)[0]))
    assert np.array_equal(bits(Vo), ref.to_bf16_bits(ref.values(r)[1]))
    idx = torch.full((B, H, 3), -1, dtype=torch.int32, device="cuda")
    idx[B - 1] = torch.tensor([cap - 3, -1, cap - 1], dtype=torch.int32)
    idx[6, :, 0] = cap - 1
    o2 = torch.empty_like(o)
    l2 = torch.empty_like(lse)
    hs2.hs2_sparse_attn_q4(q, cache, idx, o2, l2, shape)
    qh, oh, lh = host_f64(q), host_f64(o2), l2.cpu().numpy()
    for g in range(H):
        h = slice(4 * g, 4 * g + 4)
        ref.check(oh[B - 1, h], lh[B - 1, h], qh[B - 1, h], r[[1, 0], g], SC)
        ref.check(oh[6, h], lh[6, h], qh[6, h], r[[2], g], SC)
        ref.check(oh[0, h], lh[0, h], qh[0, h], r[:0, g], SC)


def test_attention_graphs_that_share_a_workspace(hs2):
    """Two captured steps over one workspace replay in turn, each with the
    lengths of the moment, and equal eager calls bit for bit."""
    import torch
    lens, H, Hq, cap = [300, 41, 0], 2, 16, 700
    recs = [make_cache([700] * 3, cap, H, 100 + i) for i in range(2)]
    qs = [rand_q(3, Hq, 102 + i) for i in range(2)]
    caches = [dev(r) for r in recs]
    shape = hs2.Shape.make(cap, Hq, H)
    ws = torch.empty(hs2.workspace_size(hs2.OP_DECODE_ATTN_Q4, shape, 3), dtype=torch.uint8, device="cuda")
    n = dev(np.array(lens, np.int32))
    out = [(torch.empty(3, Hq, 128, dtype=torch.bfloat16, device="cuda"),
            torch.empty(3, Hq, device="cuda")) for _ in range(2)]
    graphs = []
    torch.cuda.synchronize()
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            hs2.hs2_decode_attn_q4(n, qs[i], caches[i], out[i][0], out[i][1], shape, ws)
        graphs.append(g)
    for step in ([300, 41, 0], [1, 700, 129], [0, 0, 5]):
        n.copy_(dev(np.array(step, np.int32)))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for i in range(2):
            check_attn(out[i][0], out[i][1], qs[i], recs[i], step, Hq)
            o, lse = run_attn(hs2, caches[i], step, Hq, qs[i])
            assert torch.equal(o, out[i][0]) and torch.equal(lse, out[i][1])
    # calls on two streams, each with a workspace of its own
    st = [torch.cuda.Stream() for _ in range(2)]
    wss = [torch.empty_like(ws) for _ in range(2)]
    torch.cuda.synchronize()
    for rep in range(5):
        for i in range(2):
            hs2.hs2_decode_attn_q4(n, qs[i], caches[i], out[i][0], out[i][1], shape, wss[i], stream=st[i])
    torch.cuda.synchronize()
    for i in range(2):
        check_attn(out[i][0], out[i][1], qs[i], recs[i], [0, 0, 5], Hq)


# ---------------------------------------------------------------------------
# sparse layers
# ---------------------------------------------------------------------------
def run_sparse(hs2, rec, idx, Hq, q, k, w, lse=True):
    import torch
    B, H, cap, _ = rec.shape
    shape = hs2.Shape.make(cap, Hq, H, k_global=k, window=w)
    o = torch.full((B, Hq, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    ls = torch.full((B, Hq), 3.0, device="cuda") if lse else None
    hs2.hs2_sparse_attn_q4(q, dev(rec), dev(idx.astype(np.int32)), o, ls, shape)
    return o, ls


@pytest.mark.parametrize("Hq,H", [(2, 2), (4, 2), (4, 1), (16, 2), (32, 2)])
@pytest.mark.parametrize("B,cap,k,w", [(1, 1, 0, 1), (3, 40, 5, 2), (2, 300, 64, 16), (5, 1500, 1024, 128),
                                       (2, 5000, 2048, 2048), (40, 600, 100, 33)])
def test_sparse_lists(hs2, Hq, H, B, cap, k, w):
    """Lists with holes anywhere, in any order, short contexts, empty rows."""
    rng = np.random.default_rng(cap + k)
    rec = make_cache([cap] * B, cap, H, cap)
    q = rand_q(B, Hq, k)
    idx = np.full((B, H, k + w), -1, np.int64)
    for b in range(B):
        for g in range(H):
            n = int(rng.integers(0, min(cap, k + w) + 1)) if (b + g) % 4 else min(cap, k + w)
            if B > 2 and b == B - 1:
                n = 0
            idx[b, g, rng.permutation(k + w)[:n]] = rng.permutation(cap)[:n]
    o, lse = run_sparse(hs2, rec, idx, Hq, q, k, w)
    oh, lh, qh = host_f64(o), lse.cpu().numpy(), host_f64(q)
    G = Hq // H
    for b in range(B):
        for g in range(H):
            h = slice(g * G, g * G + G)
            at = idx[b, g][idx[b, g] >= 0]
            ref.check(oh[b, h], lh[b, h], qh[b, h], rec[b, g, at], SC, f"row {b} head {g}, {len(at)} entries")
    o2, _ = run_sparse(hs2, rec, idx, Hq, q, k, w, lse=False)
    import torch
    assert torch.equal(o, o2)
    assert hs2.hs2_get_device_status() == hs2.OK


def test_sparse_bad_entries_and_repeats(hs2):
    import torch
    cap, H, Hq, k, w = 300, 2, 8, 64, 16
    full = make_cache([cap + 64], cap + 64, H, 5)      # spare rows behind the cache
    rec = full[:, :, :cap].copy()
    q = rand_q(1, Hq, 6)
    idx = np.random.default_rng(7).integers(0, cap, (1, H, k + w))     # repeats count again
    bad = idx.copy()
    bad[0, 0, [0, 9, 79]] = [cap, -2, 1 << 30]
    bad[0, 1, 40] = cap + 63
    clean = np.where((bad < 0) | (bad >= cap), -1, bad)
    a = run_sparse(hs2, rec, clean, Hq, q, k, w)
    assert hs2.hs2_get_device_status() == hs2.OK
    b = run_sparse(hs2, rec, bad, Hq, q, k, w)
    assert hs2.hs2_get_device_status() == hs2.ERR_BAD_INDEX
    assert hs2.hs2_get_device_status() == hs2.OK
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    oh, lh, qh = host_f64(a[0]), a[1].cpu().numpy(), host_f64(q)
    for g in range(H):
        at = clean[0, g][clean[0, g] >= 0]
        ref.check(oh[0, 4 * g:4 * g + 4], lh[0, 4 * g:4 * g + 4], qh[0, 4 * g:4 * g + 4], rec[0, g, at], SC)


# ---------------------------------------------------------------------------
# the block's decode step, and the calls together
# ---------------------------------------------------------------------------
def reference_lists(q, rec, n, k, w):
    """Selection of one (sequence, KV head) in 64 bits: list, scores."""
    K, _ = ref.values(rec[:n])
    s = SC * (q @ K.T)
    lse = ref.attend(q, rec[:n], SC)[1]
    score = np.exp(s - lse[:, None]).sum(0)
    cand = max(0, n - w)
    order = np.argsort(-score[:cand], kind="stable")[:k]
    lst = np.full(k + w, -1, np.int64)
    lst[:len(order)] = np.sort(order)
    win = np.arange(n - w, n)
    lst[k:] = np.where(win >= 0, win, -1)
    return lst, score, (score[order[-1]] if cand > k and k else math.nan)


@pytest.mark.parametrize("Hq,H,k,w,lens", [(16, 2, 256, 64, [1500, 900, 320, 319, 64, 1]),
                                           (16, 1, 128, 16, [9001, 100]),
                                           (4, 2, 64, 16, [700, 81, 80, 2]), (2, 2, 0, 16, [500, 3]),
                                           (8, 1, 2048, 32, [5000, 2081, 2080]), (1, 1, 1, 1, [3, 2, 1])])
def test_block_decode(hs2, Hq, H, k, w, lens):
    import torch
    from helpers import SEL_REL
    B, cap, L = len(lens), max(lens) + 3, 2
    rec = make_cache(lens, cap, H, 201)
    q, qs = rand_q(B, Hq, 202), [rand_q(B, Hq, 203 + i) for i in range(L)]
    shape = hs2.Shape.make(cap, Hq, H, k_global=k, window=w)
    cache = dev(rec)
    o = torch.empty(B, Hq, 128, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(B, Hq, device="cuda")
    idx = torch.full((B, H, k + w), -9, dtype=torch.int32, device="cuda")
    os_ = [torch.empty_like(o) for _ in range(L)]
    ws = torch.full((hs2.workspace_size(hs2.OP_BLOCK_DECODE_Q4, shape, B),), 0xFF, dtype=torch.uint8,
                    device="cuda")
    hs2.hs2_block_decode_q4(lens, q, cache, o, lse, idx, qs, os_, shape, ws)
    assert hs2.hs2_get_device_status() == hs2.OK
    check_attn(o, lse, q, rec, lens, Hq)
    gi, qh, G = idx.cpu().numpy().astype(np.int64), host_f64(q), Hq // H
    for b, n in enumerate(lens):
        for g in range(H):
            h = slice(g * G, g * G + G)
            want, score, kth = reference_lists(qh[b, h], rec[b, g], n, k, w)
            assert np.array_equal(gi[b, g, k:], want[k:])
            a, c = gi[b, g, :k], want[:k]
            assert (a >= 0).sum() == (c >= 0).sum() and np.all(np.diff(a[a >= 0]) > 0)
            off = np.array(sorted(set(a[a >= 0]) ^ set(c[c >= 0])), np.int64)
            # a position may differ only where its score ties with the k-th to SEL_REL
            assert off.size == 0 or np.all(np.abs(score[off] - kth) <= SEL_REL * kth)
            at = gi[b, g][gi[b, g] >= 0]
            for l in range(L):
                x = host_f64(os_[l])[b, h]
                want_l = ref.attend(host_f64(qs[l])[b, h], rec[b, g, at], SC)[1]
                ref.check(x, want_l, host_f64(qs[l])[b, h], rec[b, g, at], SC, f"layer {l} seq {b} head {g}")
    # the operators alone give what the step gave
    o1, lse1 = run_attn(hs2, cache, lens, Hq, q)
    assert torch.equal(o1, o) and torch.equal(lse1, lse)
    for l in range(L):
        x = torch.empty_like(o)
        hs2.hs2_sparse_attn_q4(qs[l], cache, idx, x, None, shape)
        assert torch.equal(x, os_[l])


@pytest.mark.parametrize("k", [1, 100, 1024, 2048])
def test_block_ties_take_the_smallest_positions(hs2, k):
    """All records of a head equal, so every candidate's score ties: the list
    holds positions 0 .. k - 1; and the workspace's end is respected."""
    import torch
    lens, H, Hq, w, cap = [4000, 2100], 2, 16, 16, 4000
    rec = np.repeat(make_cache([1], 1, H, 7)[0][None, :, :1], cap, axis=2).repeat(2, 0)
    shape = hs2.Shape.make(cap, Hq, H, k_global=k, window=w)
    need = hs2.workspace_size(hs2.OP_BLOCK_DECODE_Q4, shape, 2)
    buf = torch.full((need + 4096,), 0xAB, dtype=torch.uint8, device="cuda")
    q = rand_q(2, Hq, 8)
    o, lse = torch.empty_like(q), torch.empty(2, Hq, device="cuda")
    idx = torch.empty(2, H, k + w, dtype=torch.int32, device="cuda")
    hs2.hs2_block_decode_q4(lens, q, dev(rec), o, lse, idx, [], [], shape, buf[:need])
    for b, n in enumerate(lens):
        for g in range(H):
            assert np.array_equal(idx[b, g].cpu().numpy(), np.r_[np.arange(min(k, n - w)),
                                                                 np.full(max(0, k - (n - w)), -1),
                                                                 np.arange(n - w, n)])
    assert (buf[need:] == 0xAB).all()
    check_attn(o, lse, q, rec, lens, Hq)


def test_block_more_layers_than_one_launch_takes(hs2):
    import torch
    lens, H, Hq, k, w, L = [300, 40], 1, 8, 32, 8, 19
    rec = make_cache(lens, 300, H, 9)
    shape = hs2.Shape.make(300, Hq, H, k_global=k, window=w)
    ws = torch.empty(hs2.workspace_size(hs2.OP_BLOCK_DECODE_Q4, shape, 2), dtype=torch.uint8, device="cuda")
    cache, q = dev(rec), rand_q(2, Hq, 10)
    qs = [rand_q(2, Hq, 11 + i) for i in range(L)]
    os_ = [torch.empty_like(q) for _ in range(L)]
    o, lse = torch.empty_like(q), torch.empty(2, Hq, device="cuda")
    idx = torch.empty(2, H, k + w, dtype=torch.int32, device="cuda")
    hs2.hs2_block_decode_q4(lens, q, cache, o, lse, idx, qs, os_, shape, ws)
    gi = idx.cpu().numpy()
    for i in range(L):
        for b in range(2):
            at = gi[b, 0][gi[b, 0] >= 0]
            qh = host_f64(qs[i])[b]
            ref.check(host_f64(os_[i])[b], ref.attend(qh, rec[b, 0, at], SC)[1], qh, rec[b, 0, at], SC)


def test_captured_block_step(hs2):
    """The captured step replays on new queries and cache contents, bit for bit
    as the eager call, whatever the workspace held."""
    import torch
    lens, H, Hq, k, w, L = [900, 333], 2, 16, 128, 16, 3
    cap = 900
    shape = hs2.Shape.make(cap, Hq, H, k_global=k, window=w)
    cache = torch.empty(2, H, cap, 144, dtype=torch.uint8, device="cuda")
    q = torch.empty(2, Hq, 128, dtype=torch.bfloat16, device="cuda")
    qs = [torch.empty_like(q) for _ in range(L)]
    nb = hs2.workspace_size(hs2.OP_BLOCK_DECODE_Q4, shape, 2)
    ws = torch.full((nb,), 0xFF, dtype=torch.uint8, device="cuda")

    def outputs():
        return (torch.empty_like(q), torch.empty(2, Hq, device="cuda"),
                torch.empty(2, H, k + w, dtype=torch.int32, device="cuda"), [torch.empty_like(q) for _ in range(L)])

    out = outputs()
    g = torch.cuda.CUDAGraph()
    cache.copy_(dev(make_cache(lens, cap, H, 1)))
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        hs2.hs2_block_decode_q4(lens, q, cache, out[0], out[1], out[2], qs, out[3], shape, ws)
    for step in range(3):
        cache.copy_(dev(make_cache(lens, cap, H, 500 + step)))
        for i, t in enumerate([q, *qs]):
            t.copy_(rand_q(2, Hq, 600 + 10 * step + i))
        ws.fill_(255 - step)
        for _ in range(2):
            g.replay()
        torch.cuda.synchronize()
        want = outputs()
        ws2 = torch.full((nb,), 7 * step, dtype=torch.uint8, device="cuda")
        hs2.hs2_block_decode_q4(lens, q, cache, want[0], want[1], want[2], qs, want[3], shape, ws2)
        for a, b in zip([*out[:3], *out[3]], [*want[:3], *want[3]]):
            assert torch.equal(a, b)
    assert hs2.hs2_get_device_status() == hs2.OK


def test_serving_run(hs2):
    """As they are used: a prompt's bridged K/V quantised as written, then
    decode steps that append a token and run the block; the cache read back
    feeds the next chunk's prefill."""
    import torch
    torch.manual_seed(9)
    B, H, Hq, cap, T0, k, w = 2, 2, 16, 640, 512, 64, 16
    shape = hs2.Shape.make(cap, Hq, H, k_global=k, window=w)
    cache = torch.empty(B, H, cap, 144, dtype=torch.uint8, device="cuda")
    Kb, Vb = [], []
    for b in range(B):
        qkv = torch.randn(T0, (Hq + 2 * H) * 128, device="cuda").bfloat16()
        K = qkv[:, Hq * 128:(Hq + H) * 128].unflatten(1, (H, 128))
        V = qkv[:, (Hq + H) * 128:].unflatten(1, (H, 128))
        hs2.hs2_cache_write_q4(K, V, None, cache, shape, first=b * cap)
        Kb.append(bits(K.contiguous()))
        Vb.append(bits(V.contiguous()))
    o, lse = torch.empty(B, Hq, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(B, Hq, device="cuda")
    idx, os_ = torch.empty(B, H, k + w, dtype=torch.int32, device="cuda"), torch.empty_like(o)
    ws = torch.empty(hs2.workspace_size(hs2.OP_BLOCK_DECODE_Q4, shape, B), dtype=torch.uint8, device="cuda")
    for step in range(3):
        new = torch.randn(B, 2 * H, 128, device="cuda").bfloat16()
        n = T0 + step + 1
        slot = dev(np.array([b * cap + n - 1 for b in range(B)], np.int32))
        hs2.hs2_cache_write_q4(new[:, :H], new[:, H:], slot, cache, shape)
        for b in range(B):
            Kb[b] = np.concatenate([Kb[b], bits(new[b:b + 1, :H].contiguous())])
            Vb[b] = np.concatenate([Vb[b], bits(new[b:b + 1, H:].contiguous())])
        q, qs = rand_q(B, Hq, 300 + step), rand_q(B, Hq, 310 + step)
        hs2.hs2_block_decode_q4([n] * B, q, cache, o, lse, idx, [qs], [os_], shape, ws)
        recs = np.stack([np.moveaxis(ref.records(Kb[b], Vb[b]), 0, 1) for b in range(B)])
        check_attn(o, lse, q, recs, [n] * B, Hq, f"step {step}")
        gi, oh, qh = idx.cpu().numpy(), host_f64(os_), host_f64(qs)
        for b in range(B):
            for g in range(H):
                at = gi[b, g][gi[b, g] >= 0]
                assert len(set(at)) == len(at) == k + w
                h = slice(g * 8, g * 8 + 8)
                wl = ref.attend(qh[b, h], recs[b, g, at], SC)[1]
                ref.check(oh[b, h], wl, qh[b, h], recs[b, g, at], SC)
    # the prefix as bf16 for a prefill over it: full attention of its last row
    # agrees with the decode step's attention (the same values but for bf16
    # rounding of K and V: half a step, 2^-8, of each; with logits below 8 that
    # moves a logit by at most 2^-8 * scale * sum |q||k|)
    n = T0 + 3
    K, V = torch.empty(n, H, 128, dtype=torch.bfloat16, device="cuda"), None
    V = torch.empty_like(K)
    hs2.hs2_cache_read_q4(cache, None, K, V, shape, first=0)
    rk, rv = ref.values(np.moveaxis(recs[0], 0, 1))
    assert np.array_equal(bits(K), ref.to_bf16_bits(rk)) and np.array_equal(bits(V), ref.to_bf16_bits(rv))
    Q = torch.zeros(n, Hq, 128, dtype=torch.bfloat16, device="cuda")
    Q[-1] = q[0]
    O, L = torch.empty_like(Q), torch.empty(n, Hq, device="cuda")
    hs2.hs2_full_attn_lse(Q, K, V, O, L, hs2.Shape.make(n, Hq, H))
    qh = host_f64(q)[0]
    for h in range(Hq):
        dl = 2.0 ** -8 * SC * (np.abs(rk[:, h // 8]) @ np.abs(qh[h])).max()
        assert abs(float(L[-1, h]) - float(lse[0, h])) <= dl + 1e-4
    assert hs2.hs2_get_device_status() == hs2.OK


def test_waits_with_a_tiny_budget_end(hs2):
    """With a wait budget of one cycle the attention and the sparse kernel end,
    whether a wait was given up (reported) or its copy had landed by its second
    try; afterwards, with the default budget, they are right."""
    import torch
    lens, H, Hq = [2000, 900], 2, 16
    rec = make_cache(lens, 2000, H, 401)
    q = rand_q(2, Hq, 402)
    idx = np.tile(np.arange(80), (2, H, 1))
    assert hs2.hs2_get_device_status() == hs2.OK
    hs2.hs2_debug_set_wait_budget(1)
    try:
        run_attn(hs2, rec, lens, Hq, q)
        st = hs2.hs2_get_device_status()
        run_sparse(hs2, rec, idx, Hq, q, 64, 16)
        st2 = hs2.hs2_get_device_status()
    finally:
        hs2.hs2_debug_set_wait_budget(0)
    assert {st, st2} <= {hs2.OK, hs2.ERR_TIMEOUT}
    assert hs2.hs2_get_device_status() == hs2.OK
    o, lse = run_attn(hs2, rec, lens, Hq, q)
    check_attn(o, lse, q, rec, lens, Hq)
    assert torch.isfinite(lse).all()


def test_binding_refuses_wrong_shapes(hs2):
    import torch
    shape = hs2.Shape.make(16, 8, 2, k_global=3, window=1)
    cache = torch.zeros(2, 2, 16, 144, dtype=torch.uint8, device="cuda")
    x = torch.zeros(4, 2, 128, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(2, 8, 128, dtype=torch.bfloat16, device="cuda")
    slot = torch.zeros(4, dtype=torch.int32, device="cuda")
    idx = torch.zeros(2, 2, 4, dtype=torch.int32, device="cuda")
    for bad in (lambda: hs2.hs2_cache_write_q4(x, x[:3], None, cache, shape),
                lambda: hs2.hs2_cache_write_q4(x, x, slot[:3], cache, shape),
                lambda: hs2.hs2_cache_write_q4(x, x, slot.long(), cache, shape),
                lambda: hs2.hs2_cache_write_q4(x.float(), x, slot, cache, shape),
                lambda: hs2.hs2_cache_write_q4(x.transpose(0, 1), x, None, cache, shape),
                lambda: hs2.hs2_cache_write_q4(x, x, None, cache[:, :, :8], shape),
                lambda: hs2.hs2_cache_write_q4(x, x, None, cache.cpu(), shape),
                lambda: hs2.hs2_sparse_attn_q4(q, cache, idx[..., :3], q, None, shape),
                lambda: hs2.hs2_sparse_attn_q4(q[:1], cache, idx, q, None, shape)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(hs2.HS2Error):
        hs2.hs2_cache_write_q4(x, x, None, cache, shape, first=29)
    hs2.hs2_cache_write_q4(x[:0], x[:0], slot[:0], cache, shape)
    assert not cache.any()
