"""The operators over the 4-bit cache at the ends of their range: logits far
beyond fp32's spacing of 1, and V scales far apart."""
import numpy as np
import pytest

import q4_reference as ref
from helpers import dev, dev_bf16, host_f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hs2():
    import torch
    assert torch.cuda.is_available()
    import long_context_bridge_b200 as m
    return m


def attend(hs2, rec, lens, q, scale):
    """hs2_decode_attn_q4 over records [B, H, cap, 144]: o, lse in 64 bits."""
    import torch
    B, H, cap, _ = rec.shape
    Hq = q.shape[1]
    shape = hs2.Shape.make(cap, Hq, H, scale=scale)
    o, lse = torch.empty_like(q), torch.empty(B, Hq, device="cuda")
    ws = torch.full((hs2.workspace_size(hs2.OP_DECODE_ATTN_Q4, shape, B),), 0xFF, dtype=torch.uint8, device="cuda")
    hs2.hs2_decode_attn_q4(dev(np.asarray(lens, np.int32)), q, dev(rec), o, lse, shape, ws)
    return host_f64(o), lse.double().cpu().numpy()


def sparse(hs2, rec, idx, q, scale):
    import torch
    B, H, cap, _ = rec.shape
    shape = hs2.Shape.make(cap, q.shape[1], H, scale=scale, k_global=idx.shape[-1] - 1, window=1)
    o, lse = torch.empty_like(q), torch.empty(B, q.shape[1], device="cuda")
    hs2.hs2_sparse_attn_q4(q, dev(rec), dev(idx.astype(np.int32)), o, lse, shape)
    return host_f64(o), lse.double().cpu().numpy()


def block(hs2, rec, lens, q, scale, k, w):
    import torch
    B, H, cap, _ = rec.shape
    shape = hs2.Shape.make(cap, q.shape[1], H, scale=scale, k_global=k, window=w)
    o, os_, lse = torch.empty_like(q), torch.empty_like(q), torch.empty(B, q.shape[1], device="cuda")
    idx = torch.empty(B, H, k + w, dtype=torch.int32, device="cuda")
    ws = torch.full((hs2.workspace_size(hs2.OP_BLOCK_DECODE_Q4, shape, B),), 0xFF, dtype=torch.uint8, device="cuda")
    hs2.hs2_block_decode_q4(lens, q, dev(rec), o, lse, idx, [q], [os_], shape, ws)
    return host_f64(o), lse.double().cpu().numpy(), idx.cpu().numpy(), host_f64(os_)


# One key alone carries the softmax, so o is its V row: half a bf16 step (2^-8),
# one rounding of P x V scale to f16 (2^-11), and fp32 roundings of p, its sum
# and the joins (2^-18 together).  lse is its logit: exact group sums, then at
# most 8 roundings of 2^-24 (scale times log2 e and that constant, the product,
# the sum's logarithm added once per join, ln 2 and its product).
O_REL = 2.0 ** -8 + 2.0 ** -11 + 2.0 ** -18
LSE_REL = 2.0 ** -21


def exact_keys(n, H, mul, sign, seed):
    """Records whose logits are c * 2^a exactly with one largest, c whole: K has
    one dim other than 0 per key.  V of order 1.  Returns records, top key."""
    rng = np.random.default_rng(seed)
    K, V = np.zeros((H, n, 128)), rng.standard_normal((H, n, 128))
    top = rng.integers(0, n, H)
    for h in range(H):
        c = rng.integers(1, 6, n) if sign > 0 else -rng.integers(2, 8, n)
        c[top[h]] = 6 if sign > 0 else -1
        # the group holds 7 in a dim that no query meets, so its scale is mul
        K[h, :, 37] = 7 * mul
        K[h, :, 40] = c * mul
    return ref.records(ref.to_bf16_bits(K), ref.to_bf16_bits(V)), top


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("a", [20, 23, 25, 26, 27, 28, 30, 33, 40, 60, 90, 110])
@pytest.mark.parametrize("Hq,H", [(8, 1), (16, 1), (2, 2)])
def test_exact_large_logits(hs2, Hq, H, a, sign):
    """Logits up to 6 * 2^a, exact in fp32: the largest takes all, in the
    attention, over a list and in the block step."""
    n, G = 1300, Hq // H
    rec, top = exact_keys(n, H, 2.0 ** (a // 2), sign, 100 + a)
    q = np.zeros((1, Hq, 128))
    q[..., 40] = 2.0 ** (a - a // 2)
    q[..., 90] = 3.0            # K is 0 there
    V = ref.values(rec)[1]
    best = 6.0 * 2.0 ** a if sign > 0 else -(2.0 ** a)
    dq = dev_bf16(ref.to_bf16_bits(q))
    idx = np.tile(np.random.default_rng(a).permutation(n), (1, H, 1))
    k, w = 300, 20
    ob, lb, lists, osb = block(hs2, rec[None], [n], dq, 1.0, k, w)
    for o, lse in (attend(hs2, rec[None], [n], dq, 1.0), sparse(hs2, rec[None], idx, dq, 1.0), (ob, lb), (osb, None)):
        assert np.isfinite(o).all()
        for h in range(Hq):
            v = V[h // G, top[h // G]]
            assert np.all(np.abs(o[0, h] - v) <= O_REL * np.abs(v)), f"head {h}"
        if lse is not None:
            assert np.all(np.abs(lse - best) <= LSE_REL * abs(best))
    for g in range(H):
        assert top[g] in lists[0, g]


@pytest.mark.parametrize("mul", [3e6, 1.6e7, 3.5e7, 1e9, 1e11])
def test_random_large_logits(hs2, mul):
    """N(0, 1) keys under queries of magnitude mul (logits about 35 mul): where
    the largest logit of a head exceeds every other by more than their errors and
    40, it takes all; every output is finite and within V's extremes."""
    n, Hq, H, draws = 300, 8, 2, 12
    apart = 0
    for seed in range(draws):
        rng = np.random.default_rng(seed)
        rec = ref.records(*(ref.to_bf16_bits(rng.standard_normal((H, n, 128))) for _ in range(2)))
        qh = ref.from_bf16_bits(ref.to_bf16_bits(rng.standard_normal((1, Hq, 128)) * mul))
        dq = dev_bf16(ref.to_bf16_bits(qh))
        idx = np.tile(rng.permutation(n), (1, H, 1))
        K, V = ref.values(rec)
        for o, lse in (attend(hs2, rec[None], [n], dq, 1.0), sparse(hs2, rec[None], idx, dq, 1.0)):
            assert np.isfinite(o).all() and np.isfinite(lse).all(), f"draw {seed}"
            for h in range(Hq):
                g = h // (Hq // H)
                s = K[g] @ qh[0, h]
                # the error of a group's sum as in ref.attend, per key, and the
                # roundings behind it
                ds = np.abs(qh[0, h]).reshape(4, 32).sum(-1) @ ref.scales_k(rec[g]).T * 23 * 5 * 2.0 ** -23
                ds += LSE_REL * np.abs(s)
                best = int(np.argmax(s))
                assert np.all(np.abs(o[0, h]) <= (1 + 2.0 ** -7) * np.abs(V[g]).max(0))
                if np.sum(s + ds > s[best] - ds[best] - 40) > 1:
                    continue
                apart += 1
                assert np.all(np.abs(o[0, h] - V[g, best]) <= O_REL * np.abs(V[g, best])), f"draw {seed} head {h}"
                assert abs(lse[0, h] - s[best]) <= ds[best]
    assert apart >= draws * Hq      # of 2 * draws * Hq comparisons


@pytest.mark.parametrize("qmul,kmul,scale", [(2.0 ** -60, 2.0 ** -60, 2.0 ** 115), (2.0 ** -100, 2.0 ** -20, 2.0 ** 117),
                                             (2.0 ** 100, 2.0 ** -110, 2.0 ** 8), (2.0 ** 115, 2.0 ** -112, None),
                                             (2.0 ** -125, 2.0 ** 115, 2.0 ** 8), (2.0 ** 20, 2.0 ** 90, 2.0 ** -112)])
def test_scales_of_any_size(hs2, qmul, kmul, scale):
    """Logits of order 10 from factors at the ends of fp32."""
    n, Hq = 300, 8
    rng = np.random.default_rng(9)
    scale = 128 ** -0.5 if scale is None else scale
    sc = np.float64(np.float32(scale))
    rec = ref.records(ref.to_bf16_bits(rng.standard_normal((1, n, 128)) * kmul), ref.to_bf16_bits(rng.standard_normal((1, n, 128))))
    q = dev_bf16(ref.to_bf16_bits(rng.standard_normal((1, Hq, 128)) * qmul))
    qh = host_f64(q)
    idx = rng.permutation(n)[None, None]
    ob, lb, lists, osb = block(hs2, rec[None], [n], q, scale, 30, 20)
    for what, (o, lse) in (("attention", attend(hs2, rec[None], [n], q, scale)), ("block", (ob, lb)),
                           ("list", sparse(hs2, rec[None], idx, q, scale))):
        ref.check(o[0], lse[0], qh[0], rec[0], sc, what)
    at = lists[0, 0]
    ref.check(osb[0], ref.attend(qh[0], rec[0, at], sc)[1], qh[0], rec[0, at], sc, "sparse layer")


def check_groups(o, q, rec, scale, what):
    """o [G, 128] against the definition, each group of 32 dims for itself: the
    bound of q4_reference.check with the absolute term of f16's end taken from
    the group alone.  A weight times a V scale loses at most 2^-25 (half of f16's
    last spacing) of 2^10 (the least a largest weight stands at) times the
    group's largest scale: 2^-35 of the group's largest |V| per key."""
    want, _, A, ds = ref.attend(q, rec, scale)
    V = ref.values(rec)[1]
    n = len(rec)
    rel = 2 * 2.0 ** -11 + 2 * (ds + 2.0 ** -22) + (n / 16 + 64) * 2.0 ** -23
    for g in range(4):
        d = slice(32 * g, 32 * g + 32)
        tol = (2.0 ** -8 * np.abs(want[:, d]) + (1 + 2.0 ** -7) * rel[:, None] * A[:, d]
               + n * 2.0 ** -35 * np.abs(V[:, d]).max())
        assert np.median(tol / A[:, d]) < 2.0 ** -7, "the bound says nothing"
        bad = np.abs(o[:, d] - want[:, d]) > tol
        assert not bad.any(), f"{what}: group {g}, {bad.sum()} of {bad.size} off"


@pytest.mark.parametrize("Hq,H", [(8, 1), (16, 1), (4, 2)])
@pytest.mark.parametrize("powers", [(0, 20, 0, 0), (0, 60, -60, 5), (-110, 120, 0, 30), (-116, -100, -70, -40),
                                    (122, 122, -116, 122)])
def test_groups_of_v_far_apart(hs2, Hq, H, powers):
    """Each group of 32 dims keeps its accuracy beside groups of any magnitude."""
    n, G = 700, Hq // H
    rng = np.random.default_rng(sum(abs(p) for p in powers))
    K = rng.standard_normal((H, n, 128))
    V = np.clip(rng.standard_normal((H, n, 128)), -3, 3) * np.repeat(np.exp2(np.array(powers, np.float64)), 32)
    rec = ref.records(ref.to_bf16_bits(K), ref.to_bf16_bits(V))
    qh = ref.from_bf16_bits(ref.to_bf16_bits(rng.standard_normal((1, Hq, 128))))
    q = dev_bf16(ref.to_bf16_bits(qh))
    sc = 128 ** -0.5
    idx = np.tile(rng.permutation(n), (1, H, 1))
    ob, _, lists, osb = block(hs2, rec[None], [n], q, sc, 300, 20)
    for what, o in (("attention", attend(hs2, rec[None], [n], q, sc)[0]), ("list", sparse(hs2, rec[None], idx, q, sc)[0]),
                    ("block", ob)):
        for g in range(H):
            h = slice(g * G, g * G + G)
            check_groups(o[0, h], qh[0, h], rec[g], sc, what)
    for g in range(H):
        h = slice(g * G, g * G + G)
        check_groups(osb[0, h], qh[0, h], rec[g, lists[0, g]], sc, "sparse layer")


@pytest.mark.parametrize("spread", [8, 16, 22])
def test_keys_of_v_far_apart(hs2, spread):
    """V rows within 2^spread of each other in any order: the bound of a group
    holds over all of its keys."""
    n, Hq = 900, 8
    rng = np.random.default_rng(spread)
    K = rng.standard_normal((1, n, 128))
    V = rng.standard_normal((1, n, 128)) * np.exp2(rng.uniform(-spread, 0, (1, n, 1)))
    rec = ref.records(ref.to_bf16_bits(K), ref.to_bf16_bits(V))
    qh = ref.from_bf16_bits(ref.to_bf16_bits(rng.standard_normal((1, Hq, 128))))
    q = dev_bf16(ref.to_bf16_bits(qh))
    sc = 128 ** -0.5
    idx = rng.permutation(n)[None, None]
    for what, o in (("attention", attend(hs2, rec[None], [n], q, sc)[0]), ("list", sparse(hs2, rec[None], idx, q, sc)[0])):
        check_groups(o[0], qh[0], rec[0], sc, what)
