"""Plain numpy reference, in 64 bits, of the quantised caches and of the
operators over the 4-bit one (tests only; shares no code with the library)."""
import numpy as np

D, REC = 128, 144


def to_bf16_bits(x):
    """fp64 -> bf16 bits, round to nearest even (finite, normal range)."""
    import torch
    return torch.from_numpy(np.ascontiguousarray(x, np.float64)).to(torch.bfloat16).view(
        torch.int16).numpy().view(np.uint16)


def from_bf16_bits(b):
    return (np.asarray(b, np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def nibble_k(e):
    g, r = divmod(e, 32)
    return 8 * (4 * (r // 8) + g) + r % 8


def nibble_v(e):
    g, r = divmod(e, 32)
    return 4 * (4 * (r // 4) + g) + r % 4


NIB_K = np.array([nibble_k(e) for e in range(D)])
NIB_V = np.array([nibble_v(e) for e in range(D)])


def quantise(bits):
    """bf16 bits [..., 128] -> (codes -7..7 [..., 128], scale bf16 bits [..., 4])."""
    x = from_bf16_bits(bits).reshape(*bits.shape[:-1], 4, 32)
    with np.errstate(all="ignore"):
        amax = np.abs(x).max(-1)
        ok = np.isfinite(amax)
        s = np.maximum(from_bf16_bits(to_bf16_bits(np.where(ok, amax, 0) / 7)), 2.0 ** -120)
        c = np.clip(np.rint(np.where(ok[..., None], x, 0) / s[..., None]), -7, 7)
    sb = np.where(ok, to_bf16_bits(s), 0x7FC0).astype(np.uint16)
    return c.reshape(bits.shape).astype(np.int64), sb


def records(Kb, Vb):
    """bf16 bits K, V [..., 128] -> uint8 records [..., 144]."""
    out = np.zeros((*Kb.shape[:-1], REC), np.uint8)
    for bits, nib, at, sat in ((Kb, NIB_K, 0, 128), (Vb, NIB_V, 64, 136)):
        c, s = quantise(bits)
        n = np.zeros((*bits.shape[:-1], D), np.uint8)
        n[..., nib] = (c + 8).astype(np.uint8)
        out[..., at:at + 64] = n[..., 0::2] | (n[..., 1::2] << 4)
        out[..., sat:sat + 8] = np.ascontiguousarray(s).view(np.uint8)
    return out


def values(rec):
    """uint8 records [..., 144] -> K, V fp64 [..., 128]."""
    outs = []
    for nib, at, sat in ((NIB_K, 0, 128), (NIB_V, 64, 136)):
        b = rec[..., at:at + 64].astype(np.int64)
        n = np.stack([b & 15, b >> 4], -1).reshape(*rec.shape[:-1], D)[..., nib] - 8
        s = from_bf16_bits(np.ascontiguousarray(rec[..., sat:sat + 8]).view(np.uint16))
        with np.errstate(all="ignore"):
            outs.append(n * np.repeat(s, 32, axis=-1))
    return outs


def scales_k(rec):
    return from_bf16_bits(np.ascontiguousarray(rec[..., 128:136]).view(np.uint16))


def attend(q, rec, scale):
    """q [G, 128] fp64 over records [n, 144]: o, lse, A = sum p |v|, and the
    bound on a logit's error.

    Logit: per group two MMAs accumulate 16 products of a nibble (<= 15) with q
    onto -8 sum q, each accumulation rounding (or truncating) by at most 2^-23
    of a magnitude <= 23 sum |q|; then four fp32 multiply-adds and two
    multiplications of 2^-24 each."""
    G = q.shape[0]
    if len(rec) == 0:
        return np.zeros((G, D)), np.full(G, -np.inf), np.zeros((G, D)), np.zeros(G)
    K, V = values(rec)
    s = scale * (q @ K.T)
    m = s.max(-1, keepdims=True)
    p = np.exp(s - m)
    l = p.sum(-1, keepdims=True)
    q1 = np.abs(q).reshape(G, 4, 32).sum(-1)
    ds = scale * (q1 @ scales_k(rec).T) * 23 * (2 * 2.0 ** -23 + 6 * 2.0 ** -24)
    return p @ V / l, (m + np.log(l))[:, 0], p @ np.abs(V) / l, ds.max(-1)


def check(o, lse, q, rec, scale, what=""):
    """o [G, 128], lse [G] of the library against attend().

    o: half a bf16 step (2^-8) of its value, plus, relative to A = sum p |v|:
    two roundings of P to f16 (2^-11 each; the kernels round it once), exp2
    (2^-22) and logit errors ds of p and of its sum, and a rounding of 2^-23 per
    accumulation (one per 16 tokens, and the joins).  Below 2^-24 f16 is absolute: 2^-35 of the running
    maximum per token.  lse: ds, the sum's roundings, 2^-22 of exp2 and log2,
    and 2^-23 of its value for the last operations in fp32."""
    n = len(rec)
    want, wl, A, ds = attend(q, rec, scale)
    if n == 0:
        assert np.all(o == 0) and np.all(np.isneginf(lse)), what
        return
    acc = (n / 16 + 64) * 2.0 ** -23
    rel = 2 * 2.0 ** -11 + 2 * (ds + 2.0 ** -22) + acc
    vmax = np.abs(values(rec)[1]).max()
    assert np.isfinite(o).all() and np.isfinite(lse).all(), f"{what}: non-finite output"
    tol = 2.0 ** -8 * np.abs(want) + (1 + 2.0 ** -7) * rel[:, None] * A + n * 2.0 ** -33 * vmax
    bad = np.abs(o - want) > tol
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} off, worst "
                           f"{(np.abs(o - want) / np.maximum(tol, 1e-300)).max():.2f} x the bound")
    lt = ds + acc + 4 * 2.0 ** -22 + 2.0 ** -22 * np.abs(wl)
    assert np.all(np.abs(lse - wl) <= lt), f"{what}: lse off by {np.abs(lse - wl).max():.2e} > {lt.min():.2e}"
