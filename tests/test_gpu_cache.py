"""Rows into and out of the decode caches on the GPU: bit for bit against the
definitions (4-bit: numpy in 64 bits; e4m3: the oracle's quantiser)."""
import numpy as np
import pytest

import q4_reference as ref
import synth
from helpers import bits, dev, dev_bf16

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hs2():
    import torch
    assert torch.cuda.is_available()
    import long_context_bridge_b200 as m
    return m


def awkward_rows(n, H, seed):
    """bf16 bits [n, H, 128]: normal values of many magnitudes, and rows of
    ties, zeros, subnormals and the largest finite value."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((n, H, 128)) * np.exp2(rng.integers(-30, 30, (n, H, 1)))
    b = ref.to_bf16_bits(x)
    f = b.reshape(n * H, 128)
    for i in range(0, n * H, 5):
        kind = (i // 5) % 6
        if kind == 0:
            f[i] = ref.to_bf16_bits(rng.integers(-15, 16, 128) / 2.0)     # ties: scale 1 or near
            f[i, ::32] = 0x40E0                                            # 7.0 -> scale exactly 1
        elif kind == 1:
            f[i, 32:64] = 0
        elif kind == 2:
            f[i] = rng.integers(0, 128, 128)                               # subnormals
        elif kind == 3:
            f[i, 5] = 0x7F7F                                               # largest finite
        elif kind == 4:
            f[i] = 0x8000 | rng.integers(0x0300, 0x0400, 128)              # near the scale's floor
        else:
            f[i] = rng.integers(0x3F80, 0x4000, 128)                       # one binade, many ties
    return b


CASES = [(1, 1, 1), (3, 2, 1), (7, 1, 2), (1, 1, 8), (3, 2, 5), (4, 4, 7), (5, 2, 16), (17, 1, 40), (130, 4, 64), (1001, 8, 517)]


@pytest.mark.parametrize("n,H,cap", CASES)
@pytest.mark.parametrize("listed", [False, True])
def test_write_and_read_q4(hs2, n, H, cap, listed):
    import torch
    batch = -(-n // cap) + 1
    rng = np.random.default_rng(n)
    Kb, Vb = awkward_rows(n, H, n), awkward_rows(n, H, n + 1)
    shape = hs2.Shape.make(cap, 2 * H, H)
    first = batch * cap - n - 1 if batch * cap > n else 0     # crosses from one sequence to the next
    slots = first + np.arange(n)
    slot = None
    if listed:
        slots = rng.permutation(batch * cap)[:n]
        slots[n // 2::7] = -1
        slot = dev(slots.astype(np.int32))
    # rows cut from the rows of a fused projection: strided, heads dense
    wide = torch.zeros(n, 128 * (2 * H + 3), dtype=torch.bfloat16, device="cuda")
    K = wide[:, 128:128 * (H + 1)].unflatten(1, (H, 128))
    V = wide[:, 128 * (H + 2):128 * (2 * H + 2)].unflatten(1, (H, 128))
    K.copy_(dev_bf16(Kb))
    V.copy_(dev_bf16(Vb))
    # the copies keep subnormals
    assert np.array_equal(bits(K.contiguous()), Kb)
    cache = torch.full((batch, H, cap, 144), 0xA5, dtype=torch.uint8, device="cuda")
    hs2.hs2_cache_write_q4(K, V, slot, cache, shape, first=first)
    want = np.full((batch, H, cap, 144), 0xA5, np.uint8)
    rec = ref.records(Kb, Vb)
    for i, s in enumerate(slots):
        if s >= 0:
            want[s // cap, :, s % cap] = rec[i]
    assert np.array_equal(cache.cpu().numpy(), want)
    # read back, into rows with another stride; skipped rows stay as they were
    out = torch.full((n, H + 1, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    Ko, Vo = out[:, :H], torch.full((n, H, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    hs2.hs2_cache_read_q4(cache, slot, Ko, Vo, shape, first=first)
    Kv, Vv = ref.values(rec)
    kept = slots >= 0
    for got, val in ((Ko, Kv), (Vo, Vv)):
        g = bits(got.contiguous())
        assert np.array_equal(g[kept], ref.to_bf16_bits(val[kept]))
        assert np.all(g[~kept] == 0x40E0)
    assert np.all(bits(out[:, H].contiguous()) == 0x40E0)
    assert hs2.hs2_get_device_status() == hs2.OK


def test_write_q4_non_finite_groups(hs2):
    """A group with an infinity or a NaN reads back as NaN, the others as usual."""
    import torch
    n, H, cap = 6, 2, 6
    Kb, Vb = awkward_rows(n, H, 3), awkward_rows(n, H, 4)
    Kb[1, 0, 40] = 0x7F80
    Kb[2, 1, 3] = 0xFF80
    Vb[3, 0, 127] = 0x7FC1
    Vb[4, 1, 64] = 0xFFFF
    shape = hs2.Shape.make(cap, H, H)
    cache = torch.zeros(1, H, cap, 144, dtype=torch.uint8, device="cuda")
    hs2.hs2_cache_write_q4(dev_bf16(Kb), dev_bf16(Vb), None, cache, shape)
    rec = ref.records(Kb, Vb)
    assert np.array_equal(cache[0].permute(1, 0, 2).cpu().numpy(), rec)
    Ko = torch.empty(n, H, 128, dtype=torch.bfloat16, device="cuda")
    Vo = torch.empty_like(Ko)
    hs2.hs2_cache_read_q4(cache, None, Ko, Vo, shape)
    for got, val, at in ((Ko, ref.values(rec)[0], (1, 0, 32)), (Vo, ref.values(rec)[1], (4, 1, 64))):
        g = got.double().cpu().numpy()
        assert np.array_equal(np.isnan(g), np.isnan(val))
        assert np.isnan(g[at[0], at[1], at[2]:at[2] + 32]).all() and np.isnan(g).sum() == 64
        ok = ~np.isnan(g)
        assert np.array_equal(bits(got)[ok], ref.to_bf16_bits(np.where(ok, val, 0))[ok])


@pytest.mark.parametrize("n,H,cap", CASES)
@pytest.mark.parametrize("listed", [False, True])
def test_write_and_read_fp8(hs2, orc, n, H, cap, listed):
    import torch
    batch = -(-n // cap) + 1
    rng = np.random.default_rng(n + 7)
    Kb, Vb = awkward_rows(n, H, n + 2), awkward_rows(n, H, n + 3)
    shape = hs2.Shape.make(cap, H, H)
    first = batch * cap - n
    slots = first + np.arange(n)
    slot = None
    if listed:
        slots = rng.permutation(batch * cap)[:n]
        slots[n // 3::5] = -1
        slot = dev(slots.astype(np.int32))
    Kc = torch.full((batch, cap, H, 128), 0x5A, dtype=torch.uint8, device="cuda")
    Vc = torch.full_like(Kc, 0x5B)
    S = torch.full((batch, cap, H), -3.0, device="cuda")
    hs2.hs2_cache_write_fp8(dev_bf16(Kb), dev_bf16(Vb), slot, Kc, Vc, S, shape, first=first)
    wk, wv = np.full((batch * cap, H, 128), 0x5A, np.uint8), np.full((batch * cap, H, 128), 0x5B, np.uint8)
    ws = np.full((batch * cap, H), -3.0, np.float32)
    ok, ov, os_ = np.empty((n, H, 128), np.uint8), np.empty((n, H, 128), np.uint8), np.empty((n, H), np.float32)
    orc.lib().orc_quantize_rows(orc._p(np.ascontiguousarray(Kb)), orc._p(np.ascontiguousarray(Vb)), n * H, 128,
                                orc._p(ok), orc._p(ov), orc._p(os_))
    kept = slots >= 0
    wk[slots[kept]], wv[slots[kept]], ws[slots[kept]] = ok[kept], ov[kept], os_[kept]
    assert np.array_equal(S.cpu().numpy().reshape(-1, H), ws)
    assert np.array_equal(Kc.cpu().numpy().reshape(-1, H, 128), wk)
    assert np.array_equal(Vc.cpu().numpy().reshape(-1, H, 128), wv)
    Ko = torch.full((n, H, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    Vo = torch.full_like(Ko, 7.0)
    S2 = S * 2                                        # separate scales for K and V
    hs2.hs2_cache_read_fp8(Kc, Vc, S, S2, slot, Ko, Vo, shape, first=first)
    table = orc.e4m3_table()
    for got, codes, mul in ((Ko, ok, 1.0), (Vo, ov, 2.0)):
        # code * scale in fp32 and then bf16: the fp32 product of 4 and 24 bits rounds once
        with np.errstate(over="ignore"):
            v = (table[codes].astype(np.float32) * (os_ * np.float32(mul))[..., None]).astype(np.float64)
        g = bits(got)
        assert np.array_equal(g[kept], ref.to_bf16_bits(v)[kept])
        assert np.all(g[~kept] == 0x40E0)
    assert hs2.hs2_get_device_status() == hs2.OK


def test_write_fp8_quotients(hs2, orc):
    """Codes of 2^21 quotients over many magnitudes (signed zeros and tiny
    elements among them), equal to the oracle's."""
    import torch
    n, H = 4096, 2
    rng = np.random.default_rng(17)
    Kb, Vb = (rng.integers(0, 1 << 16, (n, H, 128)).astype(np.uint16) for _ in range(2))
    for b in (Kb, Vb):  # each row pair within 2^30 of its largest element, or without any limit
        top = rng.integers(1, 0x7F00, (n, H, 1))
        low = np.where(rng.random((n, H, 1)) < 0.8, np.maximum(top - (12 << 7), 0), 0)
        mag = low + (rng.random((n, H, 128)) * (top - low + 1)).astype(np.int64)
        b[:] = (mag | (rng.integers(0, 2, mag.shape) << 15)).astype(np.uint16)
        b[:, :, 7], b[:, :, 9] = 0x8000, 0
    shape = hs2.Shape.make(n, H, H)
    Kc = torch.empty(1, n, H, 128, dtype=torch.uint8, device="cuda")
    Vc, S = torch.empty_like(Kc), torch.empty(1, n, H, device="cuda")
    hs2.hs2_cache_write_fp8(dev_bf16(Kb), dev_bf16(Vb), None, Kc, Vc, S, shape)
    ok, ov, os_ = np.empty((n, H, 128), np.uint8), np.empty((n, H, 128), np.uint8), np.empty((n, H), np.float32)
    orc.lib().orc_quantize_rows(orc._p(Kb), orc._p(Vb), n * H, 128, orc._p(ok), orc._p(ov), orc._p(os_))
    assert np.array_equal(S[0].cpu().numpy(), os_)
    assert np.array_equal(Kc[0].cpu().numpy(), ok) and np.array_equal(Vc[0].cpu().numpy(), ov)


def test_write_fp8_equals_the_bridge(hs2):
    """Rows that hs2_bridge_kv writes, quantised as written: the cache of
    hs2_bridge_kv_fp8, bit for bit."""
    import torch
    T, H, dm = 700, 2, 256
    Hs, Wk, Wv = synth.bridge_inputs_dyadic_np(synth.BlockConfig("cache", 6, T, 8, H, d_model=dm))
    Hs, Wk, Wv = dev_bf16(Hs), dev_bf16(Wk), dev_bf16(Wv)
    shape = hs2.Shape.make(T, 8, H)
    K = torch.empty(T, H, 128, dtype=torch.bfloat16, device="cuda")
    V = torch.empty_like(K)
    hs2.hs2_bridge_kv(Hs, Wk, Wv, K, V, shape)
    want = [torch.empty(1, T, H, 128, dtype=torch.uint8, device="cuda") for _ in range(2)]
    got = [torch.empty_like(want[0]) for _ in range(2)]
    sw, sg = torch.empty(1, T, H, device="cuda"), torch.empty(1, T, H, device="cuda")
    hs2.hs2_bridge_kv_fp8(Hs, Wk, Wv, want[0], want[1], sw, shape)
    hs2.hs2_cache_write_fp8(K, V, None, got[0], got[1], sg, shape)
    assert torch.equal(sw, sg)
    for a, b in zip(want, got):
        # a negative value that rounds to zero keeps its sign on both sides
        assert torch.equal(a, b)


def test_write_fp8_non_finite_rows(hs2):
    import torch
    n, H = 5, 2
    Kb, Vb = awkward_rows(n, H, 13), awkward_rows(n, H, 14)
    Kb[1, 0, 40], Vb[3, 1, 9] = 0x7F80, 0x7FC0
    shape = hs2.Shape.make(n, H, H)
    Kc = torch.full((1, n, H, 128), 0x5A, dtype=torch.uint8, device="cuda")
    Vc, S = torch.full_like(Kc, 0x5A), torch.zeros(1, n, H, device="cuda")
    hs2.hs2_cache_write_fp8(dev_bf16(Kb), dev_bf16(Vb), None, Kc, Vc, S, shape)
    nan = np.zeros((n, H), bool)
    nan[1, 0] = nan[3, 1] = True
    assert np.array_equal(np.isnan(S[0].cpu().numpy()), nan)
    assert not Kc[0].cpu().numpy()[nan].any() and not Vc[0].cpu().numpy()[nan].any()


@pytest.mark.parametrize("fmt", ["q4", "fp8"])
def test_bad_slots_are_skipped_and_reported(hs2, fmt):
    import torch
    n, H, cap, batch = 9, 2, 8, 2
    shape = hs2.Shape.make(cap, H, H)
    K = torch.randn(n, H, 128, device="cuda").bfloat16()
    good = torch.tensor([3, -1, 15, -1, 0, 7, -1, -1, 8], dtype=torch.int32, device="cuda")
    bad = torch.tensor([3, 16, 15, -2, 0, 7, 1 << 30, -(1 << 31), 8], dtype=torch.int32, device="cuda")
    made = []
    for slot in (good, bad):
        if fmt == "q4":
            c = [torch.full((batch, H, cap, 144), 9, dtype=torch.uint8, device="cuda")]
            hs2.hs2_cache_write_q4(K, K, slot, c[0], shape)
        else:
            c = [torch.full((batch, cap, H, 128), 9, dtype=torch.uint8, device="cuda") for _ in range(2)]
            c.append(torch.zeros(batch, cap, H, device="cuda"))
            hs2.hs2_cache_write_fp8(K, K, slot, c[0], c[1], c[2], shape)
        assert hs2.hs2_get_device_status() == (hs2.OK if slot is good else hs2.ERR_BAD_INDEX)
        out = torch.zeros_like(K)
        if fmt == "q4":
            hs2.hs2_cache_read_q4(c[0], slot, out, torch.zeros_like(K), shape)
        else:
            hs2.hs2_cache_read_fp8(c[0], c[1], c[2], c[2], slot, out, torch.zeros_like(K), shape)
        assert hs2.hs2_get_device_status() == (hs2.OK if slot is good else hs2.ERR_BAD_INDEX)
        made.append((*c, out))
    for a, b in zip(*made):
        assert torch.equal(a, b)
    assert hs2.hs2_get_device_status() == hs2.OK


def test_captured_append_replays_with_new_slots(hs2):
    """A captured write and read-back on another stream takes the rows and
    slots of the moment it replays."""
    import torch
    n, H, cap = 4, 2, 32
    shape = hs2.Shape.make(cap, H, H)
    K = torch.zeros(n, H, 128, dtype=torch.bfloat16, device="cuda")
    V, out = torch.zeros_like(K), torch.zeros_like(K)
    vout = torch.zeros_like(K)
    slot = torch.zeros(n, dtype=torch.int32, device="cuda") - 1
    cache = torch.zeros(n, H, cap, 144, dtype=torch.uint8, device="cuda")
    st = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=st):
        hs2.hs2_cache_write_q4(K, V, slot, cache, shape)
        hs2.hs2_cache_read_q4(cache, slot, out, vout, shape)
    for step in range(3):
        Kb, Vb = awkward_rows(n, H, 50 + step), awkward_rows(n, H, 60 + step)
        at = np.arange(n) * cap + 3 * step
        K.copy_(dev_bf16(Kb))
        V.copy_(dev_bf16(Vb))
        slot.copy_(dev(at.astype(np.int32)))
        g.replay()
        torch.cuda.synchronize()
        rec = ref.records(Kb, Vb)
        assert np.array_equal(cache[:, :, 3 * step].cpu().numpy(), rec)
        assert np.array_equal(bits(out), ref.to_bf16_bits(ref.values(rec)[0]))
        assert np.array_equal(bits(vout), ref.to_bf16_bits(ref.values(rec)[1]))
    # an explicit stream argument
    with torch.cuda.stream(st):
        fresh = torch.zeros_like(cache)
    st.synchronize()
    hs2.hs2_cache_write_q4(K, V, slot, fresh, shape, stream=st)
    st.synchronize()
    assert np.array_equal(fresh[:, :, 6].cpu().numpy(), rec)
