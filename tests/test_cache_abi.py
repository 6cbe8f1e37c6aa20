"""Host-side checks of the cache and 4-bit calls (CPU only): every refusal comes
before any launch, and the reference quantiser's own properties hold."""
import ctypes as C

import numpy as np
import pytest

import q4_reference as ref


@pytest.fixture(scope="module")
def hs2():
    import long_context_bridge_b200 as m
    return m


OK, BAD = C.c_void_p(0x10000), C.c_void_p(0x10008)


def test_cache_rows_refusals(hs2):
    L = hs2._lib
    sh = hs2.Shape.make(100, 8, 2)
    r = lambda **k: C.byref(hs2.Shape.make(**{"T": 100, "n_q_heads": 8, "n_kv_heads": 2, **k}))  # noqa: E731

    def w(K=OK, V=OK, ldk=256, ldv=256, slot=None, first=0, n=4, cache=OK, batch=2, s=None):
        return L.hs2_cache_write_q4(K, V, ldk, ldv, slot, first, n, cache, batch,
                                    C.byref(sh) if s is None else s, None)

    INV, UNS = hs2.ERR_INVALID_ARG, hs2.ERR_UNSUPPORTED
    assert w(K=None) == INV and w(V=BAD) == INV and w(cache=None) == INV and w(cache=BAD) == INV
    assert w(ldk=248) == INV and w(ldv=260) == INV            # short rows, rows off 16 bytes
    assert w(n=-1) == INV and w(n=1 << 31) == INV
    assert w(first=-1) == INV and w(first=197) == INV and w(first=201, n=0) == INV
    assert w(slot=C.c_void_p(0x10002)) == INV
    assert w(batch=0) == INV and w(s=r(T=1 << 30), batch=4) == UNS
    assert w(s=r(head_dim=64)) == UNS and w(s=r(T=0)) == INV
    assert w(n=0, K=None, V=None) == hs2.OK                    # nothing to do
    assert w(n=0, first=200) == hs2.OK
    f = lambda Kc=OK, Vc=OK, sc=OK, n=4: L.hs2_cache_write_fp8(  # noqa: E731
        OK, OK, 256, 256, None, 0, n, Kc, Vc, sc, 2, C.byref(sh), None)
    assert f(Kc=BAD) == INV and f(Vc=None) == INV and f(sc=C.c_void_p(0x10001)) == INV
    assert f(n=0) == hs2.OK
    g = lambda ks=OK, K=OK: L.hs2_cache_read_fp8(OK, OK, ks, OK, None, 0, 4, K, OK, 256, 256, 2,  # noqa: E731
                                                 C.byref(sh), None)
    assert g(ks=None) == INV and g(K=BAD) == INV
    assert L.hs2_cache_read_q4(None, None, 0, 4, OK, OK, 256, 256, 2, C.byref(sh), None) == INV


def test_q4_attention_refusals(hs2):
    L = hs2._lib
    sh = hs2.Shape.make(4096, 32, 4)
    need = hs2.workspace_size(hs2.OP_DECODE_ATTN_Q4, sh, 8)
    INV, UNS, WS = hs2.ERR_INVALID_ARG, hs2.ERR_UNSUPPORTED, hs2.ERR_WORKSPACE

    def a(batch=8, lens=OK, q=OK, cache=OK, o=OK, lse=OK, s=sh, ws=OK, n=need):
        return L.hs2_decode_attn_q4(batch, lens, q, cache, o, lse, C.byref(s), ws, n, None)

    assert a(lens=None) == INV and a(q=BAD) == INV and a(cache=BAD) == INV and a(lse=None) == INV
    assert a(lens=C.c_void_p(0x10002)) == INV and a(batch=0) == INV
    assert a(ws=None) == WS and a(n=need - 1) == WS and a(ws=BAD) == WS
    assert a(batch=513, n=1 << 40) == UNS
    assert a(s=hs2.Shape.make(1 << 29, 32, 4), n=1 << 40) == UNS     # batch * T past 2^31 - 1
    assert a(s=hs2.Shape.make(4096, 24, 4), n=1 << 40) == UNS        # G = 6
    with pytest.raises(hs2.HS2Error):
        hs2.workspace_size(hs2.OP_DECODE_ATTN_Q4, sh, 513)
    with pytest.raises(hs2.HS2Error):
        hs2.workspace_size(hs2.OP_BLOCK_DECODE_Q4, sh, 65)

    def p(batch=8, q=OK, cache=OK, idx=OK, o=OK, lse=None, s=sh):
        return L.hs2_sparse_attn_q4(batch, q, cache, idx, o, lse, C.byref(s), None)

    assert p(q=None) == INV and p(idx=C.c_void_p(0x10002)) == INV and p(o=BAD) == INV
    assert p(batch=-1) == INV and p(s=hs2.Shape.make(4096, 32, 4, window=0)) == INV
    assert p(s=hs2.Shape.make(4096, 32, 4, k_global=2049)) == UNS

    nb = hs2.workspace_size(hs2.OP_BLOCK_DECODE_Q4, sh, 2)
    arr = C.cast((C.c_void_p * 1)(0x10001), C.POINTER(C.c_void_p))
    good = C.cast((C.c_void_p * 1)(0x10000), C.POINTER(C.c_void_p))

    def b(lens=(10, 4096), cache=OK, n_sparse=1, qs=good, ws=OK, n=nb, lse=OK):
        return L.hs2_block_decode_q4(2, (C.c_int64 * 2)(*lens), OK, cache, OK, lse, OK, n_sparse, qs,
                                     good, C.byref(sh), ws, n, None)

    assert b(lens=(0, 5)) == INV and b(lens=(5, 4097)) == INV and b(cache=None) == INV
    assert b(qs=arr) == INV and b(n_sparse=-1) == INV and b(n=nb - 1) == WS and b(lse=BAD) == INV


def test_binding_refusals(hs2):
    """The binding checks devices, types and shapes before it calls."""
    import torch
    sh = hs2.Shape.make(16, 8, 2)
    x = torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    c = torch.zeros(1, 2, 16, 144, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        hs2.hs2_cache_write_q4(x, x, None, c, sh)
    with pytest.raises(ValueError, match="CUDA"):
        hs2.hs2_sparse_attn_q4(x, c, None, x, None, sh)
    with pytest.raises(ValueError, match="CUDA"):
        hs2.hs2_cache_read_fp8(None, c, x, x, None, x, x, sh)


def test_reference_layout_is_a_permutation():
    assert sorted(ref.NIB_K) == list(range(128)) and sorted(ref.NIB_V) == list(range(128))


def test_reference_quantiser_rounding():
    """Codes within [-7, 7], each value within half a step of the input, exact
    ties to the even code, the floor of the scale, non-finite groups."""
    rng = np.random.default_rng(5)
    x = rng.standard_normal((64, 128)) * np.exp2(rng.integers(-20, 20, (64, 1)))
    b = ref.to_bf16_bits(x)
    c, s = ref.quantise(b)
    v, _ = ref.values(ref.records(b, b))
    step = np.repeat(ref.from_bf16_bits(s), 32, -1)
    assert c.min() >= -7 and c.max() <= 7
    # the scale is amax / 7 rounded down by at most 2^-8 of it: 7 steps then fall short
    # of the largest |x| by at most 7 * 2^-8 of a step, less than half of one
    assert np.all(np.abs(v - ref.from_bf16_bits(b)) <= 0.5 * step)
    t = np.zeros((1, 128))
    t[0, :4] = [7.0, 2.5, -3.5, 0.5]                      # scale exactly 1
    c, s = ref.quantise(ref.to_bf16_bits(t))
    assert list(c[0, :4]) == [7, 2, -4, 0] and s[0, 0] == 0x3F80
    t[0, :4] = [1e-38, 0, np.inf, 0]
    c, s = ref.quantise(ref.to_bf16_bits(t))
    assert s[0, 0] == 0x7FC0 and not c.any() and s[0, 1] == 0x0380  # 2^-120
