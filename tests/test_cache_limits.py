"""Limits of the cache and 4-bit calls that the header states (CPU only: they
are refused before any launch)."""
import ctypes as C

import pytest


@pytest.fixture(scope="module")
def hs2():
    import long_context_bridge_b200 as m
    return m


OK = C.c_void_p(0x10000)


@pytest.mark.parametrize("T,Hkv,batch", [(1, 65536, 1), ((1 << 31) - 1, 1, 2), (1 << 28, 4, 8)])
def test_sizes_past_the_limits_are_refused(hs2, T, Hkv, batch):
    L, UNS = hs2._lib, hs2.ERR_UNSUPPORTED
    sh = hs2.Shape.make(T, Hkv, Hkv, k_global=1, window=1)
    s, ld, big = C.byref(sh), Hkv * 128, 1 << 60
    lens = (C.c_int64 * batch)(*[1] * batch)
    assert L.hs2_cache_write_q4(OK, OK, ld, ld, None, 0, 1, OK, batch, s, None) == UNS
    assert L.hs2_cache_read_q4(OK, None, 0, 1, OK, OK, ld, ld, batch, s, None) == UNS
    assert L.hs2_cache_write_fp8(OK, OK, ld, ld, None, 0, 1, OK, OK, OK, batch, s, None) == UNS
    assert L.hs2_cache_read_fp8(OK, OK, OK, OK, None, 0, 1, OK, OK, ld, ld, batch, s, None) == UNS
    assert L.hs2_decode_attn_q4(batch, OK, OK, OK, OK, OK, s, OK, big, None) == UNS
    assert L.hs2_sparse_attn_q4(batch, OK, OK, OK, OK, None, s, None) == UNS
    assert L.hs2_block_decode_q4(batch, lens, OK, OK, OK, OK, OK, 0, None, None, s, OK, big, None) == UNS
    for op in (hs2.OP_DECODE_ATTN_Q4, hs2.OP_BLOCK_DECODE_Q4):
        with pytest.raises(hs2.HS2Error):
            hs2.workspace_size(op, sh, batch)
