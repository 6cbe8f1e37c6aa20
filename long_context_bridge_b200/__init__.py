"""Python binding of libhs2 (the HySparse2 cross-decoder block for B200).

Argument marshalling only: every function checks tensor dtypes, devices and
contiguity, then calls the C entry point of the same name with raw device
pointers and the current CUDA stream.  All computation runs in the library's
CUDA kernels.  There is no fallback: if ``libhs2.so`` is missing or fails to
load, importing this package raises.
"""
from __future__ import annotations

import ctypes as C
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libhs2.so")

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_WORKSPACE, ERR_CUDA, ERR_TIMEOUT, ERR_BAD_INDEX = range(7)
(OP_BRIDGE, OP_FULL_ATTN, OP_SELECT, OP_SPARSE, OP_BLOCK_PREFILL, OP_BLOCK_DECODE, OP_SPARSE_PLAN,
 OP_DECODE_ATTN_Q4, OP_BLOCK_DECODE_Q4) = range(9)
Q4_RECORD_BYTES = 144   # one token's K and V of one KV head in the 4-bit cache


class HS2Error(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {_lib.hs2_status_string(status).decode()} (status {status})")
        self.status = status


class Shape(C.Structure):
    """hs2_shape: T, n_q_heads, n_kv_heads, head_dim, scale, k_global, window."""
    _fields_ = [("T", C.c_int64), ("n_q_heads", C.c_int32), ("n_kv_heads", C.c_int32),
                ("head_dim", C.c_int32), ("scale", C.c_float), ("k_global", C.c_int32),
                ("window", C.c_int32)]

    @classmethod
    def make(cls, T, n_q_heads, n_kv_heads, head_dim=128, scale=None, k_global=1024, window=128):
        if scale is None:
            scale = head_dim ** -0.5
        return cls(int(T), int(n_q_heads), int(n_kv_heads), int(head_dim), float(scale),
                   int(k_global), int(window))


def _load(path: str = LIB_PATH):
    if not os.path.exists(path):
        raise ImportError(f"libhs2.so not built at {path}: run long_context_bridge_b200/build.py")
    L = C.CDLL(path)
    P, I32, I64, SZ = C.c_void_p, C.c_int32, C.c_int64, C.c_size_t
    SP = C.POINTER(Shape)
    PP = C.POINTER(C.c_void_p)
    sigs = {
        "hs2_bridge_kv": [P, I32, P, P, P, P, SP, P],
        "hs2_bridge_kv_fp8": [P, I32, P, P, P, P, P, SP, P],
        "hs2_full_attn_lse": [P, P, P, P, P, SP, P],
        "hs2_select_topk": [P, P, P, P, P, SP, P, SZ, P],
        "hs2_select_topk_noalloc": [P, P, P, P, P, SP, P],
        "hs2_sparse_attn": [P, P, P, P, P, P, SP, P],
        "hs2_sparse_attn_layers": [I32, PP, P, P, P, PP, PP, SP, P],
        "hs2_sparse_plan": [P, SP, P, SZ, P],
        "hs2_sparse_attn_planned": [P, P, P, P, P, P, SP, P],
        "hs2_block_prefill": [P, I32, P, P, P, P, P, P, P, P, I32, PP, PP, SP, P, SZ, P],
        "hs2_block_decode": [I32, C.POINTER(C.c_int64), P, P, P, P, P, P, P, P, I32, PP, PP, SP,
                             P, SZ, P],
        "hs2_block_prefill_rows": [I64, P, P, P, P, P, P, I32, PP, PP, SP, P, SZ, P],
        "hs2_debug_read_probe": [P, SZ, I32, P, P],
        "hs2_debug_set_select_speculation": [C.c_float],
        "hs2_decode_cp_attn": [I32, C.POINTER(C.c_int64), C.POINTER(C.c_int64),
                               C.POINTER(C.c_int64), P, P, P, P, P, P, SP, P, SZ, P],
        "hs2_decode_cp_select": [I32, C.POINTER(C.c_int64), C.POINTER(C.c_int64),
                                 C.POINTER(C.c_int64), I32, P, P, P, P, SP, P, SZ, P],
        "hs2_decode_cp_sparse": [I32, C.POINTER(C.c_int64), C.POINTER(C.c_int64),
                                 C.POINTER(C.c_int64), I32, P, P, P, P, P, P, I32, PP, P, SP, P],
        "hs2_decode_cp_finish": [I32, I32, I32, P, PP, SP, P],
        "hs2_cache_write_fp8": [P, P, I64, I64, P, I64, I64, P, P, P, I32, SP, P],
        "hs2_cache_read_fp8": [P, P, P, P, P, I64, I64, P, P, I64, I64, I32, SP, P],
        "hs2_cache_write_q4": [P, P, I64, I64, P, I64, I64, P, I32, SP, P],
        "hs2_cache_read_q4": [P, P, I64, I64, P, P, I64, I64, I32, SP, P],
        "hs2_decode_attn_q4": [I32, P, P, P, P, P, SP, P, SZ, P],
        "hs2_sparse_attn_q4": [I32, P, P, P, P, P, SP, P],
        "hs2_block_decode_q4": [I32, C.POINTER(C.c_int64), P, P, P, P, P, I32, PP, PP, SP, P, SZ,
                                P],
    }
    for name, args in sigs.items():
        fn = getattr(L, name)
        fn.argtypes = args
        fn.restype = C.c_int
    L.hs2_workspace_size.argtypes = [I32, SP, I32, I32]
    L.hs2_workspace_size.restype = SZ
    L.hs2_get_device_status.argtypes = [P]
    L.hs2_get_device_status.restype = C.c_int
    L.hs2_status_string.argtypes = [C.c_int]
    L.hs2_status_string.restype = C.c_char_p
    L.hs2_kernel_launches.restype = C.c_uint64
    L.hs2_debug_set_wait_budget.argtypes = [C.c_int64]
    L.hs2_debug_set_wait_budget.restype = C.c_int
    return L


_lib = _load()

EXPORTED = ["hs2_bridge_kv", "hs2_bridge_kv_fp8", "hs2_full_attn_lse", "hs2_select_topk", "hs2_select_topk_noalloc",
            "hs2_sparse_attn", "hs2_sparse_attn_layers", "hs2_sparse_plan", "hs2_sparse_attn_planned",
            "hs2_block_prefill", "hs2_block_decode", "hs2_workspace_size",
            "hs2_get_device_status", "hs2_status_string", "hs2_kernel_launches",
            "hs2_debug_set_wait_budget", "hs2_debug_read_probe", "hs2_block_prefill_rows",
            "hs2_debug_set_select_speculation",
            "hs2_decode_cp_attn",
            "hs2_decode_cp_select",
            "hs2_decode_cp_sparse", "hs2_decode_cp_finish",
            "hs2_cache_write_fp8", "hs2_cache_read_fp8", "hs2_cache_write_q4",
            "hs2_cache_read_q4", "hs2_decode_attn_q4", "hs2_sparse_attn_q4",
            "hs2_block_decode_q4"]


def _ptr(t, dtype, what, nullable=False):
    if t is None:
        if nullable:
            return None
        raise ValueError(f"{what} is required")
    if not isinstance(t, torch.Tensor) or t.device.type != "cuda":
        raise ValueError(f"{what} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{what} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    return C.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        return C.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, torch.cuda.Stream):
        return C.c_void_p(stream.cuda_stream)
    return C.c_void_p(int(stream))


def _check(status, what):
    if status != OK:
        raise HS2Error(status, what)


BF16, F32, I32T, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


def workspace_size(op: int, shape: Shape, batch: int = 1, d_model: int = 0) -> int:
    n = _lib.hs2_workspace_size(op, C.byref(shape), batch, d_model)
    if n == C.c_size_t(-1).value:
        raise HS2Error(ERR_INVALID_ARG, "hs2_workspace_size")
    return int(n)


def hs2_bridge_kv(H, W_k, W_v, K, V, shape: Shape, stream=None):
    _check(_lib.hs2_bridge_kv(_ptr(H, BF16, "H"), H.shape[-1], _ptr(W_k, BF16, "W_k"),
                              _ptr(W_v, BF16, "W_v"), _ptr(K, BF16, "K"), _ptr(V, BF16, "V"),
                              C.byref(shape), _stream(stream)), "hs2_bridge_kv")


def hs2_bridge_kv_fp8(H, W_k, W_v, Kc, Vc, scale, shape: Shape, stream=None):
    _check(_lib.hs2_bridge_kv_fp8(_ptr(H, BF16, "H"), H.shape[-1], _ptr(W_k, BF16, "W_k"),
                                  _ptr(W_v, BF16, "W_v"), _ptr(Kc, U8, "Kc"), _ptr(Vc, U8, "Vc"),
                                  _ptr(scale, F32, "scale"), C.byref(shape), _stream(stream)),
           "hs2_bridge_kv_fp8")


def hs2_full_attn_lse(Q, K, V, O, lse, shape: Shape, stream=None):
    _check(_lib.hs2_full_attn_lse(_ptr(Q, BF16, "Q"), _ptr(K, BF16, "K"), _ptr(V, BF16, "V"),
                                  _ptr(O, BF16, "O"), _ptr(lse, F32, "lse"), C.byref(shape),
                                  _stream(stream)), "hs2_full_attn_lse")


def hs2_select_topk(Q, K, lse, idx, kth, shape: Shape, workspace, stream=None):
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib.hs2_select_topk(_ptr(Q, BF16, "Q"), _ptr(K, BF16, "K"), _ptr(lse, F32, "lse"),
                                _ptr(idx, I32T, "idx"), _ptr(kth, F32, "kth", True),
                                C.byref(shape), _ptr(workspace, U8, "workspace", True), nbytes,
                                _stream(stream)), "hs2_select_topk")


def hs2_select_topk_noalloc(Q, K, lse, idx, kth, shape: Shape, stream=None):
    """hs2_select_topk on the library's own scratch, for callers that cannot
    allocate device memory; see include/hs2.h for its limits."""
    _check(_lib.hs2_select_topk_noalloc(_ptr(Q, BF16, "Q"), _ptr(K, BF16, "K"),
                                        _ptr(lse, F32, "lse"), _ptr(idx, I32T, "idx"),
                                        _ptr(kth, F32, "kth", True), C.byref(shape),
                                        _stream(stream)), "hs2_select_topk_noalloc")


def hs2_sparse_attn(Q, K, V, idx, O, lse, shape: Shape, stream=None):
    _check(_lib.hs2_sparse_attn(_ptr(Q, BF16, "Q"), _ptr(K, BF16, "K"), _ptr(V, BF16, "V"),
                                _ptr(idx, I32T, "idx"), _ptr(O, BF16, "O"),
                                _ptr(lse, F32, "lse", True), C.byref(shape), _stream(stream)),
           "hs2_sparse_attn")


def hs2_sparse_plan(idx, shape: Shape, plan, stream=None):
    nbytes = plan.numel() * plan.element_size()
    _check(_lib.hs2_sparse_plan(_ptr(idx, I32T, "idx"), C.byref(shape), _ptr(plan, U8, "plan"),
                                nbytes, _stream(stream)), "hs2_sparse_plan")


def hs2_sparse_attn_planned(Q, K, V, plan, O, lse, shape: Shape, stream=None):
    _check(_lib.hs2_sparse_attn_planned(_ptr(Q, BF16, "Q"), _ptr(K, BF16, "K"), _ptr(V, BF16, "V"),
                                        _ptr(plan, U8, "plan"), _ptr(O, BF16, "O"),
                                        _ptr(lse, F32, "lse", True), C.byref(shape),
                                        _stream(stream)), "hs2_sparse_attn_planned")


def _ptr_array(ts, dtype, what):
    arr = (C.c_void_p * max(1, len(ts)))()
    for i, t in enumerate(ts):
        arr[i] = _ptr(t, dtype, f"{what}[{i}]").value
    return C.cast(arr, C.POINTER(C.c_void_p)), arr


def hs2_sparse_attn_layers(Qs, K, V, idx, Os, lses, shape: Shape, stream=None):
    qs, _keep_q = _ptr_array(Qs, BF16, "Q")
    os_, _keep_o = _ptr_array(Os, BF16, "O")
    ls = None
    if lses is not None:
        ls = (C.c_void_p * max(1, len(lses)))(*[_ptr(t, F32, "lse", True) for t in lses])
    _check(_lib.hs2_sparse_attn_layers(len(Qs), qs, _ptr(K, BF16, "K"), _ptr(V, BF16, "V"),
                                       _ptr(idx, I32T, "idx"), os_, ls, C.byref(shape),
                                       _stream(stream)), "hs2_sparse_attn_layers")


def hs2_block_prefill(H, W_k, W_v, K, V, Q_full, O_full, lse, idx, Q_sparse, O_sparse,
                      shape: Shape, workspace, stream=None):
    qs, _keep_q = _ptr_array(Q_sparse, BF16, "Q_sparse")
    os_, _keep_o = _ptr_array(O_sparse, BF16, "O_sparse")
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib.hs2_block_prefill(
        _ptr(H, BF16, "H", True), 0 if H is None else H.shape[-1], _ptr(W_k, BF16, "W_k", True),
        _ptr(W_v, BF16, "W_v", True), _ptr(K, BF16, "K"), _ptr(V, BF16, "V"),
        _ptr(Q_full, BF16, "Q_full"), _ptr(O_full, BF16, "O_full"), _ptr(lse, F32, "lse"),
        _ptr(idx, I32T, "idx"), len(Q_sparse), qs, os_, C.byref(shape),
        _ptr(workspace, U8, "workspace", True), nbytes, _stream(stream)), "hs2_block_prefill")


def hs2_block_prefill_rows(q_begin, K, V, Q_full, O_full, lse, idx, Q_sparse, O_sparse,
                           shape: Shape, workspace, stream=None):
    qs, _keep_q = _ptr_array(Q_sparse, BF16, "Q_sparse")
    os_, _keep_o = _ptr_array(O_sparse, BF16, "O_sparse")
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib.hs2_block_prefill_rows(
        int(q_begin), _ptr(K, BF16, "K"), _ptr(V, BF16, "V"), _ptr(Q_full, BF16, "Q_full"),
        _ptr(O_full, BF16, "O_full"), _ptr(lse, F32, "lse"), _ptr(idx, I32T, "idx"),
        len(Q_sparse), qs, os_, C.byref(shape), _ptr(workspace, U8, "workspace", True), nbytes,
        _stream(stream)), "hs2_block_prefill_rows")


def hs2_block_decode(seq_len, q_full, Kc, Vc, k_scale, v_scale, o_full, lse, idx, q_sparse,
                     o_sparse, shape: Shape, workspace, stream=None):
    B = len(seq_len)
    lens = (C.c_int64 * B)(*[int(x) for x in seq_len])
    qs, _keep_q = _ptr_array(q_sparse, BF16, "q_sparse")
    os_, _keep_o = _ptr_array(o_sparse, BF16, "o_sparse")
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib.hs2_block_decode(
        B, lens, _ptr(q_full, BF16, "q_full"), _ptr(Kc, U8, "Kc"), _ptr(Vc, U8, "Vc"),
        _ptr(k_scale, F32, "k_scale"), _ptr(v_scale, F32, "v_scale"), _ptr(o_full, BF16, "o_full"),
        _ptr(lse, F32, "lse"), _ptr(idx, I32T, "idx"), len(q_sparse), qs, os_, C.byref(shape),
        _ptr(workspace, U8, "workspace", True), nbytes, _stream(stream)), "hs2_block_decode")



def _i64s(xs):
    return (C.c_int64 * len(xs))(*[int(x) for x in xs])


DECODE_REC_FLOATS = 130   # softmax-state record: m, l, o[128]


def hs2_decode_cp_attn(seq_len, slice_lo, slice_hi, q_full, Kc, Vc, k_scale, v_scale, attn_rec,
                       shape: Shape, workspace, stream=None):
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib.hs2_decode_cp_attn(
        len(seq_len), _i64s(seq_len), _i64s(slice_lo), _i64s(slice_hi),
        _ptr(q_full, BF16, "q_full"), _ptr(Kc, U8, "Kc"), _ptr(Vc, U8, "Vc"),
        _ptr(k_scale, F32, "k_scale"), _ptr(v_scale, F32, "v_scale"),
        _ptr(attn_rec, F32, "attn_rec"), C.byref(shape), _ptr(workspace, U8, "workspace", True),
        nbytes, _stream(stream)), "hs2_decode_cp_attn")


def hs2_decode_cp_select(seq_len, slice_lo, slice_hi, n_ranks, attn_recs, o_full, lse, sel_rec,
                         shape: Shape, workspace, stream=None):
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib.hs2_decode_cp_select(
        len(seq_len), _i64s(seq_len), _i64s(slice_lo), _i64s(slice_hi), int(n_ranks),
        _ptr(attn_recs, F32, "attn_recs"), _ptr(o_full, BF16, "o_full"), _ptr(lse, F32, "lse"),
        _ptr(sel_rec, I32T, "sel_rec"), C.byref(shape), _ptr(workspace, U8, "workspace", True),
        nbytes, _stream(stream)), "hs2_decode_cp_select")


def hs2_decode_cp_sparse(seq_len, slice_lo, slice_hi, n_ranks, sel_recs, idx, Kc, Vc, k_scale,
                         v_scale, q_sparse, sparse_rec, shape: Shape, stream=None):
    qs, _keep_q = _ptr_array(q_sparse, BF16, "q_sparse")
    _check(_lib.hs2_decode_cp_sparse(
        len(seq_len), _i64s(seq_len), _i64s(slice_lo), _i64s(slice_hi), int(n_ranks),
        _ptr(sel_recs, I32T, "sel_recs"), _ptr(idx, I32T, "idx"), _ptr(Kc, U8, "Kc"),
        _ptr(Vc, U8, "Vc"), _ptr(k_scale, F32, "k_scale"), _ptr(v_scale, F32, "v_scale"),
        len(q_sparse), qs, _ptr(sparse_rec, F32, "sparse_rec", True), C.byref(shape),
        _stream(stream)), "hs2_decode_cp_sparse")


def hs2_decode_cp_finish(n_ranks, sparse_recs, o_sparse, shape: Shape, stream=None):
    os_, _keep_o = _ptr_array(o_sparse, BF16, "o_sparse")
    batch = o_sparse[0].shape[0]
    _check(_lib.hs2_decode_cp_finish(batch, int(n_ranks), len(o_sparse),
                                     _ptr(sparse_recs, F32, "sparse_recs"), os_, C.byref(shape),
                                     _stream(stream)), "hs2_decode_cp_finish")


# ---------------------------------------------------------------------------
# rows into and out of a decode cache; the 4-bit cache
# ---------------------------------------------------------------------------
# These calls run once per decode step and layer, so their marshalling is kept
# short: pointers as plain ints, one pass of checks per tensor, and the device
# is only switched when the tensors do not live on the current one.
def _on(t, dtype, what, dev):
    """Checked device pointer of a dense tensor on device index `dev` (a CPU
    tensor's index is -1)."""
    if isinstance(t, torch.Tensor):
        if t.dtype is dtype and t.get_device() == dev and t.is_contiguous():
            return t.data_ptr()
        if not t.is_cuda:
            raise ValueError(f"{what} must be a CUDA tensor")
        if t.dtype is not dtype:
            raise ValueError(f"{what} must be {dtype}, got {t.dtype}")
        if t.get_device() != dev:
            raise ValueError(f"{what} is on cuda:{t.get_device()}, the cache on cuda:{dev}")
        raise ValueError(f"{what} must be contiguous")
    raise ValueError(f"{what} must be a CUDA tensor")


def _shaped(t, shape, what):
    try:
        size = t.shape
    except AttributeError:
        raise ValueError(f"{what} must be a CUDA tensor") from None
    if size != shape:
        raise ValueError(f"{what} must be {shape}, got {tuple(size)}")


def _run(fn, what, dev, stream, args):
    """fn(*args, stream) with device `dev` current, on `stream` or, where that
    is None, on that device's current stream."""
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(dev)  # .current_stream(dev).cuda_stream
    elif isinstance(stream, torch.cuda.Stream):
        stream = stream.cuda_stream
    if torch._C._cuda_getDevice() == dev:  # the tensors' existence implies initialised CUDA
        status = fn(*args, stream)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, stream)
    if status != OK:
        raise HS2Error(status, what)


def _rows(t, n, n_heads, what, dev):
    """Pointer and token stride of K or V rows [n, n_kv_heads, 128] bf16, dense
    but for that stride."""
    if isinstance(t, torch.Tensor):
        if t.dtype is BF16 and t.get_device() == dev and t.shape == (n, n_heads, 128):
            ld, head, dim = t.stride()
            if n == 0 or (dim == 1 and (head == 128 or n_heads == 1)):
                return t.data_ptr(), ld if n > 1 else n_heads * 128
            raise ValueError(f"the heads of {what} must be dense (strides [ld, 128, 1])")
        if not t.is_cuda:
            raise ValueError(f"{what} must be a CUDA tensor")
        if t.dtype is not BF16:
            raise ValueError(f"{what} must be {BF16}, got {t.dtype}")
        if t.get_device() != dev:
            raise ValueError(f"{what} is on cuda:{t.get_device()}, the cache on cuda:{dev}")
        raise ValueError(f"{what} must be [{n}, {n_heads}, 128], got {tuple(t.shape)}")
    raise ValueError(f"{what} must be a CUDA tensor")


def _row_args(K, V, slot, n_heads, dev):
    try:
        n = len(K)
    except TypeError:  # no tensor, or one without rows: _rows says so
        n = 0
    k, ldk = _rows(K, n, n_heads, "K", dev)
    v, ldv = _rows(V, n, n_heads, "V", dev)
    if slot is not None:
        _shaped(slot, (n,), "slot")
        slot = _on(slot, I32T, "slot", dev)
    return k, v, ldk, ldv, slot, n


def _q4_cache(cache, shape):
    """Device index, pointer and batch of a 4-bit cache [batch, n_kv_heads, T, 144]."""
    if not isinstance(cache, torch.Tensor) or not cache.is_cuda:
        raise ValueError("cache must be a CUDA tensor")
    dev, size = cache.get_device(), cache.shape
    batch = size[0] if size else 0
    if size != (batch, shape.n_kv_heads, shape.T, Q4_RECORD_BYTES):
        raise ValueError(f"cache must be [batch, {shape.n_kv_heads}, {shape.T}, {Q4_RECORD_BYTES}],"
                         f" got {tuple(size)}")
    return dev, _on(cache, U8, "cache", dev), batch


def _fp8_cache(Kc, Vc, scales, shape):
    """Device index, batch and pointers of an e4m3 cache and its scales."""
    if not isinstance(Kc, torch.Tensor) or not Kc.is_cuda:
        raise ValueError("Kc must be a CUDA tensor")
    dev, size = Kc.get_device(), Kc.shape
    batch = size[0] if size else 0
    rows = (batch, shape.T, shape.n_kv_heads)
    codes = (*rows, 128)
    _shaped(Kc, codes, "Kc")
    _shaped(Vc, codes, "Vc")
    ptrs = [_on(Kc, U8, "Kc", dev), _on(Vc, U8, "Vc", dev)]
    for s in scales:
        _shaped(s, rows, "scale")
        ptrs.append(_on(s, F32, "scale", dev))
    return dev, batch, ptrs


def hs2_cache_write_q4(K, V, slot, cache, shape: Shape, first=0, stream=None):
    """Quantises rows K, V [n, n_kv_heads, 128] (any token stride) into the
    4-bit cache [batch, n_kv_heads, T, 144] at slot [n] int32, or (slot None)
    at first, first + 1, ...; see include/hs2.h."""
    dev, c, batch = _q4_cache(cache, shape)
    k, v, ldk, ldv, sl, n = _row_args(K, V, slot, shape.n_kv_heads, dev)
    _run(_lib.hs2_cache_write_q4, "hs2_cache_write_q4", dev, stream,
         (k, v, ldk, ldv, sl, int(first), n, c, batch, C.byref(shape)))


def hs2_cache_read_q4(cache, slot, K, V, shape: Shape, first=0, stream=None):
    """Cache rows (slots as in hs2_cache_write_q4) as bf16 into K, V; a row
    whose slot is -1 stays as it was."""
    dev, c, batch = _q4_cache(cache, shape)
    k, v, ldk, ldv, sl, n = _row_args(K, V, slot, shape.n_kv_heads, dev)
    _run(_lib.hs2_cache_read_q4, "hs2_cache_read_q4", dev, stream,
         (c, sl, int(first), n, k, v, ldk, ldv, batch, C.byref(shape)))


def hs2_cache_write_fp8(K, V, slot, Kc, Vc, scale, shape: Shape, first=0, stream=None):
    """The e4m3 form of hs2_cache_write_q4: codes Kc, Vc [batch, T, n_kv_heads,
    128] and one fp32 scale per (token, KV head), the cache of hs2_block_decode."""
    dev, batch, ptrs = _fp8_cache(Kc, Vc, (scale,), shape)
    k, v, ldk, ldv, sl, n = _row_args(K, V, slot, shape.n_kv_heads, dev)
    _run(_lib.hs2_cache_write_fp8, "hs2_cache_write_fp8", dev, stream,
         (k, v, ldk, ldv, sl, int(first), n, *ptrs, batch, C.byref(shape)))


def hs2_cache_read_fp8(Kc, Vc, k_scale, v_scale, slot, K, V, shape: Shape, first=0, stream=None):
    """The e4m3 form of hs2_cache_read_q4."""
    dev, batch, ptrs = _fp8_cache(Kc, Vc, (k_scale, v_scale), shape)
    k, v, ldk, ldv, sl, n = _row_args(K, V, slot, shape.n_kv_heads, dev)
    _run(_lib.hs2_cache_read_fp8, "hs2_cache_read_fp8", dev, stream,
         (*ptrs, sl, int(first), n, k, v, ldk, ldv, batch, C.byref(shape)))


def _workspace(ws, dev):
    return (None, 0) if ws is None else (_on(ws, U8, "workspace", dev), ws.numel())


def hs2_decode_attn_q4(seq_len, q, cache, o, lse, shape: Shape, workspace, stream=None):
    """Attention of one new token per sequence over the 4-bit cache, with its
    lse; seq_len is a device int32 [batch] tensor read when the call runs."""
    dev, c, batch = _q4_cache(cache, shape)
    heads = (batch, shape.n_q_heads, 128)
    _shaped(seq_len, (batch,), "seq_len")
    _shaped(q, heads, "q")
    _shaped(o, heads, "o")
    _shaped(lse, heads[:2], "lse")
    _run(_lib.hs2_decode_attn_q4, "hs2_decode_attn_q4", dev, stream,
         (batch, _on(seq_len, I32T, "seq_len", dev), _on(q, BF16, "q", dev), c,
          _on(o, BF16, "o", dev), _on(lse, F32, "lse", dev), C.byref(shape),
          *_workspace(workspace, dev)))


def hs2_sparse_attn_q4(q, cache, idx, o, lse, shape: Shape, stream=None):
    """Attention of one new token per sequence over the positions in idx
    [batch, n_kv_heads, k_global + window] of the 4-bit cache; lse may be None."""
    dev, c, batch = _q4_cache(cache, shape)
    heads = (batch, shape.n_q_heads, 128)
    _shaped(q, heads, "q")
    _shaped(o, heads, "o")
    _shaped(idx, (batch, shape.n_kv_heads, shape.k_global + shape.window), "idx")
    if lse is not None:
        _shaped(lse, heads[:2], "lse")
        lse = _on(lse, F32, "lse", dev)
    _run(_lib.hs2_sparse_attn_q4, "hs2_sparse_attn_q4", dev, stream,
         (batch, _on(q, BF16, "q", dev), c, _on(idx, I32T, "idx", dev), _on(o, BF16, "o", dev), lse,
          C.byref(shape)))


def hs2_block_decode_q4(seq_len, q_full, cache, o_full, lse, idx, q_sparse, o_sparse, shape: Shape,
                        workspace, stream=None):
    """hs2_block_decode over the 4-bit cache; seq_len is a host sequence of ints."""
    dev, c, batch = _q4_cache(cache, shape)
    layers = len(q_sparse)
    if len(seq_len) != batch or len(o_sparse) != layers:
        raise ValueError("seq_len must hold one length per sequence, o_sparse one output per layer")
    heads = (batch, shape.n_q_heads, 128)
    qs, os_ = (C.c_void_p * max(1, layers))(), (C.c_void_p * max(1, layers))()
    for l in range(layers):
        _shaped(q_sparse[l], heads, "q_sparse")
        _shaped(o_sparse[l], heads, "o_sparse")
        qs[l], os_[l] = _on(q_sparse[l], BF16, "q_sparse", dev), _on(o_sparse[l], BF16, "o_sparse", dev)
    _shaped(q_full, heads, "q_full")
    _shaped(o_full, heads, "o_full")
    _shaped(lse, heads[:2], "lse")
    _shaped(idx, (batch, shape.n_kv_heads, shape.k_global + shape.window), "idx")
    PP = C.POINTER(C.c_void_p)
    _run(_lib.hs2_block_decode_q4, "hs2_block_decode_q4", dev, stream,
         (batch, _i64s(seq_len), _on(q_full, BF16, "q_full", dev), c,
          _on(o_full, BF16, "o_full", dev), _on(lse, F32, "lse", dev), _on(idx, I32T, "idx", dev),
          layers, C.cast(qs, PP), C.cast(os_, PP), C.byref(shape), *_workspace(workspace, dev)))


def hs2_get_device_status(stream=None) -> int:
    return int(_lib.hs2_get_device_status(_stream(stream)))


def hs2_debug_set_wait_budget(cycles: int) -> None:
    """Testing hook: spin budget of the kernels' bounded waits (<= 0: default)."""
    _check(_lib.hs2_debug_set_wait_budget(int(cycles)), "hs2_debug_set_wait_budget")


def hs2_debug_read_probe(buf, reps: int, sink, stream=None) -> None:
    """Measurement hook: `reps` passes of 16-byte loads over the uint8 buffer."""
    _check(_lib.hs2_debug_read_probe(_ptr(buf, U8, "buf"), buf.numel(), int(reps),
                                     _ptr(sink, I32T, "sink"), _stream(stream)),
           "hs2_debug_read_probe")


def hs2_debug_set_select_speculation(factor: float) -> None:
    """Testing hook: starting fraction of the selection's speculative floor."""
    _check(_lib.hs2_debug_set_select_speculation(float(factor)),
           "hs2_debug_set_select_speculation")


def hs2_kernel_launches() -> int:
    return int(_lib.hs2_kernel_launches())


def hs2_status_string(status: int) -> str:
    return _lib.hs2_status_string(status).decode()
