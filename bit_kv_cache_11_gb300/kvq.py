"""Thin Python binding of the C ABI in ``include/kvq.h`` (argument marshalling
only: every step of the path runs in the CUDA library ``libkvq.so``).

The functions carry the C names.  Device arguments are torch CUDA tensors (or
raw device addresses as ints); streams default to torch's current stream.
Importing this module raises if the library has not been built — there is no
CPU fallback.
"""
from __future__ import annotations

import ctypes
import os

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libkvq.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"CUDA library not built: {LIB_PATH} is missing. Build it with "
        "`python -c \"import __graft_entry__ as g; g.build()\"` or "
        "`python -m bit_kv_cache_11_gb300.build`.")

_lib = ctypes.CDLL(LIB_PATH)

KVQ_OK = 0
KVQ_ERR_INVALID_ARG = 1
KVQ_ERR_UNSUPPORTED = 2
KVQ_ERR_CAPACITY = 3
KVQ_ERR_OOM = 4
KVQ_ERR_CUDA = 5
KVQ_ERR_DEVICE_CHECK = 6
KVQ_DTYPE_FP16 = 0
KVQ_DTYPE_BF16 = 1
KVQ_PAGED_ERR_WAIT = 1
KVQ_PAGED_ERR_BAD_PAGE = 2
KVQ_PAGED_ERR_NO_PAGES = 4
KVQ_PAGED_ERR_LENGTH = 8
KVQ_PAGED_ERR_NONFINITE = 16
KVQ_AXIS_CHANNEL = 0
KVQ_AXIS_TOKEN = 1


class kvq_config(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int), ("n_q_heads", ctypes.c_int), ("n_kv_heads", ctypes.c_int),
                ("head_dim", ctypes.c_int), ("max_ctx", ctypes.c_int), ("bits_k", ctypes.c_int),
                ("bits_v", ctypes.c_int), ("group", ctypes.c_int), ("axis_k", ctypes.c_int),
                ("axis_v", ctypes.c_int), ("keys_pre_rope", ctypes.c_int), ("rope_base", ctypes.c_float),
                ("n_sink", ctypes.c_int), ("residual", ctypes.c_int), ("fp8", ctypes.c_int),
                ("n_outliers", ctypes.c_int)]


class kvq_buffers(ctypes.Structure):
    _fields_ = [("blocks", ctypes.c_void_p), ("k_tail", ctypes.c_void_p), ("v_tail", ctypes.c_void_p),
                ("block_bytes", ctypes.c_size_t), ("off_kc", ctypes.c_size_t),
                ("off_km", ctypes.c_size_t), ("off_vc", ctypes.c_size_t), ("off_vm", ctypes.c_size_t),
                ("blocks_per_pair", ctypes.c_int), ("n_pairs", ctypes.c_int), ("T_q", ctypes.c_int),
                ("T_tail", ctypes.c_int), ("code_order_k", ctypes.c_int), ("code_order_v", ctypes.c_int),
                ("k_sink", ctypes.c_void_p), ("v_sink", ctypes.c_void_p), ("T_sink", ctypes.c_int),
                ("tail_rows", ctypes.c_int), ("k_tail_buffer", ctypes.c_void_p * 2),
                ("v_tail_buffer", ctypes.c_void_p * 2), ("ragged", ctypes.c_int),
                ("off_ko", ctypes.c_size_t), ("off_vo", ctypes.c_size_t),
                ("n_outliers", ctypes.c_int)]


class kvq_paged_pool(ctypes.Structure):
    _fields_ = [("k_pages", ctypes.c_void_p), ("v_pages", ctypes.c_void_p),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("n_pages", ctypes.c_int), ("n_kv_heads", ctypes.c_int),
                ("page_size", ctypes.c_int), ("head_dim", ctypes.c_int)]


_P = ctypes.c_void_p
_I = ctypes.c_int
_L = ctypes.c_longlong
_S = ctypes.c_int  # kvq_status
_CFG = ctypes.POINTER(kvq_config)
_POOL = ctypes.POINTER(kvq_paged_pool)

_sigs = {
    "kvq_config_check": (_S, [_CFG]),
    "kvq_cache_bytes": (_S, [_CFG, ctypes.POINTER(ctypes.c_size_t)]),
    "kvq_create": (_S, [_CFG, ctypes.POINTER(_P)]),
    "kvq_destroy": (_S, [_P]),
    "kvq_quantize_prefill": (_S, [_P, _P, _P, _I, _P]),
    "kvq_append": (_S, [_P, _P, _P, _I, _P]),
    "kvq_quantize_prefill_ragged": (_S, [_P, _P, _P, ctypes.POINTER(_I), _I, _P]),
    "kvq_append_ragged": (_S, [_P, _P, _P, ctypes.POINTER(_I), _I, _P]),
    "kvq_get_row_state": (_S, [_P, _I] + [ctypes.POINTER(_I)] * 4),
    "kvq_decode_attention": (_S, [_P, _P, _P, ctypes.c_float, _P]),
    "kvq_append_decode": (_S, [_P, _P, _P, _I, _P, _P, ctypes.c_float, _P]),
    "kvq_dequantize": (_S, [_P, _P, _P, _P]),
    "kvq_decode_attention_noalloc": (_S, [_CFG, _P, _P, _P, _I, _I, _P, _P, ctypes.c_float, _P, _P]),
    "kvq_get_state": (_S, [_P, ctypes.POINTER(_I), ctypes.POINTER(_I)]),
    "kvq_get_buffers": (_S, [_P, ctypes.POINTER(kvq_buffers)]),
    "kvq_check_device_error": (_S, [_P, _P]),
    "kvq_launch_count": (ctypes.c_uint64, []),
    "kvq_debug_fail_allocations": (_S, [_I, _I]),
    "kvq_debug_set_device_error": (_S, [_P, _I]),
    "kvq_debug_set_wait_limit": (_S, [_P, _I]),
    "kvq_status_string": (ctypes.c_char_p, [_S]),
    "kvq_paged_pool_check": (_S, [_POOL]),
    "kvq_paged_plan": (_S, [_P, _P, _I, _P, _I, _P, _I, _P, _I, _I, _P, _P, _P, _P, _P, _P]),
    "kvq_paged_store": (_S, [_POOL, _P, _P, _I, _L, _L, _P, _I, _P, _P]),
    "kvq_paged_workspace_bytes": (_S, [_POOL, ctypes.POINTER(ctypes.c_size_t)]),
    "kvq_paged_attention": (_S, [_POOL, _P, _I, _L, _P, _L, _I, _I, _P, _I, _P, _P, _I, _I,
                                 ctypes.c_float, _I, _P, ctypes.c_size_t, _P, _P]),
}
for _name, (_res, _args) in _sigs.items():
    _fn = getattr(_lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args


class KvqError(RuntimeError):
    def __init__(self, status: int, call: str):
        self.status = status
        super().__init__(f"{call}: {kvq_status_string(status)} (status {status})")


def _check(status: int, call: str) -> None:
    if status != KVQ_OK:
        raise KvqError(status, call)


def _ptr(x) -> int | None:
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream or None
    if isinstance(stream, int):
        return stream or None
    return stream.cuda_stream or None


def make_config(batch, n_q_heads, n_kv_heads, head_dim, max_ctx, bits_k=2, bits_v=2, group=32,
                axis_k=KVQ_AXIS_CHANNEL, axis_v=KVQ_AXIS_TOKEN, keys_pre_rope=False,
                rope_base=10000.0, n_sink=0, residual=0, fp8=False, n_outliers=0) -> kvq_config:
    return kvq_config(int(batch), int(n_q_heads), int(n_kv_heads), int(head_dim), int(max_ctx),
                      int(bits_k), int(bits_v), int(group), int(axis_k), int(axis_v),
                      1 if keys_pre_rope else 0, float(rope_base), int(n_sink), int(residual),
                      1 if fp8 else 0, int(n_outliers))


# ---- the C calls, same names ------------------------------------------------

def kvq_status_string(status: int) -> str:
    return _lib.kvq_status_string(int(status)).decode()


def kvq_config_check(cfg: kvq_config) -> int:
    return _lib.kvq_config_check(ctypes.byref(cfg))


def kvq_cache_bytes(cfg: kvq_config) -> int:
    n = ctypes.c_size_t(0)
    _check(_lib.kvq_cache_bytes(ctypes.byref(cfg), ctypes.byref(n)), "kvq_cache_bytes")
    return n.value


def kvq_create(cfg: kvq_config) -> int:
    h = _P()
    _check(_lib.kvq_create(ctypes.byref(cfg), ctypes.byref(h)), "kvq_create")
    return h.value


def kvq_destroy(handle) -> None:
    _check(_lib.kvq_destroy(handle), "kvq_destroy")


def kvq_quantize_prefill(handle, k, v, T: int | None = None, stream=None) -> None:
    if T is None:
        T = k.shape[-2]
    _check(_lib.kvq_quantize_prefill(handle, _ptr(k), _ptr(v), int(T), _stream(stream)),
           "kvq_quantize_prefill")


def _ints(values):
    vals = [int(x) for x in values]
    return (_I * max(len(vals), 1))(*vals)


def kvq_quantize_prefill_ragged(handle, k, v, lengths, T_stride: int | None = None,
                                stream=None) -> None:
    """k, v: [batch][n_kv_heads][T_stride][head_dim]; row b holds lengths[b] tokens."""
    if T_stride is None:
        T_stride = k.shape[-2]
    _check(_lib.kvq_quantize_prefill_ragged(handle, _ptr(k), _ptr(v), _ints(lengths),
                                            int(T_stride), _stream(stream)),
           "kvq_quantize_prefill_ragged")


def kvq_append_ragged(handle, k, v, n_rows, n_stride: int | None = None, stream=None) -> None:
    """k, v: [batch][n_kv_heads][n_stride][head_dim]; row b appends n_rows[b] tokens."""
    if n_stride is None:
        n_stride = k.shape[-2]
    _check(_lib.kvq_append_ragged(handle, _ptr(k), _ptr(v), _ints(n_rows), int(n_stride),
                                  _stream(stream)), "kvq_append_ragged")


def kvq_get_row_state(handle, row: int) -> tuple[int, int, int, int]:
    """(T_sink, T_q, T_tail, tail_buffer) of batch row `row`."""
    vals = [_I(0) for _ in range(4)]
    _check(_lib.kvq_get_row_state(handle, int(row), *[ctypes.byref(x) for x in vals]),
           "kvq_get_row_state")
    return tuple(x.value for x in vals)


def kvq_append(handle, k, v, n: int | None = None, stream=None) -> None:
    if n is None:
        n = k.shape[-2]
    _check(_lib.kvq_append(handle, _ptr(k), _ptr(v), int(n), _stream(stream)), "kvq_append")


def kvq_decode_attention(handle, q, out, softmax_scale: float, stream=None) -> None:
    _check(_lib.kvq_decode_attention(handle, _ptr(q), _ptr(out), float(softmax_scale),
                                     _stream(stream)), "kvq_decode_attention")


def kvq_append_decode(handle, k, v, n: int, q, out, softmax_scale: float, stream=None) -> None:
    _check(_lib.kvq_append_decode(handle, _ptr(k) if n else None, _ptr(v) if n else None, int(n),
                                  _ptr(q), _ptr(out), float(softmax_scale), _stream(stream)),
           "kvq_append_decode")


def kvq_decode_attention_noalloc(cfg: kvq_config, blocks, k_tail, v_tail, T_q: int, T_tail: int,
                                 q, out, softmax_scale: float, device_error=None,
                                 stream=None) -> None:
    """Decode over a packed cache the caller owns, allocating no device memory
    (see include/kvq.h for who needs this and for the workspace limit)."""
    _check(_lib.kvq_decode_attention_noalloc(ctypes.byref(cfg), _ptr(blocks), _ptr(k_tail),
                                             _ptr(v_tail), int(T_q), int(T_tail), _ptr(q),
                                             _ptr(out), float(softmax_scale), _ptr(device_error),
                                             _stream(stream)), "kvq_decode_attention_noalloc")


def kvq_dequantize(handle, k_out, v_out, stream=None) -> None:
    _check(_lib.kvq_dequantize(handle, _ptr(k_out), _ptr(v_out), _stream(stream)), "kvq_dequantize")


def kvq_get_state(handle) -> tuple[int, int]:
    tq, tt = _I(0), _I(0)
    _check(_lib.kvq_get_state(handle, ctypes.byref(tq), ctypes.byref(tt)), "kvq_get_state")
    return tq.value, tt.value


def kvq_get_buffers(handle) -> kvq_buffers:
    b = kvq_buffers()
    _check(_lib.kvq_get_buffers(handle, ctypes.byref(b)), "kvq_get_buffers")
    return b


def kvq_check_device_error(handle, stream=None) -> int:
    return _lib.kvq_check_device_error(handle, _stream(stream))


def kvq_launch_count() -> int:
    return int(_lib.kvq_launch_count())


def kvq_debug_fail_allocations(after: int, n: int) -> None:
    _check(_lib.kvq_debug_fail_allocations(after, n), "kvq_debug_fail_allocations")


def kvq_debug_set_device_error(handle, value: int) -> None:
    _check(_lib.kvq_debug_set_device_error(handle, value), "kvq_debug_set_device_error")


def kvq_debug_set_wait_limit(handle, limit: int) -> None:
    _check(_lib.kvq_debug_set_wait_limit(handle, limit), "kvq_debug_set_wait_limit")


# ---- the paged 8-bit cache ----------------------------------------------------
#
# The calls take the tensors a serving program keeps: E4M3 pages
# [n_pages][n_kv_heads][page_size][head_dim] with fp32 scales
# [n_pages][n_kv_heads], int32 tables and lengths (include/kvq.h has the
# arithmetic and the contracts).  They run on the tensors' device, on torch's
# current stream of it unless `stream` is given, and can be captured.

def _bad(call: str, what: str):
    raise KvqError(KVQ_ERR_INVALID_ARG, f"{call}: {what}")


def _paged_device(call: str, device):
    """Checks that `device` is a CUDA device; returns its index."""
    if device.type != "cuda":
        _bad(call, f"tensors must be on a CUDA device, not {device}")
    return device.index


def _ints_of(call: str, name: str, x, device, size: int, ndim: int = 1):
    """x: contiguous int32 on `device` with at least `size` elements."""
    import torch
    if (x.dtype is not torch.int32 or x.dim() != ndim or x.device != device
            or x.numel() < size or not x.is_contiguous()):
        _bad(call, f"{name} must be a contiguous int32 tensor of {ndim} dimension(s) and at least "
                   f"{size} elements on {device}")
    return x.data_ptr()


def _on_device(index: int, fn, *args):
    """Runs fn(*args) with CUDA device `index` current."""
    import torch
    if torch.cuda.current_device() == index:
        return fn(*args)
    with torch.cuda.device(index):
        return fn(*args)


def _raw_stream(index: int, stream):
    if stream is None:
        import torch
        return torch._C._cuda_getCurrentRawStream(index) or None
    if isinstance(stream, int):
        return stream or None
    return stream.cuda_stream or None


def _error_ptr(call: str, error, device):
    return None if error is None else _ints_of(call, "error", error, device, 1)


def _pool_of(call: str, k_pages, v_pages, k_scale, v_scale) -> kvq_paged_pool:
    import torch
    if (k_pages.dtype is not torch.float8_e4m3fn or v_pages.dtype is not torch.float8_e4m3fn
            or k_pages.dim() != 4 or v_pages.shape != k_pages.shape
            or not k_pages.is_contiguous() or not v_pages.is_contiguous()):
        _bad(call, "k_pages and v_pages must be contiguous float8_e4m3fn tensors "
                   "[n_pages][n_kv_heads][page_size][head_dim]")
    n, h, ps, d = k_pages.shape
    device = k_pages.device
    for x in (k_scale, v_scale):
        if (x.dtype is not torch.float32 or x.shape != (n, h) or not x.is_contiguous()
                or x.device != device):
            _bad(call, f"scales must be contiguous float32 tensors [{n}][{h}] on {device}")
    if v_pages.device != device:
        _bad(call, f"v_pages must be on {device}")
    return kvq_paged_pool(k_pages.data_ptr(), v_pages.data_ptr(), k_scale.data_ptr(),
                          v_scale.data_ptr(), n, h, ps, d)


def _rows_of(call: str, name: str, x, heads: int, dim: int, device):
    """x: [tokens][heads][dim], heads and dims contiguous; returns its token stride."""
    import torch
    if x.dim() != 3 or x.shape[1] != heads or x.shape[2] != dim or x.device != device:
        _bad(call, f"{name} must be [tokens][{heads}][{dim}] on {device}")
    st, sh, sd = x.stride()
    if sd != 1 or (sh != dim and heads > 1):
        _bad(call, f"{name}: the heads and channels of a token must be contiguous")
    return st if x.shape[0] > 1 else heads * dim


def _dtype_of(call: str, name: str, x) -> int:
    import torch
    if x.dtype is torch.float16:
        return KVQ_DTYPE_FP16
    if x.dtype is torch.bfloat16:
        return KVQ_DTYPE_BF16
    _bad(call, f"{name} must be float16 or bfloat16, not {x.dtype}")


def kvq_paged_pool_check(n_pages: int, n_kv_heads: int, page_size: int, head_dim: int) -> int:
    pool = kvq_paged_pool(None, None, None, None, int(n_pages), int(n_kv_heads), int(page_size),
                          int(head_dim))
    return _lib.kvq_paged_pool_check(ctypes.byref(pool))


def kvq_paged_plan(ctx_len, new_len, block_table, free_pages, n_free, page_size: int,
                   n_tokens: int, cu_new=None, seq_len=None, slots=None, n_left=None, error=None,
                   stream=None):
    """Block tables and slots of a serving step.

    ctx_len, new_len: int32 [batch], cached and new tokens of each request;
    block_table: int32 [batch][max_pages], written in place; free_pages: int32
    stack of free page ids of which n_free[0] are left.  Returns (cu_new
    [batch + 1], seq_len [batch], slots [n_tokens], n_left [1])."""
    import torch
    call = "kvq_paged_plan"
    device = ctx_len.device
    index = _paged_device(call, device)
    batch, n_tokens = ctx_len.numel(), int(n_tokens)
    if block_table.dim() != 2 or block_table.shape[0] != batch or n_tokens < 0:
        _bad(call, f"block_table must be [{batch}][max_pages] and n_tokens >= 0")
    made = [n for n, x in ((n_tokens, slots), (batch + 1, cu_new), (batch, seq_len), (1, n_left))
            if x is None]
    if made:
        parts = iter(torch.empty(sum(made), dtype=torch.int32, device=device).split(made))
        slots = next(parts) if slots is None else slots
        cu_new = next(parts) if cu_new is None else cu_new
        seq_len = next(parts) if seq_len is None else seq_len
        n_left = next(parts) if n_left is None else n_left
    i = _ints_of
    status = _on_device(
        index, _lib.kvq_paged_plan, i(call, "ctx_len", ctx_len, device, batch),
        i(call, "new_len", new_len, device, batch), batch,
        i(call, "block_table", block_table, device, 1, 2), block_table.shape[1],
        i(call, "free_pages", free_pages, device, 0), free_pages.numel(),
        i(call, "n_free", n_free, device, 1), int(page_size), n_tokens,
        i(call, "cu_new", cu_new, device, batch + 1), i(call, "seq_len", seq_len, device, batch),
        i(call, "slots", slots, device, n_tokens), i(call, "n_left", n_left, device, 1),
        _error_ptr(call, error, device), _raw_stream(index, stream))
    if status:
        _check(status, call)
    return cu_new, seq_len, slots, n_left


def kvq_paged_store(k, v, slots, k_pages, v_pages, k_scale, v_scale, error=None,
                    stream=None) -> None:
    """Stores keys and values k, v (fp16 or bf16 [tokens][n_kv_heads][head_dim],
    any token stride that is a multiple of 8) at their slots (int32 [tokens])."""
    call = "kvq_paged_store"
    device = k_pages.device
    index = _paged_device(call, device)
    pool = _pool_of(call, k_pages, v_pages, k_scale, v_scale)
    dtype = _dtype_of(call, "k", k)
    if v.dtype is not k.dtype or v.shape != k.shape:
        _bad(call, "k and v must have the same type and shape")
    ks = _rows_of(call, "k", k, pool.n_kv_heads, pool.head_dim, device)
    vs = _rows_of(call, "v", v, pool.n_kv_heads, pool.head_dim, device)
    n = k.shape[0]
    status = _on_device(index, _lib.kvq_paged_store, ctypes.byref(pool), k.data_ptr(),
                        v.data_ptr(), dtype, ks, vs, _ints_of(call, "slots", slots, device, n), n,
                        _error_ptr(call, error, device), _raw_stream(index, stream))
    if status:
        _check(status, call)


_paged_workspaces: dict = {}


def _paged_workspace(pool: kvq_paged_pool, index: int, stream):
    """The attention's workspace.  Calls on one stream run one after the other
    and share one; a captured call gets its own from the capture's memory,
    with the counters cleared by the graph, so graphs share nothing."""
    import torch
    key = (index, stream, pool.head_dim)
    capturing = torch.cuda.is_current_stream_capturing()
    ws = None if capturing else _paged_workspaces.get(key)
    if ws is None:
        n = ctypes.c_size_t(0)
        _check(_lib.kvq_paged_workspace_bytes(ctypes.byref(pool), ctypes.byref(n)),
               "kvq_paged_workspace_bytes")
        ws = torch.empty(n.value, dtype=torch.uint8, device=f"cuda:{index}")
        ws[:1024].zero_()
        if not capturing:
            torch.cuda.current_stream(index).synchronize()  # `stream` may be another one
            _paged_workspaces[key] = ws
    return ws


def kvq_paged_attention(q, k_pages, v_pages, k_scale, v_scale, block_table, cu_new, seq_len,
                        max_new: int = 1, softmax_scale: float | None = None, window: int = 0,
                        out=None, workspace=None, error=None, stream=None):
    """Attention of the new tokens over the pages; returns out, in q's type.

    q: fp16 or bf16 [tokens][n_q_heads][head_dim]; request b's new tokens are
    rows cu_new[b] .. cu_new[b + 1], the last of its seq_len[b] tokens;
    max_new: the most new tokens of a request; window: how many tokens back a
    token sees (0: all).  `workspace`: a uint8 tensor of
    kvq_paged_workspace_bytes whose first 1024 bytes are zero, for callers
    that overlap calls on streams of their own."""
    import torch
    call = "kvq_paged_attention"
    device = k_pages.device
    index = _paged_device(call, device)
    pool = _pool_of(call, k_pages, v_pages, k_scale, v_scale)
    dtype = _dtype_of(call, "q", q)
    heads = q.shape[1] if q.dim() == 3 else 0
    qs = _rows_of(call, "q", q, heads, pool.head_dim, device)
    n = q.shape[0]
    if out is None:
        out = torch.empty(n, heads, pool.head_dim, dtype=q.dtype, device=device)
        os_ = heads * pool.head_dim
    else:
        if out.dtype is not q.dtype or out.shape != q.shape:
            _bad(call, "out must have q's type and shape")
        os_ = _rows_of(call, "out", out, heads, pool.head_dim, device)
    batch = seq_len.numel()
    if block_table.dim() != 2 or block_table.shape[0] != batch:
        _bad(call, f"block_table must be [{batch}][max_pages]")
    if softmax_scale is None:
        softmax_scale = pool.head_dim ** -0.5
    st = _raw_stream(index, stream)
    if workspace is None:
        workspace = _on_device(index, _paged_workspace, pool, index, st)
    elif workspace.dtype is not torch.uint8 or workspace.device != device \
            or not workspace.is_contiguous():
        _bad(call, f"workspace must be a contiguous uint8 tensor on {device}")
    i = _ints_of
    status = _on_device(
        index, _lib.kvq_paged_attention, ctypes.byref(pool), q.data_ptr(), dtype, qs,
        out.data_ptr(), os_, n, heads, i(call, "block_table", block_table, device, 1, 2),
        block_table.shape[1], i(call, "cu_new", cu_new, device, batch + 1),
        i(call, "seq_len", seq_len, device, batch), batch, int(max_new), softmax_scale,
        int(window), workspace.data_ptr(), workspace.numel(), _error_ptr(call, error, device), st)
    if status:
        _check(status, call)
    return out


# ---- convenience -------------------------------------------------------------

class _DeviceArray:
    """Exposes a library-owned device range to torch without copying."""

    def __init__(self, ptr: int, shape, typestr: str):
        self.__cuda_array_interface__ = {"shape": tuple(shape), "typestr": typestr,
                                         "data": (int(ptr), False), "version": 3, "strides": None}


def device_view(ptr: int, shape, typestr: str = "|u1"):
    import torch
    return torch.as_tensor(_DeviceArray(ptr, shape, typestr), device="cuda")


class KVCache:
    """One layer's packed KV cache on the current CUDA device.

    Keyword arguments are those of ``make_config`` (the fields of
    ``kvq_config``): batch, n_q_heads, n_kv_heads, head_dim, max_ctx,
    bits_k / bits_v (2, 4, 8), group (32, 64, 128), axis_k / axis_v,
    keys_pre_rope / rope_base, n_sink and residual (fp16 windows), fp8 (E4M3
    codes, 8-bit sides), n_outliers (elements kept in fp16 per block and
    side).  A typical decode loop::

        cache = KVCache(batch=8, n_q_heads=32, n_kv_heads=32, head_dim=128,
                        max_ctx=8192, bits_k=2, bits_v=2)
        cache.prefill(k, v)                    # [B][Hkv][T][D] fp16 on the GPU
        for step in range(n):
            out = cache.append_decode(k1, v1, q)   # [B][Hkv][1][D], [B][Hq][D]

    ``prefill_ragged`` / ``append_ragged`` take per-row lengths (a serving
    batch of sequences of different lengths, batch <= 64); ``row_state``
    reports each row's sink, quantized and tail counts.
    """

    def __init__(self, **cfg_kw):
        self.cfg = make_config(**cfg_kw)
        self.handle = kvq_create(self.cfg)

    @property
    def gqa(self) -> int:
        return self.cfg.n_q_heads // self.cfg.n_kv_heads

    def close(self) -> None:
        if self.handle:
            kvq_destroy(self.handle)
            self.handle = None

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def prefill(self, k, v, stream=None):
        kvq_quantize_prefill(self.handle, k, v, k.shape[-2], stream)

    def prefill_ragged(self, k, v, lengths, stream=None):
        kvq_quantize_prefill_ragged(self.handle, k, v, lengths, k.shape[-2], stream)

    def append_ragged(self, k, v, n_rows, stream=None):
        kvq_append_ragged(self.handle, k, v, n_rows, k.shape[-2], stream)

    def row_state(self, row: int) -> tuple[int, int, int, int]:
        """(T_sink, T_q, T_tail, tail_buffer) of batch row `row`."""
        return kvq_get_row_state(self.handle, row)

    def append(self, k, v, stream=None):
        kvq_append(self.handle, k, v, k.shape[-2], stream)

    def decode(self, q, out=None, softmax_scale=None, stream=None):
        import torch
        if out is None:
            out = torch.empty(q.shape, dtype=torch.float32, device=q.device)
        if softmax_scale is None:
            softmax_scale = self.cfg.head_dim ** -0.5
        kvq_decode_attention(self.handle, q, out, softmax_scale, stream)
        return out

    def append_decode(self, k, v, q, out=None, softmax_scale=None, stream=None):
        """Appends k, v ([batch][n_kv_heads][n][head_dim] fp16) and decodes q,
        in one launch when no group is completed."""
        import torch
        if out is None:
            out = torch.empty(q.shape, dtype=torch.float32, device=q.device)
        if softmax_scale is None:
            softmax_scale = self.cfg.head_dim ** -0.5
        n = 0 if k is None else k.shape[-2]
        kvq_append_decode(self.handle, k, v, n, q, out, softmax_scale, stream)
        return out

    def dequantize(self, stream=None):
        import torch
        tq, _ = self.state
        shape = (self.cfg.batch, self.cfg.n_kv_heads, tq, self.cfg.head_dim)
        k = torch.empty(shape, dtype=torch.float32, device="cuda")
        v = torch.empty(shape, dtype=torch.float32, device="cuda")
        kvq_dequantize(self.handle, k, v, stream)
        return k, v

    @property
    def state(self) -> tuple[int, int]:
        return kvq_get_state(self.handle)

    def buffers(self) -> kvq_buffers:
        return kvq_get_buffers(self.handle)

    def block_bytes_view(self):
        """uint8 [P][NB][block_bytes] view of the packed blocks (no copy)."""
        b = self.buffers()
        return device_view(b.blocks, (b.n_pairs, b.blocks_per_pair, b.block_bytes))

    def tail_views(self):
        """fp16 [P][tail_rows][D] views of the active K and V tails (no copy)."""
        b = self.buffers()
        shape = (b.n_pairs, b.tail_rows, self.cfg.head_dim)
        k = device_view(b.k_tail, shape, "<f2")
        v = device_view(b.v_tail, shape, "<f2")
        return k, v

    def row_tail_views(self, row: int):
        """fp16 [n_kv_heads][tail_rows][D] views of row `row`'s K and V tails."""
        b = self.buffers()
        buf = self.row_state(row)[3]
        shape = (b.n_pairs, b.tail_rows, self.cfg.head_dim)
        h = self.cfg.n_kv_heads
        k = device_view(b.k_tail_buffer[buf], shape, "<f2")[row * h:(row + 1) * h]
        v = device_view(b.v_tail_buffer[buf], shape, "<f2")[row * h:(row + 1) * h]
        return k, v

    def sink_views(self):
        """fp16 [P][n_sink][D] views of the K and V sink windows (no copy);
        None when the cache has no sink window."""
        b = self.buffers()
        if not b.k_sink:
            return None
        shape = (b.n_pairs, self.cfg.n_sink, self.cfg.head_dim)
        return device_view(b.k_sink, shape, "<f2"), device_view(b.v_sink, shape, "<f2")

    def check(self, stream=None) -> None:
        _check(kvq_check_device_error(self.handle, stream), "kvq_check_device_error")


class PagedCache:
    """One layer's paged 8-bit KV cache: a pool of E4M3 pages with a
    power-of-two scale for each page and kv head.

    The requests' tables and lengths are the caller's; a serving step is::

        cache = PagedCache(n_pages=4096, page_size=64, n_q_heads=32, n_kv_heads=8,
                           head_dim=128)
        cu, seq, slots, left = cache.plan(ctx_len, new_len, block_table, free_pages, n_free,
                                          n_tokens)
        cache.store(k, v, slots)        # [n_tokens][n_kv_heads][head_dim] fp16 or bf16
        out = cache.attention(q, block_table, cu, seq, max_new=1)

    The step's plan serves every layer's cache.  ``check`` raises for what the
    kernels flagged since the last check (a page id outside the pool, a free
    stack that ran out, a non-finite key or value)."""

    def __init__(self, n_pages, page_size, n_q_heads, n_kv_heads, head_dim, device="cuda"):
        import torch
        _check(kvq_paged_pool_check(n_pages, n_kv_heads, page_size, head_dim),
               "kvq_paged_pool_check")
        if n_q_heads < 1 or n_q_heads % n_kv_heads:
            _bad("PagedCache", "n_q_heads must be a multiple of n_kv_heads")
        self.n_q_heads = int(n_q_heads)
        self.page_size = int(page_size)
        shape = (n_pages, n_kv_heads, page_size, head_dim)
        zeros = lambda s, t: torch.zeros(s, dtype=t, device=device)  # noqa: E731
        self.k_pages = zeros(shape, torch.uint8).view(torch.float8_e4m3fn)
        self.v_pages = zeros(shape, torch.uint8).view(torch.float8_e4m3fn)
        self.k_scale = zeros(shape[:2], torch.float32).fill_(2.0 ** -15)
        self.v_scale = zeros(shape[:2], torch.float32).fill_(2.0 ** -15)
        self.error = zeros(1, torch.int32)

    def plan(self, ctx_len, new_len, block_table, free_pages, n_free, n_tokens, stream=None):
        return kvq_paged_plan(ctx_len, new_len, block_table, free_pages, n_free, self.page_size,
                              n_tokens, error=self.error, stream=stream)

    def store(self, k, v, slots, stream=None):
        kvq_paged_store(k, v, slots, self.k_pages, self.v_pages, self.k_scale, self.v_scale,
                        error=self.error, stream=stream)

    def attention(self, q, block_table, cu_new, seq_len, max_new=1, softmax_scale=None, window=0,
                  out=None, stream=None):
        if q.dim() == 3 and q.shape[1] != self.n_q_heads:
            _bad("PagedCache.attention", f"q must have {self.n_q_heads} heads")
        return kvq_paged_attention(q, self.k_pages, self.v_pages, self.k_scale, self.v_scale,
                                   block_table, cu_new, seq_len, max_new=max_new,
                                   softmax_scale=softmax_scale, window=window, out=out,
                                   error=self.error, stream=stream)

    def check(self) -> None:
        """Synchronizes the device; raises KvqError for what the kernels flagged."""
        import torch
        torch.cuda.synchronize(self.error.device)
        bits = int(self.error.item())
        if not bits:
            return
        self.error.zero_()
        if bits & KVQ_PAGED_ERR_WAIT:  # a split that did not finish leaves its counters
            for ws in _paged_workspaces.values():
                if ws.device == self.error.device:
                    ws[:1024].zero_()
        names = ((KVQ_PAGED_ERR_WAIT, "a bounded wait ran out"),
                 (KVQ_PAGED_ERR_BAD_PAGE, "a page id outside the pool"),
                 (KVQ_PAGED_ERR_NO_PAGES, "the free stack ran out"),
                 (KVQ_PAGED_ERR_LENGTH, "a length breaks the call's contract"),
                 (KVQ_PAGED_ERR_NONFINITE, "a non-finite key or value"))
        what = ", ".join(n for b, n in names if bits & b)
        raise KvqError(KVQ_ERR_DEVICE_CHECK, f"PagedCache.check: {what}")
