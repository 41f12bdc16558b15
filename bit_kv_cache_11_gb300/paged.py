"""Binding of the paged 8-bit cache's calls (include/kvq.h): the operators of a
serving step on the tensors a serving program keeps.

Pages are float8_e4m3fn tensors [n_pages][n_kv_heads][page_size][head_dim] with
fp32 scales [n_pages][n_kv_heads]; tables, lengths and slots are int32.  The
calls run on the tensors' device, on torch's current stream of it unless
`stream` is given, and can be captured into CUDA graphs.  Arguments are checked
here, on the host; KvqError tells what is wrong.  The checks are written for
few interpreter steps: a small call costs less on the GPU than its marshalling.
"""
from __future__ import annotations

import ctypes

import torch

from . import kvq
from .kvq import (KVQ_DTYPE_BF16, KVQ_DTYPE_FP16, KVQ_ERR_DEVICE_CHECK, KVQ_ERR_INVALID_ARG,
                  KVQ_PAGED_ERR_BAD_PAGE, KVQ_PAGED_ERR_LENGTH, KVQ_PAGED_ERR_NONFINITE,
                  KVQ_PAGED_ERR_NO_PAGES, KVQ_PAGED_ERR_WAIT, KvqError, kvq_paged_pool)

_lib = kvq._lib
_check = kvq._check
_byref = ctypes.byref
_int32 = torch.int32
_fp16 = torch.float16
_bf16 = torch.bfloat16
_fp8 = torch.float8_e4m3fn
_fp32 = torch.float32
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _bad(call: str, what: str):
    raise KvqError(KVQ_ERR_INVALID_ARG, f"{call}: {what}")


def _index_of(call: str, x) -> int:
    if not x.is_cuda:
        _bad(call, f"tensors must be on a CUDA device, not {x.device}")
    return x.get_device()


def _ints(call: str, name: str, x, index: int, size: int) -> int:
    """Address of x: contiguous int32 on device `index`, at least `size` elements."""
    if (x.dtype is not _int32 or x.get_device() != index or not x.is_contiguous()
            or x.numel() < size):
        _bad(call, f"{name} must be a contiguous int32 tensor of at least {size} elements on "
                   f"cuda:{index}")
    return x.data_ptr()


def _launch(index: int, fn, *args) -> int:
    """fn(*args) with CUDA device `index` current."""
    if torch._C._cuda_getDevice() == index:
        return fn(*args)
    with torch.cuda.device(index):
        return fn(*args)


def _stream(index: int, stream):
    if stream is None:
        if _current_stream is not None:
            return _current_stream(index) or None
        return torch.cuda.current_stream(index).cuda_stream or None
    if isinstance(stream, int):
        return stream or None
    return stream.cuda_stream or None


def _pool(call: str, index: int, k_pages, v_pages, k_scale, v_scale) -> kvq_paged_pool:
    shape = k_pages.shape
    if (k_pages.dtype is not _fp8 or v_pages.dtype is not _fp8 or len(shape) != 4
            or v_pages.shape != shape or v_pages.get_device() != index
            or not k_pages.is_contiguous() or not v_pages.is_contiguous()):
        _bad(call, "k_pages and v_pages must be contiguous float8_e4m3fn tensors "
                   "[n_pages][n_kv_heads][page_size][head_dim] on one device")
    n, h, ps, d = shape
    two = (n, h)
    if (k_scale.dtype is not _fp32 or v_scale.dtype is not _fp32 or k_scale.shape != two
            or v_scale.shape != two or k_scale.get_device() != index
            or v_scale.get_device() != index or not k_scale.is_contiguous()
            or not v_scale.is_contiguous()):
        _bad(call, f"scales must be contiguous float32 tensors [{n}][{h}] on cuda:{index}")
    return kvq_paged_pool(k_pages.data_ptr(), v_pages.data_ptr(), k_scale.data_ptr(),
                          v_scale.data_ptr(), n, h, ps, d)


def _rows(call: str, name: str, x, heads: int, dim: int, index: int) -> int:
    """Token stride of x: [tokens][heads][dim], heads and channels contiguous."""
    if x.dim() != 3 or x.get_device() != index:
        _bad(call, f"{name} must be [tokens][heads][{dim}] on cuda:{index}")
    n, h, d = x.shape
    st, sh, sd = x.stride()
    if h != heads or d != dim or sd != 1 or (sh != dim and h != 1):
        _bad(call, f"{name} must be [tokens][{heads}][{dim}], a token's heads and channels "
                   "contiguous")
    return st if n > 1 else heads * dim


def _dtype(call: str, name: str, x) -> int:
    if x.dtype is _fp16:
        return KVQ_DTYPE_FP16
    if x.dtype is _bf16:
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
    call = "kvq_paged_plan"
    index = _index_of(call, ctx_len)
    batch = ctx_len.numel()
    if block_table.dim() != 2 or block_table.shape[0] != batch or n_tokens < 0:
        _bad(call, f"block_table must be [{batch}][max_pages] and n_tokens >= 0")
    a_ctx = _ints(call, "ctx_len", ctx_len, index, batch)
    if cu_new is None:
        cu_new = ctx_len.new_empty(batch + 1)
    if seq_len is None:
        seq_len = ctx_len.new_empty(batch)
    if slots is None:
        slots = ctx_len.new_empty(n_tokens)
    if n_left is None:
        n_left = ctx_len.new_empty(1)
    status = _launch(
        index, _lib.kvq_paged_plan, a_ctx, _ints(call, "new_len", new_len, index, batch), batch,
        _ints(call, "block_table", block_table, index, 1), block_table.shape[1],
        _ints(call, "free_pages", free_pages, index, 0), free_pages.numel(),
        _ints(call, "n_free", n_free, index, 1), page_size, n_tokens,
        _ints(call, "cu_new", cu_new, index, batch + 1),
        _ints(call, "seq_len", seq_len, index, batch),
        _ints(call, "slots", slots, index, n_tokens), _ints(call, "n_left", n_left, index, 1),
        None if error is None else _ints(call, "error", error, index, 1), _stream(index, stream))
    if status:
        _check(status, call)
    return cu_new, seq_len, slots, n_left


def kvq_paged_store(k, v, slots, k_pages, v_pages, k_scale, v_scale, error=None,
                    stream=None) -> None:
    """Stores keys and values k, v (fp16 or bf16 [tokens][n_kv_heads][head_dim],
    any token stride that is a multiple of 8) at their slots (int32 [tokens])."""
    call = "kvq_paged_store"
    index = _index_of(call, k_pages)
    pool = _pool(call, index, k_pages, v_pages, k_scale, v_scale)
    dtype = _dtype(call, "k", k)
    if v.dtype is not k.dtype or v.shape != k.shape:
        _bad(call, "k and v must have the same type and shape")
    heads, dim = pool.n_kv_heads, pool.head_dim
    ks = _rows(call, "k", k, heads, dim, index)
    vs = _rows(call, "v", v, heads, dim, index)
    n = k.shape[0]
    status = _launch(index, _lib.kvq_paged_store, _byref(pool), k.data_ptr(), v.data_ptr(), dtype,
                     ks, vs, _ints(call, "slots", slots, index, n), n,
                     None if error is None else _ints(call, "error", error, index, 1),
                     _stream(index, stream))
    if status:
        _check(status, call)


_paged_workspaces: dict = {}


def _paged_workspace(pool: kvq_paged_pool, index: int, stream):
    """The attention's workspace.  Calls on one stream run one after the other
    and share one; a captured call gets its own from the capture's memory,
    with the counters cleared by the graph, so graphs share nothing."""
    capturing = torch._C._cuda_isCurrentStreamCapturing()
    if not capturing:
        ws = _paged_workspaces.get((index, stream, pool.head_dim))
        if ws is not None:
            return ws
    n = ctypes.c_size_t(0)
    _check(_lib.kvq_paged_workspace_bytes(_byref(pool), _byref(n)), "kvq_paged_workspace_bytes")
    ws = torch.empty(n.value, dtype=torch.uint8, device=f"cuda:{index}")
    ws[:1024].zero_()
    if not capturing:
        torch.cuda.current_stream(index).synchronize()  # `stream` may be another one
        _paged_workspaces[(index, stream, pool.head_dim)] = ws
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
    call = "kvq_paged_attention"
    index = _index_of(call, k_pages)
    pool = _pool(call, index, k_pages, v_pages, k_scale, v_scale)
    dtype = _dtype(call, "q", q)
    if q.dim() != 3:
        _bad(call, "q must be [tokens][n_q_heads][head_dim]")
    n, heads, dim = q.shape
    qs = _rows(call, "q", q, heads, pool.head_dim, index)
    if out is None:
        out = q.new_empty(q.shape)
        os_ = heads * dim
    else:
        if out.dtype is not q.dtype or out.shape != q.shape:
            _bad(call, "out must have q's type and shape")
        os_ = _rows(call, "out", out, heads, dim, index)
    batch = seq_len.numel()
    if block_table.dim() != 2 or block_table.shape[0] != batch:
        _bad(call, f"block_table must be [{batch}][max_pages]")
    st = _stream(index, stream)
    if workspace is None:
        workspace = _launch(index, _paged_workspace, pool, index, st)
    elif (workspace.dtype is not torch.uint8 or workspace.get_device() != index
          or not workspace.is_contiguous()):
        _bad(call, f"workspace must be a contiguous uint8 tensor on cuda:{index}")
    status = _launch(
        index, _lib.kvq_paged_attention, _byref(pool), q.data_ptr(), dtype, qs, out.data_ptr(),
        os_, n, heads, _ints(call, "block_table", block_table, index, 1), block_table.shape[1],
        _ints(call, "cu_new", cu_new, index, batch + 1),
        _ints(call, "seq_len", seq_len, index, batch), batch, max_new,
        dim ** -0.5 if softmax_scale is None else softmax_scale, window, workspace.data_ptr(),
        workspace.numel(), None if error is None else _ints(call, "error", error, index, 1), st)
    if status:
        _check(status, call)
    return out


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
