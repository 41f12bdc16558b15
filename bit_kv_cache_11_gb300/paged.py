"""Binding of the paged 8-bit cache's calls (include/kvq.h): the operators of a
serving step on the tensors a serving program keeps.

Pages are float8_e4m3fn tensors [n_pages][n_kv_heads][page_size][head_dim] with
fp32 scales [n_pages][n_kv_heads]; tables, lengths and slots are int32.  The
calls run on the tensors' device, on torch's current stream of it unless
`stream` is given (a stream or its address), and can be captured into CUDA
graphs.  Arguments are checked on the host (csrc/paged_bind.cpp); KvqError
tells what is wrong.  `error` is an optional int32 tensor that the kernels OR
the KVQ_PAGED_ERR_* bits into.  Nothing here has a gradient.
"""
from __future__ import annotations

import ctypes

import torch

from . import kvq
from .kvq import (KVQ_ERR_DEVICE_CHECK, KVQ_ERR_INVALID_ARG, KVQ_PAGED_ERR_BAD_PAGE,
                  KVQ_PAGED_ERR_LENGTH, KVQ_PAGED_ERR_NONFINITE, KVQ_PAGED_ERR_NO_PAGES,
                  KVQ_PAGED_ERR_WAIT, KvqError, kvq_paged_pool)

try:
    from . import _paged_bind
except ImportError as e:
    raise ImportError("the binding _paged_bind.so is not built; build it with "
                      "`python -m bit_kv_cache_11_gb300.build`") from e

_paged_bind.set_error_class(KvqError)
_plan = _paged_bind.plan
_store = _paged_bind.store
_attention = _paged_bind.attention
_append = _paged_bind.append


def _sizes(*sizes):
    """A pool's sizes as C ints: those beyond 32 bits as its ends, which no call takes."""
    return (max(-(1 << 31), min(int(n), (1 << 31) - 1)) for n in sizes)


def kvq_paged_pool_check(n_pages: int, n_kv_heads: int, page_size: int, head_dim: int) -> int:
    """Status of a pool's sizes (KVQ_OK when the calls take such a pool)."""
    pool = kvq_paged_pool(None, None, None, None, *_sizes(n_pages, n_kv_heads, page_size, head_dim))
    return kvq._lib.kvq_paged_pool_check(ctypes.byref(pool))


def kvq_paged_workspace_bytes(n_pages: int, n_kv_heads: int, page_size: int,
                              head_dim: int) -> int:
    """Bytes of the attention's workspace for such a pool."""
    pool = kvq_paged_pool(None, None, None, None, *_sizes(n_pages, n_kv_heads, page_size, head_dim))
    n = ctypes.c_size_t(0)
    kvq._check(kvq._lib.kvq_paged_workspace_bytes(ctypes.byref(pool), ctypes.byref(n)),
               "kvq_paged_workspace_bytes")
    return n.value


def kvq_paged_plan(ctx_len, new_len, block_table, free_pages, n_free, page_size: int,
                   n_tokens: int, cu_new=None, seq_len=None, slots=None, n_left=None, error=None,
                   stream=None, positions=None):
    """Block tables and slots of a serving step.

    ctx_len, new_len: int32 [batch], cached and new tokens of each request;
    block_table: int32 [batch][max_pages], written in place; free_pages: int32
    stack of free page ids of which n_free[0] are left.  Returns (cu_new
    [batch + 1], seq_len [batch], slots [n_tokens], n_left [1]); the stack's
    new height is n_left[0].  A request that the stack cannot serve keeps
    seq_len = ctx_len and gets slots -1: its rows of the attention's output
    mean nothing, and its step can be made again when pages are free.
    `positions`, an int32 tensor [n_tokens], gets every new token's position
    (0 behind the last one); it overlaps none of the other tensors."""
    return _plan(ctx_len, new_len, block_table, free_pages, n_free, page_size, n_tokens, cu_new,
                 seq_len, slots, n_left, error, stream, positions)


def kvq_paged_store(k, v, slots, k_pages, v_pages, k_scale, v_scale, error=None,
                    stream=None) -> None:
    """Stores keys and values k, v (fp16 or bf16 [tokens][n_kv_heads][head_dim],
    any token stride that is a multiple of 8) at their slots (int32 [tokens],
    negative: nowhere)."""
    _store(k, v, slots, k_pages, v_pages, k_scale, v_scale, error, stream)


def kvq_paged_append(k, v, slots, k_pages, v_pages, k_scale, v_scale, angles, interleaved=False,
                     q=None, q_out=None, error=None, stream=None):
    """kvq_paged_store with the keys turned on the way by their tokens' angles
    (kvq_rotary_angles: fp32 [tokens][rotary_dim / 2][2]); the step's queries q
    [tokens][n_q_heads][head_dim], where given, are turned too.  Returns them
    (q_out, which may be q itself, or a new tensor), or None.  The same bits as
    kvq_rotate of k and q followed by kvq_paged_store."""
    return _append(k, v, slots, k_pages, v_pages, k_scale, v_scale, angles, interleaved, q, q_out,
                   error, stream)


def kvq_paged_attention(q, k_pages, v_pages, k_scale, v_scale, block_table, cu_new, seq_len,
                        max_new: int = 1, softmax_scale: float | None = None, window: int = 0,
                        out=None, workspace=None, error=None, stream=None):
    """Attention of the new tokens over the pages; returns out, in q's type.

    q: fp16 or bf16 [tokens][n_q_heads][head_dim]; request b's new tokens are
    rows cu_new[b] .. cu_new[b + 1], the last of its seq_len[b] tokens;
    max_new: the most new tokens of a request; softmax_scale: 1 / sqrt(head_dim)
    unless given; window: how many tokens back a token sees (0: all).
    `workspace`: a uint8 tensor of kvq_paged_workspace_bytes whose first 1024
    bytes are zero.  Without it, the calls of a stream share one, which is kept
    (12.6 MB for head_dim 128, 6.4 MB for 64), and the calls that a stream
    captures into one graph share another, which goes when the graph does."""
    return _attention(q, k_pages, v_pages, k_scale, v_scale, block_table, cu_new, seq_len, max_new,
                      softmax_scale, window, out, workspace, error, stream)


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
        self._make_pool(n_pages, n_kv_heads, page_size, head_dim, device)
        if n_q_heads < 1 or n_q_heads % n_kv_heads:
            raise KvqError(KVQ_ERR_INVALID_ARG,
                           f"{type(self).__name__}: n_q_heads must be a multiple of n_kv_heads")
        self.n_q_heads = int(n_q_heads)
        self.page_size = int(page_size)
        self.error = torch.zeros(1, dtype=torch.int32, device=device)

    def _make_pool(self, n_pages, n_kv_heads, page_size, head_dim, device):
        kvq._check(kvq_paged_pool_check(n_pages, n_kv_heads, page_size, head_dim),
                   "kvq_paged_pool_check")
        shape = (n_pages, n_kv_heads, page_size, head_dim)
        zeros = lambda s, t: torch.zeros(s, dtype=t, device=device)  # noqa: E731
        self.k_pages = zeros(shape, torch.uint8).view(torch.float8_e4m3fn)
        self.v_pages = zeros(shape, torch.uint8).view(torch.float8_e4m3fn)
        self.k_scale = zeros(shape[:2], torch.float32).fill_(2.0 ** -15)
        self.v_scale = zeros(shape[:2], torch.float32).fill_(2.0 ** -15)

    def _pool(self):
        return self.k_pages, self.v_pages, self.k_scale, self.v_scale

    _store_call = staticmethod(kvq_paged_store)
    _append_call = staticmethod(kvq_paged_append)
    _attention_call = staticmethod(kvq_paged_attention)

    def plan(self, ctx_len, new_len, block_table, free_pages, n_free, n_tokens, stream=None,
             positions=None):
        return kvq_paged_plan(ctx_len, new_len, block_table, free_pages, n_free, self.page_size,
                              n_tokens, error=self.error, stream=stream, positions=positions)

    def store(self, k, v, slots, stream=None):
        self._store_call(k, v, slots, *self._pool(), error=self.error, stream=stream)

    def append(self, k, v, slots, angles, interleaved=False, q=None, q_out=None, stream=None):
        """store with the keys, and the queries q where given, turned by `angles`."""
        return self._append_call(k, v, slots, *self._pool(), angles, interleaved=interleaved, q=q,
                                 q_out=q_out, error=self.error, stream=stream)

    def attention(self, q, block_table, cu_new, seq_len, max_new=1, softmax_scale=None, window=0,
                  out=None, stream=None):
        if q.dim() == 3 and q.shape[1] != self.n_q_heads:
            raise KvqError(KVQ_ERR_INVALID_ARG,
                           f"{type(self).__name__}.attention: q must have {self.n_q_heads} heads")
        return self._attention_call(q, *self._pool(), block_table, cu_new, seq_len, max_new=max_new,
                                    softmax_scale=softmax_scale, window=window, out=out,
                                    error=self.error, stream=stream)

    def check(self) -> None:
        """Synchronizes the device; raises KvqError for what the kernels flagged."""
        torch.cuda.synchronize(self.error.device)
        bits = int(self.error.item())
        if not bits:
            return
        self.error.zero_()
        names = ((KVQ_PAGED_ERR_WAIT, "a bounded wait ran out"),
                 (KVQ_PAGED_ERR_BAD_PAGE, "a page id outside the pool"),
                 (KVQ_PAGED_ERR_NO_PAGES, "the free stack ran out"),
                 (KVQ_PAGED_ERR_LENGTH, "a length breaks the call's contract"),
                 (KVQ_PAGED_ERR_NONFINITE, "a non-finite key or value"))
        what = ", ".join(n for b, n in names if bits & b)
        raise KvqError(KVQ_ERR_DEVICE_CHECK, f"{type(self).__name__}.check: {what}")
