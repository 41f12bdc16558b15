"""Binding of the paged 4-bit cache's calls (include/kvq.h): the paged cache of
paged.py over pages of 4-bit codes with an fp16 step and minimum for each token,
kv head and group of 32 channels.

Codes are uint8 tensors [n_pages][n_kv_heads][page_size][head_dim / 2], metadata
fp16 tensors [n_pages][n_kv_heads][page_size][head_dim / 32][2]; tables, lengths
and slots are those of kvq_paged_plan.  What paged.py says of streams, graphs,
errors and gradients holds here too.
"""
from __future__ import annotations

import ctypes

import torch

from . import kvq
from .kvq import kvq_paged4_pool
from .paged import PagedCache, _paged_bind, _sizes

_append = _paged_bind.append4
_read = _paged_bind.read4
_attention = _paged_bind.attention4


def kvq_paged4_pool_check(n_pages: int, n_kv_heads: int, page_size: int, head_dim: int) -> int:
    """Status of a pool's sizes (KVQ_OK when the calls take such a pool)."""
    pool = kvq_paged4_pool(None, None, None, None, *_sizes(n_pages, n_kv_heads, page_size, head_dim))
    return kvq._lib.kvq_paged4_pool_check(ctypes.byref(pool))


def kvq_paged4_workspace_bytes(n_pages: int, n_kv_heads: int, page_size: int,
                               head_dim: int) -> int:
    """Bytes of the attention's workspace for such a pool."""
    pool = kvq_paged4_pool(None, None, None, None, *_sizes(n_pages, n_kv_heads, page_size, head_dim))
    n = ctypes.c_size_t(0)
    kvq._check(kvq._lib.kvq_paged4_workspace_bytes(ctypes.byref(pool), ctypes.byref(n)),
               "kvq_paged4_workspace_bytes")
    return n.value


def kvq_paged4_append(k, v, slots, k_codes, v_codes, k_meta, v_meta, angles=None, interleaved=False,
                      q=None, q_out=None, error=None, stream=None):
    """Stores keys and values k, v (fp16 or bf16 [tokens][n_kv_heads][head_dim],
    any token stride that is a multiple of 8) at their slots (int32 [tokens],
    negative: nowhere).  With `angles` (kvq_rotary_angles) the keys are turned on
    the way, and so are the step's queries q where given; they are returned
    (q_out, which may be q itself, or a new tensor)."""
    return _append(k, v, slots, k_codes, v_codes, k_meta, v_meta, angles, interleaved, q, q_out,
                   error, stream)


def kvq_paged4_read(slots, k_codes, v_codes, k_meta, v_meta, k=None, v=None, error=None,
                    stream=None):
    """The stored keys and values of slots (int32 [tokens]; a negative one gives
    zeros) as fp16 [tokens][n_kv_heads][head_dim]: (k, v)."""
    return _read(slots, k_codes, v_codes, k_meta, v_meta, k, v, error, stream)


def kvq_paged4_attention(q, k_codes, v_codes, k_meta, v_meta, block_table, cu_new, seq_len,
                         max_new: int = 1, softmax_scale: float | None = None, window: int = 0,
                         out=None, workspace=None, error=None, stream=None):
    """Attention of the new tokens over the pages; returns out, in q's type.
    Arguments and workspaces as for kvq_paged_attention."""
    return _attention(q, k_codes, v_codes, k_meta, v_meta, block_table, cu_new, seq_len, max_new,
                      softmax_scale, window, out, workspace, error, stream)


class PagedCache4(PagedCache):
    """One layer's paged 4-bit KV cache: PagedCache's calls over 4-bit pages, 5
    bits a value instead of 8.

    A step with rotary positions is::

        cache = PagedCache4(n_pages=4096, page_size=64, n_q_heads=32, n_kv_heads=8,
                            head_dim=128)
        cu, seq, slots, left = cache.plan(ctx_len, new_len, block_table, free_pages, n_free,
                                          n_tokens, positions=positions)
        angles = kvq_rotary_angles(positions, turns)
        q = cache.append(k, v, slots, angles, q=q)
        out = cache.attention(q, block_table, cu, seq, max_new=1)

    The step's plan and angles serve every layer's cache."""

    def _make_pool(self, n_pages, n_kv_heads, page_size, head_dim, device):
        kvq._check(kvq_paged4_pool_check(n_pages, n_kv_heads, page_size, head_dim),
                   "kvq_paged4_pool_check")
        codes = (n_pages, n_kv_heads, page_size, head_dim // 2)
        meta = (n_pages, n_kv_heads, page_size, head_dim // 32, 2)
        self.k_codes, self.v_codes = (torch.zeros(codes, dtype=torch.uint8, device=device) for _ in "kv")
        self.k_meta, self.v_meta = (torch.zeros(meta, dtype=torch.float16, device=device) for _ in "kv")

    def _pool(self):
        return self.k_codes, self.v_codes, self.k_meta, self.v_meta

    _store_call = _append_call = staticmethod(kvq_paged4_append)
    _attention_call = staticmethod(kvq_paged4_attention)

    def read(self, slots, k=None, v=None, stream=None):
        """The keys and values that `slots` hold, fp16 [slots][n_kv_heads][head_dim]."""
        return kvq_paged4_read(slots, *self._pool(), k=k, v=v, error=self.error, stream=stream)
