"""A paged key-value cache and the rotary table that goes with it.

``PagedKV`` owns the buffers the attention entry points of ``api`` work on --
the pages of every layer in one pool, the sequences' page tables, lengths and
the pages' reference counts, all on the GPU -- and calls those entry points.
Nothing here waits for the GPU: sequence ids and counts are int32 tensors on
the device, so a step that admits, extends, forks or frees sequences can be
captured into a CUDA graph.  ("Distillix" README: grouped query heads, 12 Q / 4 KV,
rotary positions with theta = 1e6; "SLM750-Edge" section 2.2.)
"""
from __future__ import annotations

import torch

from . import api


def rope_table(positions: int, head_dim: int, theta: float = 1e6, device="cuda") -> torch.Tensor:
    """float32 [positions, head_dim]: cos of head_dim / 2 angles position *
    theta^(-2 i / head_dim), then their sin, from angles in float64 (a float32
    angle of a far position is off by more than the result's last bits)."""
    inv = theta ** (-torch.arange(0, head_dim, 2, dtype=torch.float64) / head_dim)
    ang = torch.arange(positions, dtype=torch.float64)[:, None] * inv[None]
    return torch.cat([ang.cos(), ang.sin()], 1).float().to(device)


class PagedKV:
    """layers x (K, V) pages [num_pages, kv_heads, page_size, head_dim] of
    `dtype` for up to max_seqs sequences of at most max_pages pages each."""

    def __init__(self, layers: int, num_pages: int, page_size: int, kv_heads: int, head_dim: int, max_seqs: int,
                 max_pages: int, dtype=torch.bfloat16, device="cuda"):
        if dtype not in (torch.float32, torch.bfloat16):
            raise ValueError(f"dtype must be float32 or bfloat16, got {dtype}")
        self.page_size, self.kv_heads, self.head_dim = page_size, kv_heads, head_dim
        self.pool = torch.zeros(layers, 2, num_pages, kv_heads, page_size, head_dim, dtype=dtype, device=device)
        self.tables = torch.full((max_seqs, max_pages), -1, dtype=torch.int32, device=device)
        self.lengths = torch.zeros(max_seqs, dtype=torch.int32, device=device)
        self.refs = torch.zeros(num_pages, dtype=torch.int32, device=device)

    def pages(self, layer: int):
        """(k_pages, v_pages) of a layer."""
        return self.pool[layer, 0], self.pool[layer, 1]

    def extend(self, seq_ids, counts, status=None, active=None, stream=None):
        """Room for counts[i] more tokens of sequence seq_ids[i] (its length grows
        at once; the rows are written by append) -> status int32 [1]."""
        return api.bl_kv_extend(self.tables, self.lengths, self.refs, seq_ids, counts, self.page_size, status, active,
                                stream)

    def free(self, seq_ids, stream=None):
        api.bl_kv_free(self.tables, self.lengths, self.refs, seq_ids, self.page_size, stream)

    def fork(self, src, dst, status=None, stream=None):
        """dst[i] (empty) continues src[i] on its own -> status int32 [1]."""
        return api.bl_kv_fork(self.pool, self.tables, self.lengths, self.refs, src, dst, status, stream=stream)

    def compact(self, n_live=None, stream=None):
        """Pages in use to the lowest numbers -> n_live int32 [1]."""
        return api.bl_kv_compact(self.pool, self.tables, self.refs, n_live, stream=stream)

    def append(self, layer: int, q, k, v, rope=None, cu_seqlens=None, seq_ids=None, out_dtype=None, keep_kv=False,
               stream=None):
        """Rotates q and k by their positions, writes k and v into the layer's
        pages (their sequences were extended before) -> (q, k, v) rotated and
        rounded to out_dtype; k and v only with keep_kv."""
        kp, vp = self.pages(layer)
        return api.bl_rope_append(q, k, v, rope, cu_seqlens, self.lengths, seq_ids, kp, vp, self.tables, out_dtype,
                                  keep_kv=keep_kv, stream=stream)

    def attend(self, layer: int, q, seq_ids=None, window: int = 0, sinks: int = 0, scale=None, out=None, lse=None,
               return_lse=False, stream=None):
        """Attention of one token per sequence over the layer's pages."""
        kp, vp = self.pages(layer)
        return api.bl_attn_decode(q, kp, vp, self.tables, self.lengths, seq_ids, window, sinks, scale, out, lse,
                                  return_lse, stream=stream)
