"""Device-memory holder for one attention layer's paged cache (PyTorch plumbing).

Allocates the buffers include/resa.h describes as torch CUDA tensors and
builds the C structs; all computation goes through block_sparse_long_resa_b200.resa.
"""
from __future__ import annotations

from dataclasses import dataclass
from typing import Optional

import torch

from . import resa


@dataclass
class LayerCache:
    k: torch.Tensor            # [num_pages][Hkv][b][d] bf16
    v: torch.Tensor
    desc: torch.Tensor         # [num_pages][Hkv][2][d] bf16
    page_table: torch.Tensor   # [B][max_pages] int32
    seq_len: torch.Tensor      # [B] int32 (tokens incl. the decode token)

    @classmethod
    def from_problem(cls, p, device) -> "LayerCache":
        dev = torch.device(device)
        k = p.k_cache.to(dev)
        return cls(k=k, v=p.v_cache.to(dev),
                   desc=torch.zeros(p.num_pages, p.num_kv_heads, 2, p.head_dim,
                                    dtype=torch.bfloat16, device=dev),
                   page_table=p.page_table.to(dev), seq_len=p.ctx_len.to(dev).clone())

    def struct(self, seq_len=None, rows=None) -> resa.resa_cache_t:
        """The C struct; ``rows`` (int32 device tensor) restricts a call to
        those rows of the page table, in that order."""
        return resa.make_cache(self.k, self.v, self.desc, self.page_table,
                               self.seq_len if seq_len is None else seq_len, rows)

    @property
    def batch(self) -> int:
        return int(self.page_table.shape[0])

    @property
    def max_pages(self) -> int:
        return int(self.page_table.shape[1])


@dataclass
class LayerCacheQ4:
    """The same of a 4-bit cache (resa_cache_q4_t)."""
    k: torch.Tensor            # [num_pages][Hkv][b][d / 2] uint8, two codes a byte
    v: torch.Tensor
    k_sf: torch.Tensor         # [num_pages][Hkv][b][d / 16] float8_e4m3fn
    v_sf: torch.Tensor
    desc: torch.Tensor         # [num_pages][Hkv][2][d] bf16
    page_table: torch.Tensor   # [B][max_pages] int32
    seq_len: torch.Tensor      # [B] int32
    k_scale: Optional[torch.Tensor] = None   # [Hkv] fp32, positive; None: 1
    v_scale: Optional[torch.Tensor] = None

    @classmethod
    def empty(cls, num_pages: int, num_kv_heads: int, block_size: int, head_dim: int,
              page_table: torch.Tensor, k_scale=None, v_scale=None) -> "LayerCacheQ4":
        """A cache without tokens (every seq_len 0) over the pages that page_table names."""
        dev, rows = page_table.device, (num_pages, num_kv_heads, block_size)
        codes = lambda: torch.zeros(*rows, head_dim // 2, dtype=torch.uint8, device=dev)
        scales = lambda: torch.zeros(*rows, head_dim // 16, dtype=torch.float8_e4m3fn, device=dev)
        return cls(k=codes(), v=codes(), k_sf=scales(), v_sf=scales(),
                   desc=torch.zeros(num_pages, num_kv_heads, 2, head_dim, dtype=torch.bfloat16,
                                    device=dev),
                   page_table=page_table,
                   seq_len=torch.zeros(page_table.shape[0], dtype=torch.int32, device=dev),
                   k_scale=k_scale, v_scale=v_scale)

    def struct(self, seq_len=None, rows=None) -> resa.resa_cache_q4_t:
        return resa.make_cache_q4(self.k, self.k_sf, self.v, self.v_sf, self.desc, self.page_table,
                                  self.seq_len if seq_len is None else seq_len, rows,
                                  self.k_scale, self.v_scale)

    def select_struct(self, seq_len=None, rows=None) -> resa.resa_cache_t:
        """What resa_select_blocks takes: the descriptors (it reads neither keys nor values)."""
        return resa.make_cache(self.k, self.v, self.desc, self.page_table,
                               self.seq_len if seq_len is None else seq_len, rows)

    @property
    def batch(self) -> int:
        return int(self.page_table.shape[0])

    @property
    def max_pages(self) -> int:
        return int(self.page_table.shape[1])


def workspace(cfg: resa.resa_config_t, batch: int, max_pages: int, max_chunk: int, device,
              stream=None) -> torch.Tensor:
    """Allocate and zero a workspace tensor for the given sizes."""
    n = resa.resa_workspace_size(cfg, batch, max_pages, max_chunk)
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    resa.resa_workspace_init(ws, stream)
    return ws
