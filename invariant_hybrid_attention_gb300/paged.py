"""Device-side helpers for paged KV caches: allocation and page tables (PyTorch memory).

No attention arithmetic lives here; these only size and place caller-owned buffers in the
layout the C ABI expects: cache [num_pages][n_kv_heads][16][head_dim] bf16, page table
int32 [B][max_pages].
"""
from __future__ import annotations

from typing import Optional

import torch

from . import (PAGE_SIZE, g4attn_cache, g4attn_cache4, g4attn_cache8, g4attn_kv4_page_bytes, g4attn_kv8_page_bytes,
               make_cache, make_cache4, make_cache8)


ROT_DIMS = 128            # rotated columns of a global head: dims 0-63 and 256-319


def untile(t: torch.Tensor) -> torch.Tensor:
    """A cache tensor in the tiled page layout as plain rows [pages][heads][16][D]
    (D = 256: [2][32][8][8] per page-head; D = 512: two such 256-dim halves)."""
    P, H = t.shape[0], t.shape[1]
    n = t[0, 0].numel()
    D = n // PAGE_SIZE
    if D == 256:
        return t.reshape(P, H, 2, 32, 8, 8).permute(0, 1, 2, 4, 3, 5).reshape(P, H, PAGE_SIZE, 256)
    halves = t.reshape(P, H, 2, 2, 32, 8, 8).permute(0, 1, 3, 5, 2, 4, 6)   # [P][H][kg][j8][half][dg][d8]
    return halves.reshape(P, H, PAGE_SIZE, 512)


def tile(rows: torch.Tensor) -> torch.Tensor:
    """Plain rows [pages][heads][16][D] in the tiled page layout (inverse of `untile`)."""
    P, H, D = rows.shape[0], rows.shape[1], rows.shape[3]
    if D == 256:
        return rows.reshape(P, H, 2, 8, 32, 8).permute(0, 1, 2, 4, 3, 5).contiguous().reshape(P, H, 2, 32, 8, 8)
    r = rows.reshape(P, H, 2, 8, 2, 32, 8)          # [P][H][kg][j8][half][dg][d8]
    return r.permute(0, 1, 4, 2, 5, 3, 6).contiguous().reshape(P, H, 2, 2, 32, 8, 8)


def untile_v256(t: torch.Tensor) -> torch.Tensor:
    """A sliding V tensor [pages][heads][2][2][16][8][8] (two 128-dim halves per page-head block)
    as plain rows [pages][heads][16][256]."""
    P, H = t.shape[0], t.shape[1]
    r = t.reshape(P, H, 2, 2, 16, 8, 8).permute(0, 1, 3, 5, 2, 4, 6)   # [P][H][kg][j8][half][dg][d8]
    return r.reshape(P, H, PAGE_SIZE, 256)


def tile_v256(rows: torch.Tensor) -> torch.Tensor:
    """Plain rows [pages][heads][16][256] in the sliding V layout (inverse of `untile_v256`)."""
    P, H = rows.shape[0], rows.shape[1]
    r = rows.reshape(P, H, 2, 8, 2, 16, 8)          # [P][H][kg][j8][half][dg][d8]
    return r.permute(0, 1, 4, 2, 5, 3, 6).contiguous().reshape(P, H, 2, 2, 16, 8, 8)


def untile_rot(t: torch.Tensor) -> torch.Tensor:
    """A global k_rot tensor [pages][4][2][2][8][8][8] as rows [pages][4][16][128] holding dims
    0-63 then 256-319."""
    P, H = t.shape[0], t.shape[1]
    r = t.reshape(P, H, 2, 2, 8, 8, 8).permute(0, 1, 3, 5, 2, 4, 6)    # [P][H][kg][j8][half][dg][d8]
    return r.reshape(P, H, PAGE_SIZE, ROT_DIMS)


class PagedKV:
    """One layer's paged cache, pages stored as 8x8 core-matrix tiles (see include/g4attn.h).
    `v` is None on K==V (global) layers, which carry `k_rot` (the roped rotated columns)."""

    def __init__(self, num_pages: int, n_kv_heads: int, head_dim: int, shared: bool, device="cuda",
                 fill: Optional[float] = float("nan")):
        if int(head_dim) == 256:
            shape = (int(num_pages), int(n_kv_heads), 2, 32, 8, 8)
        else:
            shape = (int(num_pages), int(n_kv_heads), 2, 2, 32, 8, 8)
        self.k = torch.empty(shape, dtype=torch.bfloat16, device=device)
        # sliding V: two contiguous 128-dim halves per page-head block (see untile_v256)
        self.v = None if shared else torch.empty((int(num_pages), int(n_kv_heads), 2, 2, 16, 8, 8),
                                                 dtype=torch.bfloat16, device=device)
        self.k_rot = (torch.empty((int(num_pages), int(n_kv_heads), 2, 2, 8, 8, 8), dtype=torch.bfloat16,
                                  device=device) if shared else None)
        if fill is not None:
            for t in (self.k, self.v, self.k_rot):
                if t is not None:
                    t.fill_(fill)
        self.num_pages = int(num_pages)

    @property
    def desc(self) -> g4attn_cache:
        return make_cache(self.k, self.v, self.num_pages, self.k_rot)

    def nbytes(self) -> int:
        return sum(t.numel() * 2 for t in (self.k, self.v, self.k_rot) if t is not None)


class PagedKV8:
    """One layer's 8-bit paged cache: bytes [num_pages][n_kv_heads][block] (see include/g4attn.h)."""

    def __init__(self, layer, num_pages: int, device="cuda", fill: Optional[int] = 255):
        block = g4attn_kv8_page_bytes(layer) // int(layer.n_kv_heads)
        self.pages = torch.empty((int(num_pages), int(layer.n_kv_heads), block), dtype=torch.uint8, device=device)
        if fill is not None:
            self.pages.fill_(fill)
        self.num_pages = int(num_pages)

    @property
    def desc(self) -> g4attn_cache8:
        return make_cache8(self.pages, self.num_pages)


def untile8(pages: torch.Tensor, head_dim: int):
    """The two tensors an 8-bit cache holds, as fp32 values [pages][heads][16][columns]: sliding K' and V,
    global S and its 128 turned columns. Bytes [pages][heads][block] as in PagedKV8.pages."""
    cols = (256, 256) if int(head_dim) == 256 else (512, ROT_DIMS)
    j = torch.arange(PAGE_SIZE, device=pages.device)[:, None]
    piece = torch.arange(8, device=pages.device)[None, :] ^ (j & 6) ^ ((j & 1) << 2)
    out, at = [], 0
    for i, n in enumerate(cols):
        u = pages[..., at:at + PAGE_SIZE * n].unflatten(-1, (n // 128, PAGE_SIZE, 8, 16))[..., j, piece, :]
        e = pages[..., PAGE_SIZE * (sum(cols) + i):PAGE_SIZE * (sum(cols) + i + 1)].int()
        step = torch.where(e == 255, torch.full_like(e, 0x7FC00000), (e.clamp(8, 254) - 6) << 23).view(torch.float32)
        out.append((u.transpose(-4, -3).flatten(-3).float() - 128.0) * step[..., None])
        at += PAGE_SIZE * n
    return out


class PagedKV4:
    """One layer's 4-bit paged cache: bytes [num_pages][n_kv_heads][block] (see include/g4attn.h)."""

    def __init__(self, layer, num_pages: int, device="cuda", fill: Optional[int] = 255):
        block = g4attn_kv4_page_bytes(layer) // int(layer.n_kv_heads)
        self.pages = torch.empty((int(num_pages), int(layer.n_kv_heads), block), dtype=torch.uint8, device=device)
        if fill is not None:
            self.pages.fill_(fill)
        self.num_pages = int(num_pages)

    @property
    def desc(self) -> g4attn_cache4:
        return make_cache4(self.pages, self.num_pages)


def untile4(pages: torch.Tensor, head_dim: int):
    """The two tensors a 4-bit cache holds, as fp32 values [pages][heads][16][columns]: sliding K' and V,
    global S and its 128 turned columns. Bytes [pages][heads][block] as in PagedKV4.pages."""
    cols = (256, 256) if int(head_dim) == 256 else (512, ROT_DIMS)
    j = torch.arange(PAGE_SIZE, device=pages.device)[:, None]
    piece = torch.arange(8, device=pages.device)[None, :] ^ (j & 6) ^ ((j & 1) << 2)
    steps = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], device=pages.device)
    out, at, scale_at = [], 0, PAGE_SIZE * sum(cols) // 2
    for n in cols:
        u = pages[..., at:at + PAGE_SIZE * n // 2]
        if n == ROT_DIMS:   # [key][piece][block][half][2 bytes] -> [key][block][half][piece][2 bytes]
            u = u.unflatten(-1, (PAGE_SIZE, 4, 4, 2, 2)).movedim(-4, -2).flatten(-4)
        else:               # [segment][key][piece][block][2 bytes] -> [key][segment][block][piece][2 bytes]
            u = u.unflatten(-1, (n // 256, PAGE_SIZE, 8, 16))[..., j, piece, :].transpose(-4, -3)
            u = u.unflatten(-1, (8, 2)).transpose(-3, -2).flatten(-4)
        code = torch.stack([u & 15, u >> 4], -1).flatten(-2)                        # [pages][heads][16][n]
        s = pages[..., scale_at:scale_at + PAGE_SIZE * n // 32].unflatten(-1, (PAGE_SIZE, n // 32))
        factor = torch.where(s == 255, torch.full_like(s, float("nan"), dtype=torch.float32),
                             torch.exp2(s.float() - 127.0))
        out.append((steps[code.long()].unflatten(-1, (-1, 32)) * factor[..., None]).flatten(-2))
        at += PAGE_SIZE * n // 2
        scale_at += PAGE_SIZE * n // 32
    return out


def device_int32(values, device="cuda") -> torch.Tensor:
    return torch.as_tensor(values, dtype=torch.int32).to(device)
