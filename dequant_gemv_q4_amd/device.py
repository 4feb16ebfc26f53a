"""Torch-side plumbing around libqgemv: device buffers for packed weights and workspaces.

torch only provides device memory and the stream here; every byte of the packed layout is
written by the library's own pack kernel.
"""
from __future__ import annotations

import numpy as np
import torch

from . import _binding as B


def to_device(a, device="cuda") -> torch.Tensor:
    """Host numpy array -> contiguous device tensor (synchronous copy)."""
    a = np.ascontiguousarray(a)
    if not a.flags.writeable:
        a = a.copy()
    return torch.from_numpy(a).to(device)


def pack(fmt: int, w_gguf, N: int, K: int, device="cuda", stream=None,
         codebook=None) -> torch.Tensor:
    """GGUF-native blocks (numpy uint8 [N, row_bytes] or a device tensor) -> packed device buffer.

    codebook: the 16 signed entries of the IQ4 formats (host values), None for the others."""
    src = w_gguf if isinstance(w_gguf, torch.Tensor) else to_device(w_gguf, device)
    nbytes = B.qgemv_packed_bytes(fmt, N, K)
    if nbytes < 0:
        raise ValueError(f"invalid format/shape for packing: fmt={fmt} N={N} K={K}")
    out = torch.empty(nbytes, dtype=torch.uint8, device=src.device)
    if codebook is None:
        B.qgemv_pack(fmt, src, N, K, out, stream=stream)
    else:
        B.qgemv_pack_codebook(fmt, src, N, K, codebook, out, stream=stream)
    return out


def workspace(op: int, fmt: int, N: int, K: int, nb: int, n_exp: int = 0, topk: int = 0,
              device="cuda") -> torch.Tensor | None:
    """Zero-filled workspace of the size the operation needs (None if it needs none)."""
    n = B.qgemv_workspace_bytes(op, fmt, N, K, nb, n_exp, topk)
    if n < 0:
        raise ValueError("invalid sizes for the workspace query")
    if n == 0:
        return None
    return torch.zeros(n, dtype=torch.uint8, device=device)


def kv_pages(kv_type: int, n_pages: int, page_size: int, n_kv_heads: int, head_dim: int,
             device="cuda") -> tuple[torch.Tensor, torch.Tensor]:
    """Uninitialised page arrays of a key-value cache, packed (page_stride = n_kv_heads * block):
    K [n_pages][n_kv_heads][page_size][head_dim] and V [n_pages][n_kv_heads][head_dim][page_size]; of
    the 8-bit types uint8 [n_pages][n_kv_heads][page_size * (head_dim + 4)], whose parts
    :func:`kv_parts` shows."""
    if kv_type in (B.I8, B.F8):
        shape = (n_pages, n_kv_heads, page_size * (head_dim + 4))
        return tuple(torch.empty(shape, dtype=torch.uint8, device=device) for _ in range(2))
    dt = {B.F16: torch.float16, B.BF16: torch.bfloat16}[kv_type]
    return (torch.empty((n_pages, n_kv_heads, page_size, head_dim), dtype=dt, device=device),
            torch.empty((n_pages, n_kv_heads, head_dim, page_size), dtype=dt, device=device))


def kv_parts(kv_type: int, k_pages: torch.Tensor, v_pages: torch.Tensor, page_size: int,
             head_dim: int) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor]:
    """Views of 8-bit page arrays as :func:`kv_pages` makes them: codes of K [..][page_size][head_dim]
    (int8 or float8_e4m3fn) and their scales [..][page_size], then codes of V [..][head_dim][page_size]
    and theirs.  A value is scale * code."""
    dt = {B.I8: torch.int8, B.F8: torch.float8_e4m3fn}[kv_type]
    n = page_size * head_dim
    return (k_pages[..., :n].unflatten(-1, (page_size, head_dim)).view(dt),
            k_pages[..., n:].view(torch.float32),
            v_pages[..., :n].unflatten(-1, (head_dim, page_size)).view(dt),
            v_pages[..., n:].view(torch.float32))


def attn_workspace(op: int, n_seq: int, n_q_heads: int, n_kv_heads: int, head_dim: int,
                   device="cuda") -> torch.Tensor:
    """Zero-filled workspace of an attention-side operation (OP_KV_APPEND, OP_QKV_APPEND, OP_ATTN,
    OP_ATTN_PROMPT, OP_ATTN_SHARED)."""
    n = B.qgemv_attn_workspace_bytes(op, n_seq, n_q_heads, n_kv_heads, head_dim)
    if n < 0:
        raise ValueError("invalid sizes for the workspace query")
    return torch.zeros(n, dtype=torch.uint8, device=device)
