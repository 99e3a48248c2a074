"""Python binding of the calls of libpkv.so over a cache that grows by chunks and is read in part (include/pkv.h, "chunks,
tables and selected pages").

The ``pkv_*`` functions are thin wrappers of the same-named C calls; the others take the description of the problem from the
tensors. Argument marshalling only: the work runs in the library's CUDA kernels, on the device of the tensors.
"""

from __future__ import annotations

import ctypes
import math

import torch

from ._lib import Problem, Prompt, check, load
from .prompts import _addr, _byref, _call, _device, _fits, _handle, _new, _num_sms, _pool, _rows, _scratch, _seqs, _start, _table

__all__ = ["pkv_chunk_workspace_bytes", "pkv_chunk_attention", "chunk_attention"]


def pkv_chunk_workspace_bytes(num_sms: int | None = None) -> int:
    """Bytes of the workspace of a chunk's attention (num_sms None: that of the current device)."""
    if num_sms is None:
        num_sms = _num_sms(torch.cuda.current_device())
    n = ctypes.c_size_t(0)
    check(load().pkv_chunk_workspace_bytes(int(num_sms), _byref(n)), "pkv_chunk_workspace_bytes")
    return int(n.value)


def _chunk(dev, problem, prompt, q, k_pool, v_pool, cu_seqlens, start, block_table, scale, ws, out, stream) -> None:
    n = prompt.num_seqs
    _call(dev, "pkv_chunk_attention", _byref(problem), _byref(prompt), q.data_ptr(), _addr(k_pool, torch.float16, "k_pool"),
          _addr(v_pool, torch.float16, "v_pool"), _seqs(cu_seqlens, n), _start(start, n), _table(block_table, problem), scale,
          _num_sms(dev), _addr(ws, torch.uint8, "ws"), ws.numel(), out.data_ptr(), _handle(stream, dev))


def pkv_chunk_attention(problem: Problem, prompt: Prompt, q, k_pool, v_pool, cu_seqlens, start, block_table, scale, ws, out,
                        stream=None) -> None:
    dev = _device(q, k_pool, v_pool, cu_seqlens, start, block_table, ws, out)
    _fits(q, "q", prompt, prompt.num_q_heads, prompt.q_stride)
    _fits(out, "out", prompt, prompt.num_q_heads, prompt.out_stride)
    _pool(k_pool, "k_pool", problem, prompt)
    _pool(v_pool, "v_pool", problem, prompt)
    _chunk(dev, problem, prompt, q, k_pool, v_pool, cu_seqlens, start, block_table, scale, ws, out, stream)


# ------------------------------------------------------------------------------- the same, described by the tensors
def _pools(k_pool: torch.Tensor, v_pool: torch.Tensor, d: int) -> int:
    """Checks a pair of FP16 pools; their KV heads."""
    if k_pool.dim() != 4 or k_pool.shape[3] != d or v_pool.shape != k_pool.shape:
        raise ValueError(f"k_pool and v_pool must be [num_pages, page_size, Hkv, {d}]")
    return k_pool.shape[2]


def chunk_attention(q: torch.Tensor, k_pool: torch.Tensor, v_pool: torch.Tensor, cu_seqlens: torch.Tensor,
                    block_table: torch.Tensor, start: torch.Tensor | None = None, scale: float | None = None,
                    out: torch.Tensor | None = None, ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Attention of packed new tokens over the FP16 pages that hold them and what came before (include/pkv.h,
    pkv_chunk_attention). Returns out [tokens, Hq, d] fp16.

    q [tokens, Hq, d] fp16, the heads of a token contiguous and the tokens at any distance; k_pool, v_pool [num_pages, 16, Hkv,
    d] fp16; cu_seqlens [num_seqs + 1], block_table [num_seqs, max_pages], start [num_seqs] (tokens that each row held before;
    None: none) int32 on the device. Keep ws (pkv_chunk_workspace_bytes, alloc_workspace) over the steps of a loop. Rows of an
    `out` given by the caller that belong to no sequence keep their values; in one made here they are undefined.
    """
    qs = _rows(q, "q")
    t, hq, d = q.shape
    hkv = _pools(k_pool, v_pool, d)
    dev = _device(q, k_pool, v_pool, cu_seqlens, start, block_table, ws, out)
    if out is None:
        out = _new((t, hq, d), dev, stream)
        os = hq * d
    else:
        os = _rows(out, "out", hq, t, d)
    b, pages = block_table.shape
    problem = Problem(b, hq, hkv, d, k_pool.shape[1], k_pool.shape[0], pages)
    prompt = Prompt(cu_seqlens.numel() - 1, t, hq, hkv, d, 0, qs, hkv * d, hkv * d, os)
    if ws is None:
        ws = _scratch(pkv_chunk_workspace_bytes(_num_sms(dev)), None, dev, stream)
    _chunk(dev, problem, prompt, q, k_pool, v_pool, cu_seqlens, start, block_table,
           1.0 / math.sqrt(d) if scale is None else scale, ws, out, stream)
    return out
