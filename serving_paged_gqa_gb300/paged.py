"""Python binding of the calls of libpkv.so over a cache that grows by chunks and is read in part (include/pkv.h, "chunks,
tables and selected pages").

The ``pkv_*`` functions are thin wrappers of the same-named C calls; the others take the description of the problem from the
tensors. Argument marshalling only: the work runs in the library's CUDA kernels, on the device of the tensors.
"""

from __future__ import annotations

import ctypes
import functools
import math

import torch

from ._lib import PKV_PROMPT_WS_BYTES, Problem, Prompt, check, load
from .prompts import _addr, _byref, _call, _device, _fits, _handle, _new, _num_sms, _pool, _rows, _scratch, _seqs, _start, _table

__all__ = [
    "pkv_chunk_workspace_bytes", "pkv_chunk_attention", "pkv_tables_grow", "pkv_tables_release", "pkv_page_bounds",
    "pkv_sparse_workspace_bytes", "pkv_select_pages", "pkv_sparse_decode_step",
    "chunk_attention", "tables_grow", "tables_release", "page_bounds", "sparse_problem", "select_pages", "sparse_decode",
]


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


def _ptrs(dev: int, dtype, *wants) -> list:
    """The addresses of tensors (tensor, entries, name) on the device; of None, None. (The calls on tables and bounds take less time
    on the GPU than here, so a tensor is looked at once, and what was wrong with it is found out afterwards.)"""
    at = []
    for t, n, name in wants:
        if t is None:
            at.append(None)
        elif t.dtype is dtype and t.numel() == n and t.get_device() == dev and t.is_contiguous():
            at.append(t.data_ptr())
        elif t.get_device() != dev:
            raise ValueError(f"the tensors must be on one device: {name} is on {t.device}, others on cuda:{dev}")
        elif t.numel() != n:
            raise ValueError(f"{name} must have {n} entries, got {t.numel()}")
        else:
            at.append(_addr(t, dtype, name))
    return at


def _ints(t, name: str, n: int) -> int:
    """The address of a tensor of n integers."""
    if t.numel() != n:
        raise ValueError(f"{name} must have {n} entries, got {t.numel()}")
    return _addr(t, torch.int32, name)


@functools.lru_cache(maxsize=256)
def _described(*args):
    """A reference to the description of these sizes, for calls that only read it."""
    return _byref(Problem(*args))


@functools.lru_cache(maxsize=256)
def _packed(num_seqs, tokens, hkv, d):
    """The same for contiguous packed keys."""
    return _byref(Prompt(num_seqs, tokens, hkv, hkv, d, 0, hkv * d, hkv * d, hkv * d, hkv * d))


def _shape(block_table: torch.Tensor, batch: int | None = None, pages: int | None = None) -> tuple[int, int]:
    if block_table.dim() != 2 or (batch is not None and tuple(block_table.shape) != (batch, pages)):
        raise ValueError(f"block_table must have shape ({'B' if batch is None else batch}, {'max_pages' if pages is None else pages})")
    return block_table.shape


def _grow(dev, problem, b, num_pages, entries, new_tokens, seq_lens, block_table, free_pages, free_count, cu_seqlens, start, slots,
          positions, seq_lens_out, free_count_out, ws, stream) -> None:
    cap = slots.numel() if slots is not None else positions.numel() if positions is not None else 0
    n, lens, table, pages, count, cu, first, pos, lens_out, count_out = _ptrs(
        dev, torch.int32, (new_tokens, b, "new_tokens"), (seq_lens, b, "seq_lens"), (block_table, entries, "block_table"),
        (free_pages, num_pages, "free_pages"), (free_count, 1, "free_count"), (cu_seqlens, b + 1, "cu_seqlens"), (start, b, "start"),
        (positions, cap, "positions"), (seq_lens_out, b, "seq_lens_out"), (free_count_out, 1, "free_count_out"))
    to, = _ptrs(dev, torch.int64, (slots, cap, "slots"))
    nbytes = ws.numel()
    wsp, = _ptrs(dev, torch.uint8, (ws, nbytes, "ws"))
    if cap == 0 and wsp:
        # Slots or positions without entries have no address, which would say that none are asked for and any number fits. Any other
        # address does: nothing is written to 0 entries.
        to = None if slots is None else wsp
        pos = None if positions is None else wsp + 16
    _call(dev, "pkv_tables_grow", problem, n, lens, table, pages, count, cu, first, to, pos, cap, lens_out, count_out, _num_sms(dev),
          wsp, nbytes, _handle(stream, dev))


def pkv_tables_grow(problem: Problem, new_tokens, seq_lens, block_table, free_pages, free_count, cu_seqlens, start, slots,
                    positions, seq_lens_out, free_count_out, ws, stream=None) -> None:
    b, width = _shape(block_table, problem.batch, problem.max_pages_per_seq)
    _grow(_device(new_tokens), _byref(problem), b, problem.num_pages, b * width, new_tokens, seq_lens, block_table, free_pages,
          free_count, cu_seqlens, start, slots, positions, seq_lens_out, free_count_out, ws, stream)


def _release(dev, problem, b, num_pages, entries, released, seq_lens, block_table, free_pages, free_count, seq_lens_out,
             free_count_out, ws, stream) -> None:
    ended, lens, table, pages, count, lens_out, count_out = _ptrs(
        dev, torch.int32, (released, b, "released"), (seq_lens, b, "seq_lens"), (block_table, entries, "block_table"),
        (free_pages, num_pages, "free_pages"), (free_count, 1, "free_count"), (seq_lens_out, b, "seq_lens_out"),
        (free_count_out, 1, "free_count_out"))
    nbytes = ws.numel()
    wsp, = _ptrs(dev, torch.uint8, (ws, nbytes, "ws"))
    _call(dev, "pkv_tables_release", problem, ended, lens, table, pages, count, lens_out, count_out, _num_sms(dev), wsp, nbytes,
          _handle(stream, dev))


def pkv_tables_release(problem: Problem, released, seq_lens, block_table, free_pages, free_count, seq_lens_out, free_count_out,
                       ws, stream=None) -> None:
    b, width = _shape(block_table, problem.batch, problem.max_pages_per_seq)
    _release(_device(released), _byref(problem), b, problem.num_pages, b * width, released, seq_lens, block_table, free_pages,
             free_count, seq_lens_out, free_count_out, ws, stream)


def _bounds(t: torch.Tensor, problem: Problem) -> int:
    want = (problem.num_pages, problem.num_kv_heads, 2, problem.head_dim)
    if t.shape != want:
        raise ValueError(f"bounds must have shape {want}, got {tuple(t.shape)}")
    return _addr(t, torch.float16, "bounds")


def _page_bounds(dev, problem, prompt, n, entries, cu_seqlens, start, k_pool, block_table, bounds, ws, stream) -> None:
    cu, first, table = _ptrs(dev, torch.int32, (cu_seqlens, n + 1, "cu_seqlens"), (start, n, "start"),
                             (block_table, entries, "block_table"))
    k, out = _ptrs(dev, torch.float16, (k_pool, k_pool.numel(), "k_pool"), (bounds, bounds.numel(), "bounds"))
    nbytes = ws.numel()
    wsp, = _ptrs(dev, torch.uint8, (ws, nbytes, "ws"))
    _call(dev, "pkv_page_bounds", problem, prompt, cu, first, k, table, out, _num_sms(dev), wsp, nbytes, _handle(stream, dev))


def pkv_page_bounds(problem: Problem, prompt: Prompt, cu_seqlens, start, k_pool, block_table, bounds, ws, stream=None) -> None:
    dev = _device(k_pool)
    _pool(k_pool, "k_pool", problem, prompt)
    _bounds(bounds, problem)
    b, width = _shape(block_table, problem.batch, problem.max_pages_per_seq)
    _page_bounds(dev, _byref(problem), _byref(prompt), prompt.num_seqs, b * width, cu_seqlens, start, k_pool, block_table, bounds, ws,
                 stream)


def pkv_sparse_workspace_bytes(problem: Problem, num_sms: int | None = None) -> int:
    """Bytes of the workspace of a page selection and the step over its pages (num_sms None: that of the current device)."""
    if num_sms is None:
        num_sms = _num_sms(torch.cuda.current_device())
    n = ctypes.c_size_t(0)
    check(load().pkv_sparse_workspace_bytes(_byref(problem), int(num_sms), _byref(n)), "pkv_sparse_workspace_bytes")
    return int(n.value)


def _queries(t: torch.Tensor, name: str, problem: Problem) -> int:
    want = (problem.batch, problem.num_q_heads, problem.head_dim)
    if t.shape != want:
        raise ValueError(f"{name} must have shape {want}, got {tuple(t.shape)}")
    return _addr(t, torch.float16, name)


def _selected(pages: torch.Tensor, problem: Problem) -> int:
    if pages.dim() != 3 or pages.shape[:2] != (problem.batch, problem.num_kv_heads):
        raise ValueError(f"pages must be [{problem.batch}, {problem.num_kv_heads}, select]")
    return _addr(pages, torch.int32, "pages")


def pkv_select_pages(problem: Problem, q, bounds, block_table, seq_lens, pages, ws, stream=None) -> None:
    dev = _device(q, bounds, block_table, seq_lens, pages, ws)
    _call(dev, "pkv_select_pages", _byref(problem), _queries(q, "q", problem), _bounds(bounds, problem),
          _table(block_table, problem), _ints(seq_lens, "seq_lens", problem.batch), pages.shape[-1], _num_sms(dev),
          _addr(ws, torch.uint8, "ws"), ws.numel(), _selected(pages, problem), _handle(stream, dev))


def pkv_sparse_decode_step(problem: Problem, q, k_pool, v_pool, block_table, seq_lens, pages, scale, ws, out,
                           stream=None) -> None:
    dev = _device(q, k_pool, v_pool, block_table, seq_lens, pages, ws, out)
    want = (problem.num_pages, problem.page_size, problem.num_kv_heads, problem.head_dim)
    for t, name in ((k_pool, "k_pool"), (v_pool, "v_pool")):
        if t.shape != want:
            raise ValueError(f"{name} must have shape {want}, got {tuple(t.shape)}")
    _call(dev, "pkv_sparse_decode_step", _byref(problem), _queries(q, "q", problem), _addr(k_pool, torch.float16, "k_pool"),
          _addr(v_pool, torch.float16, "v_pool"), _table(block_table, problem), _ints(seq_lens, "seq_lens", problem.batch),
          _selected(pages, problem), pages.shape[-1], scale, _num_sms(dev), _addr(ws, torch.uint8, "ws"), ws.numel(),
          _queries(out, "out", problem), _handle(stream, dev))


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


def tables_grow(new_tokens: torch.Tensor, seq_lens: torch.Tensor, block_table: torch.Tensor, free_pages: torch.Tensor,
                free_count: torch.Tensor, cu_seqlens: torch.Tensor | None = None, start: torch.Tensor | None = None,
                slots: torch.Tensor | None = None, positions: torch.Tensor | None = None,
                seq_lens_out: torch.Tensor | None = None, free_count_out: torch.Tensor | None = None,
                ws: torch.Tensor | None = None, stream=None):
    """Pages and packed rows for the rows' new tokens (include/pkv.h, pkv_tables_grow). Returns cu_seqlens, start.

    new_tokens, seq_lens [B], block_table [B, max_pages], free_pages [num_pages], free_count [1] int32 on the device: row b
    holds seq_lens[b] tokens and gets new_tokens[b] more; the first free_count entries of free_pages are the stack of free
    pages. block_table gets the new pages' entries; seq_lens_out and free_count_out (None: seq_lens and free_count themselves)
    the lengths and the stack's height afterwards; cu_seqlens [B + 1] and start [B] (made here where they are not given) what
    prompt_append and chunk_attention take; slots (int64) and positions (int32), one entry for each packed new token, where
    they are given, the token's page * 16 + slot and its position. Rows whose new tokens they have no entries for get nothing (none
    has where they have no entries at all).
    """
    b = new_tokens.numel()
    dev = _device(new_tokens)
    if cu_seqlens is None:
        cu_seqlens = _new((b + 1,), dev, stream, torch.int32)
    if start is None:
        start = _new((b,), dev, stream, torch.int32)
    num_pages, width = free_pages.numel(), _shape(block_table)[1]
    _grow(dev, _described(b, 1, 1, 128, 16, num_pages, width), b, num_pages, b * width, new_tokens, seq_lens, block_table, free_pages,
          free_count, cu_seqlens, start, slots, positions, seq_lens if seq_lens_out is None else seq_lens_out,
          free_count if free_count_out is None else free_count_out, _scratch(PKV_PROMPT_WS_BYTES, ws, dev, stream), stream)
    return cu_seqlens, start


def tables_release(released: torch.Tensor, seq_lens: torch.Tensor, block_table: torch.Tensor, free_pages: torch.Tensor,
                   free_count: torch.Tensor, seq_lens_out: torch.Tensor | None = None,
                   free_count_out: torch.Tensor | None = None, ws: torch.Tensor | None = None, stream=None) -> None:
    """The pages of the rows with released != 0 back on the stack (include/pkv.h, pkv_tables_release); released [B] int32, the
    others as for tables_grow."""
    b = released.numel()
    dev = _device(released)
    num_pages, width = free_pages.numel(), _shape(block_table)[1]
    _release(dev, _described(b, 1, 1, 128, 16, num_pages, width), b, num_pages, b * width, released, seq_lens, block_table, free_pages,
             free_count, seq_lens if seq_lens_out is None else seq_lens_out,
             free_count if free_count_out is None else free_count_out, _scratch(PKV_PROMPT_WS_BYTES, ws, dev, stream), stream)


def page_bounds(k_pool: torch.Tensor, cu_seqlens: torch.Tensor, block_table: torch.Tensor, bounds: torch.Tensor,
                start: torch.Tensor | None = None, ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Bounds of the pages that packed new tokens went to (include/pkv.h, pkv_page_bounds). Returns bounds.

    k_pool [num_pages, 16, Hkv, d]; bounds [num_pages, Hkv, 2, d] fp16, the least and the greatest key of each page; cu_seqlens,
    start and block_table as for the prompt_append that wrote the tokens. (Nothing here knows how many new tokens there are but
    the device: the work is bounded by the pages of the table.)
    """
    if k_pool.dim() != 4:
        raise ValueError("k_pool must be [num_pages, page_size, Hkv, d]")
    pages, ps, hkv, d = k_pool.shape
    if bounds.shape != (pages, hkv, 2, d):
        raise ValueError(f"bounds must have shape ({pages}, {hkv}, 2, {d}), got {tuple(bounds.shape)}")
    b, width = _shape(block_table)
    dev = _device(k_pool)
    n = cu_seqlens.numel() - 1
    # Packed rows are not read, and where the sequences begin among them is not known: any place is in order.
    _page_bounds(dev, _described(b, hkv, hkv, d, ps, pages, width), _packed(n, 0x7fffffff if width else 0, hkv, d), n, b * width,
                 cu_seqlens, start, k_pool, block_table, bounds, _scratch(PKV_PROMPT_WS_BYTES, ws, dev, stream), stream)
    return bounds


def sparse_problem(q: torch.Tensor, k_pool: torch.Tensor, block_table: torch.Tensor) -> Problem:
    """The problem of a step over selected pages: q [B, Hq, d], k_pool [num_pages, 16, Hkv, d], block_table [B, max_pages]."""
    b, hq, d = q.shape
    return Problem(b, hq, k_pool.shape[2], d, k_pool.shape[1], k_pool.shape[0], block_table.shape[1])


def select_pages(q: torch.Tensor, bounds: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor, select: int,
                 pages: torch.Tensor | None = None, ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The pages that a decode step attends to (include/pkv.h, pkv_select_pages). Returns pages [B, Hkv, select] int32.

    q [B, Hq, d] fp16; bounds [num_pages, Hkv, 2, d] (page_bounds); block_table [B, max_pages], seq_lens [B] int32. Keep ws
    (pkv_sparse_workspace_bytes, alloc_workspace) over the steps of a loop; sparse_decode takes the same.
    """
    if bounds.dim() != 4:
        raise ValueError("bounds must be [num_pages, Hkv, 2, d]")
    b, hq, d = q.shape
    problem = Problem(b, hq, bounds.shape[1], d, 16, bounds.shape[0], block_table.shape[1])
    dev = _device(q)
    if pages is None:
        pages = _new((b, bounds.shape[1], int(select)), dev, stream, torch.int32)
    elif pages.shape[-1] != select:
        raise ValueError(f"pages has room for {pages.shape[-1]} pages, select is {select}")
    if ws is None:
        ws = _scratch(pkv_sparse_workspace_bytes(problem, _num_sms(dev)), None, dev, stream)
    pkv_select_pages(problem, q, bounds, block_table, seq_lens, pages, ws, stream)
    return pages


def sparse_decode(q: torch.Tensor, k_pool: torch.Tensor, v_pool: torch.Tensor, block_table: torch.Tensor,
                  seq_lens: torch.Tensor, pages: torch.Tensor, scale: float | None = None, out: torch.Tensor | None = None,
                  ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """One decode step over the pages that select_pages chose (include/pkv.h, pkv_sparse_decode_step). Returns out [B, Hq, d].

    q [B, Hq, d] fp16; k_pool, v_pool [num_pages, 16, Hkv, d]; block_table [B, max_pages], seq_lens [B], pages [B, Hkv,
    select] int32 on the device.
    """
    _pools(k_pool, v_pool, q.shape[-1])
    problem = sparse_problem(q, k_pool, block_table)
    dev = _device(q)
    if out is None:
        out = _new(tuple(q.shape), dev, stream)
    if ws is None:
        ws = _scratch(pkv_sparse_workspace_bytes(problem, _num_sms(dev)), None, dev, stream)
    pkv_sparse_decode_step(problem, q, k_pool, v_pool, block_table, seq_lens, pages,
                           1.0 / math.sqrt(q.shape[2]) if scale is None else scale, ws, out, stream)
    return out
