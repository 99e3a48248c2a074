"""Python binding of the prompt and 4-bit-cache calls of libpkv.so (include/pkv.h, "prompts and the 4-bit cache").

The ``pkv_*`` functions are thin wrappers of the same-named C calls; ``prompt_attention``, ``prompt_append``,
``q4_prompt_append``, ``q4_read`` and ``q4_decode`` take the description of the problem from the tensors. Argument
marshalling only: the work runs in the library's CUDA kernels, on the device of the tensors.
"""

from __future__ import annotations

import ctypes
import math

import torch

from ._lib import PKV_PROMPT_WS_BYTES, PKV_Q4_BLOCK_BYTES, Problem, Prompt, check, load
from .binding import alloc_workspace

__all__ = [
    "make_prompt", "pkv_check_prompt", "pkv_prompt_attention", "pkv_prompt_append", "pkv_q4_prompt_append",
    "pkv_q4_read", "pkv_q4_pool_bytes", "pkv_q4_workspace_bytes", "pkv_q4_decode_step", "pkv_q4_decode_step_append",
    "prompt_attention", "prompt_append", "q4_problem", "q4_prompt_append", "q4_read", "q4_decode",
]

# The marshalling of a call is on the path of every small step, so it stays with integers: pointers and streams are
# passed as numbers, devices are compared by their index.
_byref = ctypes.byref
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = torch.cuda.current_device
_functions: dict[str, object] = {}
_sms: dict[int, int] = {}


def _num_sms(device: int) -> int:
    n = _sms.get(device)
    if n is None:
        n = _sms[device] = torch.cuda.get_device_properties(device).multi_processor_count
    return n


def _device(first: torch.Tensor, *others) -> int:
    """The index of the device that all tensors are on."""
    i = first.get_device()
    if i < 0:
        raise ValueError("the tensors must be CUDA tensors")
    for t in others:
        if t is not None and t.get_device() != i:
            raise ValueError(f"the tensors must be on one device: {t.device} and {first.device}")
    return i


def _handle(stream, device: int) -> int:
    """The stream's handle; None: the device's current stream."""
    if stream is None:
        return _raw_stream(device) if _raw_stream else torch.cuda.current_stream(device).cuda_stream
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


def _call(device: int, name: str, *args) -> None:
    """Calls the library with `device` current (it launches on the current device)."""
    fn = _functions.get(name)
    if fn is None:
        fn = _functions[name] = getattr(load(), name)
    if device == _current_device():
        rc = fn(*args)
    else:
        with torch.cuda.device(device):
            rc = fn(*args)
    if rc != 0:
        check(rc, name)


def _addr(t: torch.Tensor | None, dtype, name: str) -> int | None:
    if t is None:
        return None
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _rows(t: torch.Tensor, name: str, heads: int | None = None, rows: int | None = None, d: int | None = None) -> int:
    """Checks a packed [tokens, heads, d] tensor whose tokens may be strided; returns the distance between tokens."""
    shape = t.shape
    if len(shape) != 3 or t.dtype != torch.float16:
        raise ValueError(f"{name} must be a float16 tensor [tokens, heads, d]")
    n, h, dim = shape
    if (heads is not None and h != heads) or (rows is not None and n != rows) or (d is not None and dim != d):
        raise ValueError(f"{name} has shape {tuple(shape)}, expected [{rows}, {heads}, {d}]")
    s0, s1, s2 = t.stride()
    if (s2 != 1 and dim > 1) or (s1 != dim and h > 1):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    return s0 if n > 1 else h * dim


def make_prompt(num_seqs, total_tokens, num_q_heads, num_kv_heads, head_dim, q_stride=None, k_stride=None,
                v_stride=None, out_stride=None) -> Prompt:
    """A prompt description; a stride that is not given is that of a contiguous tensor."""
    hq, hkv, d = int(num_q_heads), int(num_kv_heads), int(head_dim)
    return Prompt(int(num_seqs), int(total_tokens), hq, hkv, d, 0, hq * d if q_stride is None else int(q_stride),
                  hkv * d if k_stride is None else int(k_stride), hkv * d if v_stride is None else int(v_stride),
                  hq * d if out_stride is None else int(out_stride))


def pkv_check_prompt(prompt: Prompt) -> int:
    return load().pkv_check_prompt(_byref(prompt))


def _fits(t: torch.Tensor, name: str, prompt: Prompt, heads: int, stride: int) -> int:
    """Checks that a packed tensor is the one that the prompt describes; its address."""
    s = _rows(t, name, heads, prompt.total_tokens, prompt.head_dim)
    if s != stride and prompt.total_tokens > 1:
        raise ValueError(f"{name}: its tokens are {s} elements apart, the prompt says {stride}")
    return t.data_ptr()


def _seqs(cu_seqlens: torch.Tensor, num_seqs: int) -> int:
    if cu_seqlens.numel() != num_seqs + 1:
        raise ValueError(f"cu_seqlens must have {num_seqs + 1} entries")
    return _addr(cu_seqlens, torch.int32, "cu_seqlens")


def _start(start, num_seqs: int) -> int | None:
    if start is not None and start.numel() != num_seqs:
        raise ValueError(f"start must have {num_seqs} entries")
    return _addr(start, torch.int32, "start")


def _table(block_table: torch.Tensor, problem: Problem) -> int:
    if tuple(block_table.shape) != (problem.batch, problem.max_pages_per_seq):
        raise ValueError(f"block_table must have shape ({problem.batch}, {problem.max_pages_per_seq})")
    return _addr(block_table, torch.int32, "block_table")


def _pool(t: torch.Tensor, name: str, problem: Problem, prompt: Prompt) -> None:
    """Checks that a pool is the one that the problem describes (the kernels bound their pages by the problem)."""
    if name == "pool":
        want = (problem.num_pages, prompt.num_kv_heads, PKV_Q4_BLOCK_BYTES)
    else:
        want = (problem.num_pages, problem.page_size, prompt.num_kv_heads, prompt.head_dim)
    if t.shape != want:
        raise ValueError(f"{name} must have shape {want}, got {tuple(t.shape)}")


def _attention(dev, prompt, q, k, v, cu_seqlens, scale, ws, out, stream) -> None:
    _call(dev, "pkv_prompt_attention", _byref(prompt), q.data_ptr(), k.data_ptr(), v.data_ptr(),
          _seqs(cu_seqlens, prompt.num_seqs), scale, _num_sms(dev), _addr(ws, torch.uint8, "ws"), ws.numel(),
          out.data_ptr(), _handle(stream, dev))


def pkv_prompt_attention(prompt: Prompt, q, k, v, cu_seqlens, scale, ws, out, stream=None) -> None:
    dev = _device(q, k, v, cu_seqlens, ws, out)
    _fits(q, "q", prompt, prompt.num_q_heads, prompt.q_stride)
    _fits(k, "k", prompt, prompt.num_kv_heads, prompt.k_stride)
    _fits(v, "v", prompt, prompt.num_kv_heads, prompt.v_stride)
    _fits(out, "out", prompt, prompt.num_q_heads, prompt.out_stride)
    _attention(dev, prompt, q, k, v, cu_seqlens, scale, ws, out, stream)


def _append(dev, problem, prompt, k, v, cu_seqlens, start, k_pool, v_pool, block_table, ws, stream) -> None:
    n = prompt.num_seqs
    _call(dev, "pkv_prompt_append", _byref(problem), _byref(prompt), k.data_ptr(), v.data_ptr(), _seqs(cu_seqlens, n),
          _start(start, n), _addr(k_pool, torch.float16, "k_pool"), _addr(v_pool, torch.float16, "v_pool"),
          _table(block_table, problem), _num_sms(dev), _addr(ws, torch.uint8, "ws"), ws.numel(), _handle(stream, dev))


def _q4_append(dev, problem, prompt, k, v, cu_seqlens, start, pool, block_table, ws, stream) -> None:
    n = prompt.num_seqs
    _call(dev, "pkv_q4_prompt_append", _byref(problem), _byref(prompt), k.data_ptr(), v.data_ptr(),
          _seqs(cu_seqlens, n), _start(start, n), _addr(pool, torch.uint8, "pool"), _table(block_table, problem),
          _num_sms(dev), _addr(ws, torch.uint8, "ws"), ws.numel(), _handle(stream, dev))


def _q4_read(dev, problem, prompt, cu_seqlens, start, pool, block_table, k_out, v_out, ws, stream) -> None:
    n = prompt.num_seqs
    _call(dev, "pkv_q4_read", _byref(problem), _byref(prompt), _seqs(cu_seqlens, n), _start(start, n),
          _addr(pool, torch.uint8, "pool"), _table(block_table, problem), k_out.data_ptr(), v_out.data_ptr(),
          _num_sms(dev), _addr(ws, torch.uint8, "ws"), ws.numel(), _handle(stream, dev))


def pkv_prompt_append(problem: Problem, prompt: Prompt, k, v, cu_seqlens, start, k_pool, v_pool, block_table, ws,
                      stream=None) -> None:
    _fits(k, "k", prompt, prompt.num_kv_heads, prompt.k_stride)
    _fits(v, "v", prompt, prompt.num_kv_heads, prompt.v_stride)
    _pool(k_pool, "k_pool", problem, prompt)
    _pool(v_pool, "v_pool", problem, prompt)
    _append(_device(k, v, cu_seqlens, start, k_pool, v_pool, block_table, ws), problem, prompt, k, v, cu_seqlens, start,
            k_pool, v_pool, block_table, ws, stream)


def pkv_q4_prompt_append(problem: Problem, prompt: Prompt, k, v, cu_seqlens, start, pool, block_table, ws,
                         stream=None) -> None:
    _fits(k, "k", prompt, prompt.num_kv_heads, prompt.k_stride)
    _fits(v, "v", prompt, prompt.num_kv_heads, prompt.v_stride)
    _pool(pool, "pool", problem, prompt)
    _q4_append(_device(k, v, cu_seqlens, start, pool, block_table, ws), problem, prompt, k, v, cu_seqlens, start, pool,
               block_table, ws, stream)


def pkv_q4_read(problem: Problem, prompt: Prompt, cu_seqlens, start, pool, block_table, k_out, v_out, ws,
                stream=None) -> None:
    _fits(k_out, "k_out", prompt, prompt.num_kv_heads, prompt.k_stride)
    _fits(v_out, "v_out", prompt, prompt.num_kv_heads, prompt.v_stride)
    _pool(pool, "pool", problem, prompt)
    _q4_read(_device(pool, k_out, v_out, cu_seqlens, start, block_table, ws), problem, prompt, cu_seqlens, start, pool,
             block_table, k_out, v_out, ws, stream)


def pkv_q4_pool_bytes(problem: Problem) -> int:
    n = ctypes.c_size_t(0)
    check(load().pkv_q4_pool_bytes(_byref(problem), _byref(n)), "pkv_q4_pool_bytes")
    return int(n.value)


def pkv_q4_workspace_bytes(problem: Problem, num_sms: int | None = None) -> int:
    """Bytes of the workspace of a 4-bit decode step (num_sms None: that of the current device)."""
    if num_sms is None:
        num_sms = _num_sms(torch.cuda.current_device())
    n = ctypes.c_size_t(0)
    check(load().pkv_q4_workspace_bytes(_byref(problem), int(num_sms), _byref(n)), "pkv_q4_workspace_bytes")
    return int(n.value)


def _step_tensors(problem: Problem, q, pool, block_table, seq_lens, out, k_new=None, v_new=None) -> None:
    b, hq, hkv, d = problem.batch, problem.num_q_heads, problem.num_kv_heads, problem.head_dim
    for t, name, want in ((q, "q", (b, hq, d)), (out, "out", (b, hq, d)), (k_new, "k_new", (b, hkv, d)),
                          (v_new, "v_new", (b, hkv, d)), (pool, "pool", (problem.num_pages, hkv, PKV_Q4_BLOCK_BYTES))):
        if t is not None and t.shape != want:
            raise ValueError(f"{name} must have shape {want}, got {tuple(t.shape)}")
    if seq_lens.numel() != b:
        raise ValueError(f"seq_lens must have {b} entries")


def _step(problem, q, k_new, v_new, pool, block_table, seq_lens, scale, ws, out, stream) -> None:
    dev = _device(q, k_new, v_new, pool, block_table, seq_lens, ws, out)
    _step_tensors(problem, q, pool, block_table, seq_lens, out, k_new, v_new)
    f16 = torch.float16
    head = (_byref(problem), _addr(q, f16, "q"))
    tail = (_addr(pool, torch.uint8, "pool"), _table(block_table, problem), _addr(seq_lens, torch.int32, "seq_lens"),
            scale, _num_sms(dev), _addr(ws, torch.uint8, "ws"), ws.numel(), _addr(out, f16, "out"),
            _handle(stream, dev))
    if k_new is None and v_new is None:
        _call(dev, "pkv_q4_decode_step", *head, *tail)
    else:
        _call(dev, "pkv_q4_decode_step_append", *head, _addr(k_new, f16, "k_new"), _addr(v_new, f16, "v_new"), *tail)


def pkv_q4_decode_step(problem: Problem, q, pool, block_table, seq_lens, scale, ws, out, stream=None) -> None:
    _step(problem, q, None, None, pool, block_table, seq_lens, scale, ws, out, stream)


def pkv_q4_decode_step_append(problem: Problem, q, k_new, v_new, pool, block_table, seq_lens, scale, ws, out,
                              stream=None) -> None:
    if k_new is None or v_new is None:
        raise ValueError("k_new and v_new are required")
    _step(problem, q, k_new, v_new, pool, block_table, seq_lens, scale, ws, out, stream)


# ------------------------------------------------------------------------------- the same, described by the tensors
def _other(stream, device: int) -> torch.cuda.Stream | None:
    """`stream` as a torch stream where it is not the device's current one."""
    if stream is None:
        return None
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    return None if stream == torch.cuda.current_stream(device) else stream


def _scratch(nbytes: int, ws, device: int, stream):
    """The caller's workspace, or one for this call alone."""
    if ws is not None:
        return ws
    other = _other(stream, device)
    with torch.cuda.device(device):
        if other is None:
            return alloc_workspace(nbytes, device)
        with torch.cuda.stream(other):
            return alloc_workspace(nbytes, device)


def _new(shape, device: int, stream) -> torch.Tensor:
    out = torch.empty(shape, dtype=torch.float16, device=device)
    other = _other(stream, device)
    if other is not None:
        other.wait_stream(torch.cuda.current_stream(device))  # the memory may still be read on the current stream
        out.record_stream(other)
    return out


def prompt_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor,
                     scale: float | None = None, out: torch.Tensor | None = None, ws: torch.Tensor | None = None,
                     stream=None) -> torch.Tensor:
    """Causal grouped-query attention over packed prompts (include/pkv.h, pkv_prompt_attention). Returns out.

    q [tokens, Hq, d], k, v [tokens, Hkv, d] fp16, the heads of a token contiguous and the tokens at any distance (q, k
    and v may be slices of one projection); cu_seqlens [num_seqs + 1] int32 on the device. Rows of an `out` given by
    the caller that belong to no sequence keep their values; in one made here they are undefined.
    """
    qs = _rows(q, "q")
    t, hq, d = q.shape
    ks = _rows(k, "k", None, t, d)
    hkv = k.shape[1]
    vs = _rows(v, "v", hkv, t, d)
    dev = _device(q, k, v, cu_seqlens, ws, out)
    if out is None:
        out = _new((t, hq, d), dev, stream)
        os = hq * d
    else:
        os = _rows(out, "out", hq, t, d)
    prompt = Prompt(cu_seqlens.numel() - 1, t, hq, hkv, d, 0, qs, ks, vs, os)
    _attention(dev, prompt, q, k, v, cu_seqlens, 1.0 / math.sqrt(d) if scale is None else scale,
               _scratch(PKV_PROMPT_WS_BYTES, ws, dev, stream), out, stream)
    return out


def prompt_append(k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor, k_pool: torch.Tensor,
                  v_pool: torch.Tensor, block_table: torch.Tensor, start: torch.Tensor | None = None,
                  ws: torch.Tensor | None = None, stream=None) -> None:
    """Packed prompts' K/V into the FP16 pages (include/pkv.h, pkv_prompt_append).

    k, v [tokens, Hkv, d] as for prompt_attention; k_pool, v_pool [num_pages, page_size, Hkv, d]; block_table
    [num_seqs, max_pages] int32; start [num_seqs] int32: tokens that each row holds already (None: none).
    """
    ks = _rows(k, "k")
    t, hkv, d = k.shape
    vs = _rows(v, "v", hkv, t, d)
    if k_pool.dim() != 4 or k_pool.shape[2:] != (hkv, d) or v_pool.shape != k_pool.shape:
        raise ValueError(f"k_pool and v_pool must be [num_pages, page_size, {hkv}, {d}]")
    b, pages = block_table.shape
    problem = Problem(b, hkv, hkv, d, k_pool.shape[1], k_pool.shape[0], pages)
    prompt = Prompt(cu_seqlens.numel() - 1, t, hkv, hkv, d, 0, hkv * d, ks, vs, hkv * d)
    dev = _device(k, v, cu_seqlens, start, k_pool, v_pool, block_table, ws)
    _append(dev, problem, prompt, k, v, cu_seqlens, start, k_pool, v_pool, block_table,
            _scratch(PKV_PROMPT_WS_BYTES, ws, dev, stream), stream)


def _check_pool(pool: torch.Tensor) -> int:
    if pool.dim() != 3 or pool.dtype != torch.uint8 or pool.shape[2] != PKV_Q4_BLOCK_BYTES:
        raise ValueError(f"pool must be a uint8 tensor [num_pages, Hkv, {PKV_Q4_BLOCK_BYTES}]")
    return pool.shape[1]


def q4_problem(q: torch.Tensor, pool: torch.Tensor, block_table: torch.Tensor) -> Problem:
    """The problem of a decode step over 4-bit pages: q [B, Hq, d], pool [num_pages, Hkv, block], block_table."""
    hkv = _check_pool(pool)
    b, hq, d = q.shape
    return Problem(b, hq, hkv, d, 16, pool.shape[0], block_table.shape[1])


def q4_prompt_append(k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor, pool: torch.Tensor,
                     block_table: torch.Tensor, start: torch.Tensor | None = None, ws: torch.Tensor | None = None,
                     stream=None) -> None:
    """Packed prompts' K/V quantised into 4-bit pages (include/pkv.h, pkv_q4_prompt_append); arguments as for
    prompt_append, pool [num_pages, Hkv, PKV_Q4_BLOCK_BYTES] uint8."""
    ks = _rows(k, "k")
    t, hkv, d = k.shape
    vs = _rows(v, "v", hkv, t, d)
    if _check_pool(pool) != hkv:
        raise ValueError(f"pool has {pool.shape[1]} KV heads, k has {hkv}")
    b, pages = block_table.shape
    problem = Problem(b, hkv, hkv, d, 16, pool.shape[0], pages)
    prompt = Prompt(cu_seqlens.numel() - 1, t, hkv, hkv, d, 0, hkv * d, ks, vs, hkv * d)
    dev = _device(k, v, cu_seqlens, start, pool, block_table, ws)
    _q4_append(dev, problem, prompt, k, v, cu_seqlens, start, pool, block_table,
               _scratch(PKV_PROMPT_WS_BYTES, ws, dev, stream), stream)


def q4_read(cu_seqlens: torch.Tensor, pool: torch.Tensor, block_table: torch.Tensor,
            start: torch.Tensor | None = None, total_tokens: int | None = None, k_out: torch.Tensor | None = None,
            v_out: torch.Tensor | None = None, ws: torch.Tensor | None = None, stream=None):
    """Tokens of 4-bit pages as packed fp16 rows (include/pkv.h, pkv_q4_read). Returns k_out, v_out
    [total_tokens, Hkv, d]; give either both of them or total_tokens."""
    hkv, d = _check_pool(pool), 128
    b, pages = block_table.shape
    if (k_out is None) != (v_out is None):
        raise ValueError("give both of k_out and v_out, or neither")
    dev = _device(pool, k_out, v_out, cu_seqlens, start, block_table, ws)
    if k_out is None:
        if total_tokens is None:
            raise ValueError("give k_out and v_out, or total_tokens")
        k_out, v_out = (_new((int(total_tokens), hkv, d), dev, stream) for _ in range(2))
    t = k_out.shape[0]
    if total_tokens is not None and total_tokens != t:
        raise ValueError(f"k_out has {t} rows, total_tokens is {total_tokens}")
    prompt = Prompt(cu_seqlens.numel() - 1, t, hkv, hkv, d, 0, hkv * d, _rows(k_out, "k_out", hkv, t, d),
                    _rows(v_out, "v_out", hkv, t, d), hkv * d)
    _q4_read(dev, Problem(b, hkv, hkv, d, 16, pool.shape[0], pages), prompt, cu_seqlens, start, pool, block_table,
             k_out, v_out, _scratch(PKV_PROMPT_WS_BYTES, ws, dev, stream), stream)
    return k_out, v_out


def q4_decode(q: torch.Tensor, pool: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor,
              k_new: torch.Tensor | None = None, v_new: torch.Tensor | None = None, scale: float | None = None,
              out: torch.Tensor | None = None, ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """One decode step over 4-bit pages (include/pkv.h, pkv_q4_decode_step; with k_new and v_new [B, Hkv, d],
    pkv_q4_decode_step_append). Returns out [B, Hq, d] fp16.

    q [B, Hq, d] fp16; pool [num_pages, Hkv, PKV_Q4_BLOCK_BYTES] uint8; block_table [B, max_pages] int32; seq_lens [B]
    int32 on the device. Keep ws (pkv_q4_workspace_bytes, alloc_workspace) over the steps of a loop.
    """
    problem = q4_problem(q, pool, block_table)
    if (k_new is None) != (v_new is None):
        raise ValueError("give both of k_new and v_new, or neither")
    dev = _device(q)
    if out is None:
        out = _new(tuple(q.shape), dev, stream)
    if ws is None:
        ws = _scratch(pkv_q4_workspace_bytes(problem, _num_sms(dev)), None, dev, stream)
    scale = 1.0 / math.sqrt(q.shape[2]) if scale is None else scale
    _step(problem, q, k_new, v_new, pool, block_table, seq_lens, scale, ws, out, stream)
    return out
