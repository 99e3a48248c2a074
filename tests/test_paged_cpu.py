"""The calls over chunks, tables and selected pages on the CPU: argument checks (nothing reaches the device), sizes."""

import ctypes
import math

import pytest
import torch

import serving_paged_gqa_gb300 as pkv

vp = ctypes.c_void_p
F, I64 = ctypes.c_float, ctypes.c_int64
OK, INVAL, UNSUPPORTED, NULLPTR, SMALL, ALIGN = 0, -1, -2, -3, -4, -5


@pytest.fixture(scope="module", autouse=True)
def built():
    from serving_paged_gqa_gb300 import build

    build.build()


def at(i):
    """Aligned stand-ins at different places, never dereferenced: validation fails first."""
    return vp((1 << 24) + (i << 20))


ODD, ODD2 = vp((1 << 24) + 8), vp((1 << 24) + 2)


def problem(**kw):
    p = pkv.make_problem(2, 32, 8, 128, 16, 100, 10)
    for k, x in kw.items():
        setattr(p, k, x)
    return p


def prompt(**kw):
    p = pkv.make_prompt(2, 50, 32, 8, 128)
    for k, x in kw.items():
        setattr(p, k, x)
    return p


def chunk(pr=None, pm=None, q=at(1), k=at(2), v=at(3), cu=at(4), start=None, bt=at(5), scale=0.1, sms=152, ws=at(6), n=1 << 30, out=at(7)):
    pr, pm = problem() if pr is None else pr, prompt() if pm is None else pm
    return pkv.load().pkv_chunk_attention(ctypes.byref(pr), ctypes.byref(pm), q, k, v, cu, start, bt, F(scale), sms, ws, n, out, None)


@pytest.mark.parametrize("change,code", [
    (dict(q=None), NULLPTR), (dict(k=None), NULLPTR), (dict(v=None), NULLPTR), (dict(cu=None), NULLPTR), (dict(bt=None), NULLPTR),
    (dict(out=None), NULLPTR), (dict(ws=None), NULLPTR), (dict(q=ODD), ALIGN), (dict(k=ODD), ALIGN), (dict(v=ODD), ALIGN),
    (dict(out=ODD), ALIGN), (dict(ws=ODD), ALIGN), (dict(cu=ODD2), ALIGN), (dict(start=ODD2), ALIGN), (dict(bt=ODD2), ALIGN),
    (dict(n=1 << 20), SMALL), (dict(scale=math.nan), INVAL), (dict(scale=-1.0), INVAL), (dict(scale=2e12), INVAL), (dict(scale=math.inf), INVAL),
    (dict(sms=0), INVAL), (dict(sms=4097), INVAL), (dict(pr=problem(batch=3)), INVAL), (dict(pr=problem(num_q_heads=16)), INVAL),
    (dict(pr=problem(num_kv_heads=16)), INVAL), (dict(pr=problem(page_size=32)), UNSUPPORTED), (dict(pr=problem(num_pages=1 << 28)), UNSUPPORTED),
    (dict(pr=problem(num_pages=0)), INVAL), (dict(pm=prompt(head_dim=64)), UNSUPPORTED), (dict(pm=prompt(q_stride=100)), INVAL),
    (dict(out=at(1)), INVAL), (dict(out=at(2)), INVAL), (dict(out=at(3)), INVAL),
    (dict(pm=prompt(total_tokens=0), q=None), OK), (dict(pm=prompt(num_seqs=0), pr=problem(batch=0), q=None), OK),
])
def test_chunk_attention_refuses_before_any_work(change, code):
    assert chunk(**change) == code


def grow(pr=None, new=at(1), lens=at(2), bt=at(3), free=at(4), count=at(5), cu=at(6), start=at(7), slots=at(8), pos=at(9), cap=64,
         lens_out=at(2), count_out=at(5), sms=152, ws=at(10), n=256):
    pr = problem() if pr is None else pr
    return pkv.load().pkv_tables_grow(ctypes.byref(pr), new, lens, bt, free, count, cu, start, slots, pos, I64(cap), lens_out, count_out,
                                      sms, ws, n, None)


@pytest.mark.parametrize("change,code", [
    (dict(new=None), NULLPTR), (dict(lens=None), NULLPTR), (dict(bt=None), NULLPTR), (dict(free=None), NULLPTR), (dict(count=None), NULLPTR),
    (dict(lens_out=None), NULLPTR), (dict(count_out=None), NULLPTR), (dict(ws=None), NULLPTR), (dict(new=ODD2), ALIGN), (dict(lens=ODD2), ALIGN),
    (dict(bt=ODD2), ALIGN), (dict(free=ODD2), ALIGN), (dict(count=ODD2), ALIGN), (dict(cu=ODD2), ALIGN), (dict(start=ODD2), ALIGN),
    (dict(slots=vp((1 << 24) + 4)), ALIGN), (dict(pos=ODD2), ALIGN), (dict(ws=ODD), ALIGN), (dict(n=255), SMALL), (dict(cap=-1), INVAL),
    (dict(cap=1 << 31), INVAL), (dict(sms=0), INVAL), (dict(pr=problem(head_dim=64)), UNSUPPORTED), (dict(pr=problem(batch=5000)), UNSUPPORTED),
    (dict(start=at(2)), INVAL), (dict(cu=at(1)), INVAL), (dict(start=at(6)), INVAL), (dict(lens_out=at(1)), INVAL), (dict(count_out=at(2)), INVAL),
    (dict(bt=at(4)), INVAL), (dict(pos=at(8)), INVAL), (dict(lens_out=at(5)), INVAL),
])
def test_grow_refuses_before_any_work(change, code):
    assert grow(**change) == code


def release(pr=None, ended=at(1), lens=at(2), bt=at(3), free=at(4), count=at(5), lens_out=at(2), count_out=at(5), sms=152, ws=at(10), n=256):
    pr = problem() if pr is None else pr
    return pkv.load().pkv_tables_release(ctypes.byref(pr), ended, lens, bt, free, count, lens_out, count_out, sms, ws, n, None)


@pytest.mark.parametrize("change,code", [
    (dict(ended=None), NULLPTR), (dict(lens=None), NULLPTR), (dict(bt=None), NULLPTR), (dict(free=None), NULLPTR), (dict(count=None), NULLPTR),
    (dict(lens_out=None), NULLPTR), (dict(count_out=None), NULLPTR), (dict(ws=None), NULLPTR), (dict(ended=ODD2), ALIGN), (dict(free=ODD2), ALIGN),
    (dict(ws=ODD), ALIGN), (dict(n=0), SMALL), (dict(sms=5000), INVAL), (dict(free=at(3)), INVAL), (dict(lens_out=at(1)), INVAL),
    (dict(count_out=at(4)), INVAL), (dict(lens_out=at(4)), INVAL), (dict(pr=problem(page_size=8)), UNSUPPORTED),
])
def test_release_refuses_before_any_work(change, code):
    assert release(**change) == code


def bounds(pr=None, pm=None, cu=at(1), start=None, k=at(2), bt=at(3), bd=at(4), sms=152, ws=at(5), n=256):
    pr, pm = problem() if pr is None else pr, prompt() if pm is None else pm
    return pkv.load().pkv_page_bounds(ctypes.byref(pr), ctypes.byref(pm), cu, start, k, bt, bd, sms, ws, n, None)


@pytest.mark.parametrize("change,code", [
    (dict(cu=None), NULLPTR), (dict(k=None), NULLPTR), (dict(bt=None), NULLPTR), (dict(bd=None), NULLPTR), (dict(ws=None), NULLPTR),
    (dict(k=ODD), ALIGN), (dict(bd=ODD), ALIGN), (dict(cu=ODD2), ALIGN), (dict(start=ODD2), ALIGN), (dict(bt=ODD2), ALIGN), (dict(ws=ODD), ALIGN),
    (dict(n=10), SMALL), (dict(sms=0), INVAL), (dict(pr=problem(batch=1)), INVAL), (dict(pr=problem(num_kv_heads=4, num_q_heads=32)), INVAL),
    (dict(bd=at(2)), INVAL), (dict(pm=prompt(total_tokens=0), k=None), OK),
    (dict(pr=problem(num_q_heads=128, num_kv_heads=128, max_pages_per_seq=(1 << 27) - 1), pm=pkv.make_prompt(2, 50, 128, 128, 128)), UNSUPPORTED),
])
def test_page_bounds_refuse_before_any_work(change, code):
    assert bounds(**change) == code


def select(pr=None, q=at(1), bd=at(2), bt=at(3), lens=at(4), k=4, sms=152, ws=at(5), n=1 << 30, pages=at(6)):
    pr = problem() if pr is None else pr
    return pkv.load().pkv_select_pages(ctypes.byref(pr), q, bd, bt, lens, k, sms, ws, n, pages, None)


@pytest.mark.parametrize("change,code", [
    (dict(q=None), NULLPTR), (dict(bd=None), NULLPTR), (dict(bt=None), NULLPTR), (dict(lens=None), NULLPTR), (dict(pages=None), NULLPTR),
    (dict(ws=None), NULLPTR), (dict(q=ODD), ALIGN), (dict(bd=ODD), ALIGN), (dict(bt=ODD2), ALIGN), (dict(lens=ODD2), ALIGN), (dict(pages=ODD2), ALIGN),
    (dict(ws=ODD), ALIGN), (dict(n=1000), SMALL), (dict(k=0), INVAL), (dict(k=-3), INVAL), (dict(sms=0), INVAL), (dict(pages=at(1)), INVAL),
    (dict(pages=at(4)), INVAL), (dict(pr=problem(num_q_heads=24)), UNSUPPORTED), (dict(pr=problem(batch=0), q=None), OK),
])
def test_select_pages_refuses_before_any_work(change, code):
    assert select(**change) == code


def sparse(pr=None, q=at(1), k=at(2), v=at(3), bt=at(4), lens=at(5), pages=at(6), sel=4, scale=0.1, sms=152, ws=at(7), n=1 << 30, out=at(8)):
    pr = problem() if pr is None else pr
    return pkv.load().pkv_sparse_decode_step(ctypes.byref(pr), q, k, v, bt, lens, pages, sel, F(scale), sms, ws, n, out, None)


@pytest.mark.parametrize("change,code", [
    (dict(q=None), NULLPTR), (dict(k=None), NULLPTR), (dict(v=None), NULLPTR), (dict(bt=None), NULLPTR), (dict(lens=None), NULLPTR),
    (dict(pages=None), NULLPTR), (dict(out=None), NULLPTR), (dict(ws=None), NULLPTR), (dict(q=ODD), ALIGN), (dict(k=ODD), ALIGN), (dict(v=ODD), ALIGN),
    (dict(out=ODD), ALIGN), (dict(bt=ODD2), ALIGN), (dict(lens=ODD2), ALIGN), (dict(pages=ODD2), ALIGN), (dict(ws=ODD), ALIGN), (dict(n=1), SMALL),
    (dict(sel=0), INVAL), (dict(sel=1 << 28), INVAL), (dict(scale=math.nan), INVAL), (dict(scale=-0.5), INVAL), (dict(sms=0), INVAL), (dict(out=at(1)), INVAL),
    (dict(out=at(2)), INVAL), (dict(pr=problem(num_pages=0)), INVAL), (dict(pr=problem(num_pages=1 << 28)), UNSUPPORTED), (dict(pr=problem(batch=0), q=None), OK),
])
def test_sparse_step_refuses_before_any_work(change, code):
    assert sparse(**change) == code


def test_null_descriptions():
    lib, n = pkv.load(), ctypes.c_size_t()
    a = at(1)
    assert lib.pkv_chunk_attention(None, None, a, a, a, a, None, a, F(1), 152, a, 256, a, None) == NULLPTR
    assert lib.pkv_chunk_workspace_bytes(152, None) == NULLPTR
    assert lib.pkv_tables_grow(None, a, a, a, a, a, a, a, a, a, I64(1), a, a, 152, a, 256, None) == NULLPTR
    assert lib.pkv_tables_release(None, a, a, a, a, a, a, a, 152, a, 256, None) == NULLPTR
    assert lib.pkv_page_bounds(None, None, a, a, a, a, a, 152, a, 256, None) == NULLPTR
    assert lib.pkv_sparse_workspace_bytes(None, 152, ctypes.byref(n)) == NULLPTR
    assert lib.pkv_select_pages(None, a, a, a, a, 1, 152, a, 256, a, None) == NULLPTR
    assert lib.pkv_sparse_decode_step(None, a, a, a, a, a, a, 1, F(1), 152, a, 256, a, None) == NULLPTR


def test_sizes():
    chunk_ws = pkv.pkv_chunk_workspace_bytes(152)
    assert 256 < chunk_ws < 64 << 20 and chunk_ws % 256 == 0
    assert pkv.pkv_sparse_workspace_bytes(problem(), 152) == chunk_ws
    big = pkv.make_problem(64, 32, 8, 128, 16, 100, 8192)
    assert pkv.pkv_sparse_workspace_bytes(big, 152) >= 64 * 8 * 8192 * 12
    for sms in (0, -1, 4097):
        with pytest.raises(pkv.PkvError):
            pkv.pkv_chunk_workspace_bytes(sms)


def test_python_checks():
    f16, i32 = torch.float16, torch.int32
    q, pool = torch.zeros((5, 8, 128), dtype=f16), torch.zeros((3, 16, 2, 128), dtype=f16)
    cu, bt = torch.tensor([0, 5], dtype=i32), torch.zeros((1, 2), dtype=i32)
    good = dict(q=q, k_pool=pool, v_pool=pool, cu_seqlens=cu, block_table=bt)
    for bad in (dict(q=q.float()), dict(q=q[0]), dict(k_pool=pool[..., :64]), dict(v_pool=pool[:2]), dict(k_pool=pool[0]), {}):
        with pytest.raises(ValueError):  # the last one: tensors that are not on a GPU
            pkv.chunk_attention(**{**good, **bad})
    lens = torch.zeros(1, dtype=i32)
    for bad in (dict(new_tokens=lens), dict(free_count=torch.zeros(2, dtype=i32))):
        with pytest.raises(ValueError):
            pkv.tables_grow(**{**dict(new_tokens=lens, seq_lens=lens, block_table=bt, free_pages=lens, free_count=lens), **bad})
    with pytest.raises(ValueError):
        pkv.tables_release(lens, lens, bt, lens, lens)
    with pytest.raises(ValueError):
        pkv.page_bounds(pool[0], cu, bt, torch.zeros((3, 2, 2, 128), dtype=f16))
    with pytest.raises(ValueError):
        pkv.page_bounds(pool, cu, bt, torch.zeros((3, 2, 2, 128), dtype=f16))
    with pytest.raises(ValueError):
        pkv.select_pages(q[:1], torch.zeros((3, 2, 128), dtype=f16), bt, lens, 2)
    with pytest.raises(ValueError):
        pkv.select_pages(q[:1], torch.zeros((3, 2, 2, 128), dtype=f16), bt, lens, 2)
    with pytest.raises(ValueError):
        pkv.sparse_decode(q[:1], pool, pool[:1], bt, lens, torch.zeros((1, 2, 4), dtype=i32))
    with pytest.raises(ValueError):
        pkv.sparse_decode(q[:1], pool, pool, bt, lens, torch.zeros((1, 2, 4), dtype=i32))
