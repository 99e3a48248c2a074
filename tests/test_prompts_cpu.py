"""The prompt and 4-bit-cache calls on the CPU: argument checks (nothing reaches the device), sizes, the page format."""

import ctypes
import math

import pytest
import torch

import prompt_reference as ref
import serving_paged_gqa_gb300 as pkv

vp = ctypes.c_void_p
A = vp(1 << 20)  # an aligned stand-in, never dereferenced: validation fails first
ODD = vp((1 << 20) + 8)
F = ctypes.c_float
OK, INVAL, UNSUPPORTED, NULLPTR, SMALL, ALIGN = 0, -1, -2, -3, -4, -5


@pytest.fixture(scope="module", autouse=True)
def built():
    from serving_paged_gqa_gb300 import build

    build.build()


def prompt(**kw):
    p = pkv.make_prompt(2, 50, 32, 8, 128)
    for k, x in kw.items():
        setattr(p, k, x)
    return p


def problem(**kw):
    p = pkv.make_problem(2, 32, 8, 128, 16, 100, 10)
    for k, x in kw.items():
        setattr(p, k, x)
    return p


@pytest.mark.parametrize("change,code", [
    ({}, OK), (dict(num_seqs=0), OK), (dict(total_tokens=0), OK), (dict(num_seqs=-1), INVAL), (dict(total_tokens=-1), INVAL),
    (dict(num_q_heads=0), INVAL), (dict(num_kv_heads=0), INVAL), (dict(reserved=1), INVAL), (dict(head_dim=64), UNSUPPORTED),
    (dict(num_q_heads=33), UNSUPPORTED), (dict(num_q_heads=24), UNSUPPORTED), (dict(num_q_heads=256), UNSUPPORTED),
    (dict(num_seqs=4097), UNSUPPORTED), (dict(q_stride=4095), INVAL), (dict(q_stride=4100), INVAL), (dict(q_stride=4104), OK),
    (dict(k_stride=0), INVAL), (dict(v_stride=1016), INVAL), (dict(v_stride=-1024), INVAL), (dict(out_stride=1 << 62), INVAL),
    (dict(k_stride=6144), OK),
])
def test_check_prompt(change, code):
    assert pkv.pkv_check_prompt(prompt(**change)) == code


def attention(p=None, q=A, k=A, v=A, cu=A, scale=0.1, sms=152, ws=A, n=256, out=A):
    p = prompt() if p is None else p
    return pkv.load().pkv_prompt_attention(ctypes.byref(p), q, k, v, cu, F(scale), sms, ws, n, out, None)


@pytest.mark.parametrize("change,code", [
    (dict(q=None), NULLPTR), (dict(k=None), NULLPTR), (dict(v=None), NULLPTR), (dict(cu=None), NULLPTR), (dict(out=None), NULLPTR),
    (dict(ws=None), NULLPTR), (dict(q=ODD), ALIGN), (dict(k=ODD), ALIGN), (dict(v=ODD), ALIGN), (dict(out=ODD), ALIGN),
    (dict(cu=vp((1 << 20) + 2)), ALIGN), (dict(ws=ODD), ALIGN), (dict(n=255), SMALL), (dict(scale=math.nan), INVAL),
    (dict(scale=math.inf), INVAL), (dict(scale=-0.1), INVAL), (dict(scale=2e12), INVAL), (dict(sms=0), INVAL), (dict(sms=4097), INVAL), (dict(p=prompt(head_dim=64)), UNSUPPORTED),
    (dict(p=prompt(num_seqs=0), q=None), OK), (dict(p=prompt(total_tokens=0), q=None), OK),
])
def test_prompt_attention_refuses_before_any_work(change, code):
    assert attention(**change) == code


def test_an_output_at_the_address_of_an_input_is_refused():
    b = vp(1 << 21)
    for call in (dict(out=A, k=b, v=b), dict(q=b, out=A, v=b), dict(q=b, k=b, out=A)):
        assert attention(**call) == INVAL
    assert decode(False) == INVAL and decode(True) == INVAL


def pages(call, pr=None, p=None, k=A, v=A, cu=A, start=None, pool=A, pool2=A, bt=A, sms=152, ws=A, n=256):
    pr, p = problem() if pr is None else pr, prompt() if p is None else p
    lib, a, b = pkv.load(), ctypes.byref(pr), ctypes.byref(p)
    if call == "append":
        return lib.pkv_prompt_append(a, b, k, v, cu, start, pool, pool2, bt, sms, ws, n, None)
    if call == "q4":
        return lib.pkv_q4_prompt_append(a, b, k, v, cu, start, pool, bt, sms, ws, n, None)
    return lib.pkv_q4_read(a, b, cu, start, pool, bt, k, v, sms, ws, n, None)


@pytest.mark.parametrize("call", ["append", "q4", "read"])
@pytest.mark.parametrize("change,code", [
    (dict(k=None), NULLPTR), (dict(v=None), NULLPTR), (dict(cu=None), NULLPTR), (dict(pool=None), NULLPTR), (dict(bt=None), NULLPTR),
    (dict(ws=None), NULLPTR), (dict(k=ODD), ALIGN), (dict(v=ODD), ALIGN), (dict(pool=ODD), ALIGN), (dict(ws=ODD), ALIGN),
    (dict(start=vp((1 << 20) + 1)), ALIGN), (dict(bt=vp((1 << 20) + 1)), ALIGN), (dict(n=0), SMALL), (dict(sms=-1), INVAL), (dict(sms=1 << 30), INVAL),
    (dict(pr=problem(batch=3)), INVAL), (dict(p=prompt(num_kv_heads=4, num_q_heads=16)), INVAL), (dict(pr=problem(page_size=32)), UNSUPPORTED),
    (dict(p=prompt(k_stride=1000)), INVAL), (dict(p=prompt(total_tokens=0), k=None), OK),
    (dict(p=prompt(num_seqs=0), pr=problem(batch=0), k=None), OK),
])
def test_page_calls_refuse_before_any_work(call, change, code):
    assert pages(call, **change) == code


def decode(append, pr=None, q=A, kn=A, vn=A, pool=A, bt=A, lens=A, scale=0.1, sms=152, ws=A, n=1 << 30, out=A):
    pr = problem() if pr is None else pr
    lib = pkv.load()
    if append:
        return lib.pkv_q4_decode_step_append(ctypes.byref(pr), q, kn, vn, pool, bt, lens, F(scale), sms, ws, n, out, None)
    return lib.pkv_q4_decode_step(ctypes.byref(pr), q, pool, bt, lens, F(scale), sms, ws, n, out, None)


@pytest.mark.parametrize("append", [False, True])
@pytest.mark.parametrize("change,code", [
    (dict(q=None), NULLPTR), (dict(pool=None), NULLPTR), (dict(bt=None), NULLPTR), (dict(lens=None), NULLPTR), (dict(out=None), NULLPTR),
    (dict(ws=None), NULLPTR), (dict(q=ODD), ALIGN), (dict(pool=ODD), ALIGN), (dict(out=ODD), ALIGN), (dict(ws=ODD), ALIGN),
    (dict(bt=vp(3)), ALIGN), (dict(lens=vp(3)), ALIGN), (dict(n=16), SMALL), (dict(scale=math.nan), INVAL), (dict(scale=-math.inf), INVAL),
    (dict(scale=-2e12), INVAL), (dict(sms=0), INVAL), (dict(sms=4097), INVAL), (dict(pr=problem(head_dim=64)), UNSUPPORTED), (dict(pr=problem(num_q_heads=48)), UNSUPPORTED),
    (dict(pr=problem(batch=0), q=None), OK),
])
def test_q4_decode_refuses_before_any_work(append, change, code):
    assert decode(append, **change) == code


def test_q4_append_wants_both_new_rows():
    assert decode(True, kn=None) == NULLPTR and decode(True, vn=None) == NULLPTR
    assert decode(True, kn=ODD) == ALIGN and decode(True, vn=ODD) == ALIGN


def test_null_descriptions():
    lib, n = pkv.load(), ctypes.c_size_t()
    assert lib.pkv_check_prompt(None) == NULLPTR
    assert lib.pkv_prompt_attention(None, A, A, A, A, F(1), 152, A, 256, A, None) == NULLPTR
    assert lib.pkv_prompt_append(None, None, A, A, A, None, A, A, A, 152, A, 256, None) == NULLPTR
    assert lib.pkv_q4_pool_bytes(None, ctypes.byref(n)) == NULLPTR
    assert lib.pkv_q4_workspace_bytes(ctypes.byref(problem()), 152, None) == NULLPTR


def test_sizes():
    assert pkv.PKV_Q4_BLOCK_BYTES == ref.BLOCK == 2 * (16 * 128 // 2 + 16 * 2 * 4)
    assert pkv.pkv_q4_pool_bytes(pkv.make_problem(1, 32, 8, 128, 16, 1 << 20, 4)) == (1 << 20) * 8 * 2304
    small, large = (pkv.pkv_q4_workspace_bytes(pkv.make_problem(b, 32, 8, 128, 16, 100, 4096), 152) for b in (1, 4096))
    assert small == large and 256 <= small < 64 << 20 and small % 256 == 0
    with pytest.raises(pkv.PkvError):
        pkv.pkv_q4_workspace_bytes(pkv.make_problem(1, 32, 8, 128, 16, 100, 4), 0)


def test_page_format_has_a_place_for_every_value():
    for m in ref._byte_maps("cpu"):
        assert sorted(m.flatten().tolist()) == list(range(1024))
    g = torch.Generator().manual_seed(0)
    k, v = torch.randn((21, 2, 128), generator=g).half(), torch.randn((21, 2, 128), generator=g).half()
    pool = torch.zeros((4, 2, ref.BLOCK), dtype=torch.uint8)
    bt, pos = torch.tensor([2, 0, 3]), torch.arange(21) + 9
    ref.put_tokens(pool, bt, pos, k, v)
    for x, got in zip((k, v), ref.get_tokens(pool, bt, pos)):
        for a, b in zip(ref.quantise(x), got):
            assert torch.equal(a, b)
        w = ref.values(*got)
        step = got[1].double().repeat_interleave(64, -1)
        # half a step, and the scale's own rounding over 15 steps
        assert ((w - x.double()).abs() <= step * (0.5 + 15 * 2.0 ** -11)).all()


def test_python_checks():
    q, k = torch.zeros((5, 8, 128), dtype=torch.float16), torch.zeros((5, 2, 128), dtype=torch.float16)
    cu = torch.tensor([0, 5], dtype=torch.int32)
    for bad in (dict(q=q.float()), dict(q=q[0]), dict(k=k[:4]), dict(v=k[:, :1]), dict(k=k.transpose(0, 2).contiguous().transpose(0, 2)), {}):
        with pytest.raises(ValueError):  # the last one: tensors that are not on a GPU
            pkv.prompt_attention(**{**dict(q=q, k=k, v=k, cu_seqlens=cu), **bad})
    pool = torch.zeros((3, 2, 2304), dtype=torch.uint8)
    bt = torch.zeros((1, 2), dtype=torch.int32)
    for bad in (pool[..., :2303], pool.view(torch.int8), pool[0]):
        with pytest.raises(ValueError):
            pkv.q4_prompt_append(k, k, cu, bad, bt)
        with pytest.raises(ValueError):
            pkv.q4_decode(q[:1], bad, bt, cu[:1])
    with pytest.raises(ValueError):
        pkv.q4_prompt_append(k, k, cu, pool[:, :1], bt)
    with pytest.raises(ValueError):
        pkv.q4_decode(q[:1], pool, bt, cu)
    with pytest.raises(ValueError):
        pkv.q4_decode(q[:1], pool, bt, cu[:1], k_new=k[:1])
    with pytest.raises(ValueError):
        pkv.prompt_append(k, k, cu, pool, pool, bt)
    with pytest.raises(ValueError):
        pkv.q4_read(cu, pool, bt)
