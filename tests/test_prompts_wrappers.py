"""The pkv_* wrappers that take a described problem and prompt: they refuse tensors that the descriptions do not fit, and do
what the calls that describe the tensors themselves do."""

import ctypes
import math

import pytest
import torch

import prompt_reference as ref
import serving_paged_gqa_gb300 as pkv

D, PS, HQ, HKV, PAGES, COLS = 128, 16, 8, 2, 9, 4
SCALE = 1.0 / math.sqrt(D)
LENS = [40, 17]
T = sum(LENS)


def tensors(dev):
    """Two sequences, the tensors of every wrapper, under their arguments' names."""
    g = torch.Generator().manual_seed(11)

    def normal(*shape):
        return torch.randn(shape, generator=g).half().to(dev)

    x = normal(T, HQ + 2 * HKV, D)
    bt = torch.full((2, COLS), -1, dtype=torch.int32)
    bt[0, :3], bt[1, :2] = torch.tensor([5, 0, 8], dtype=torch.int32), torch.tensor([7, 3], dtype=torch.int32)

    def zeros(*shape, dtype=torch.float16):
        return torch.zeros(shape, dtype=dtype, device=dev)

    return dict(q=x[:, :HQ], k=x[:, HQ:HQ + HKV], v=x[:, HQ + HKV:], out=zeros(T, HQ, D), k_out=zeros(T, HKV, D), v_out=zeros(T, HKV, D),
                cu_seqlens=torch.tensor([0, LENS[0], T], dtype=torch.int32, device=dev), start=None, block_table=bt.to(dev),
                k_pool=zeros(PAGES, PS, HKV, D), v_pool=zeros(PAGES, PS, HKV, D),
                pool=zeros(PAGES, HKV, ref.BLOCK, dtype=torch.uint8), ws=zeros(256, dtype=torch.uint8),
                qt=normal(2, HQ, D), k_new=normal(2, HKV, D), v_new=normal(2, HKV, D), out_t=zeros(2, HQ, D),
                seq_lens=torch.tensor(LENS, dtype=torch.int32, device=dev), ws_t=zeros(1 << 22, dtype=torch.uint8))


def problem():
    return pkv.make_problem(2, HQ, HKV, D, PS, PAGES, COLS)


def prompt(strides=3 * [(HQ + 2 * HKV) * D]):
    return pkv.make_prompt(2, T, HQ, HKV, D, *strides)


def call(name, t):
    p, pr = problem(), prompt()
    if name == "attention":
        pkv.pkv_prompt_attention(pr, t["q"], t["k"], t["v"], t["cu_seqlens"], SCALE, t["ws"], t["out"])
    elif name == "append":
        pkv.pkv_prompt_append(p, pr, t["k"], t["v"], t["cu_seqlens"], t["start"], t["k_pool"], t["v_pool"], t["block_table"], t["ws"])
    elif name == "q4_append":
        pkv.pkv_q4_prompt_append(p, pr, t["k"], t["v"], t["cu_seqlens"], t["start"], t["pool"], t["block_table"], t["ws"])
    elif name == "q4_read":
        pkv.pkv_q4_read(p, prompt(()), t["cu_seqlens"], t["start"], t["pool"], t["block_table"], t["k_out"], t["v_out"], t["ws"])
    elif name == "step":
        pkv.pkv_q4_decode_step(p, t["qt"], t["pool"], t["block_table"], t["seq_lens"], SCALE, t["ws_t"], t["out_t"])
    else:
        pkv.pkv_q4_decode_step_append(p, t["qt"], t["k_new"], t["v_new"], t["pool"], t["block_table"], t["seq_lens"], SCALE, t["ws_t"],
                                      t["out_t"])


PAGE_CALLS = [
    ("append", "k_pool", lambda x: x[:8]), ("append", "v_pool", lambda x: x[:8]), ("append", "k_pool", lambda x: x[:, :, :1]),
    ("append", "v_pool", lambda x: x[:, :8]), ("append", "k_pool", lambda x: x.flatten(1, 2)), ("append", "k", lambda x: x.contiguous()),
    ("q4_append", "pool", lambda x: x[:8]), ("q4_append", "pool", lambda x: x[:, :1]), ("q4_append", "pool", lambda x: x[..., :2303]),
    ("q4_append", "v", lambda x: x[..., :64]), ("q4_read", "pool", lambda x: x[:8]), ("q4_read", "pool", lambda x: x[:, :1]),
    ("q4_read", "pool", lambda x: x.flatten(0, 1)), ("q4_read", "v_out", lambda x: x[:, :1]),
]
OTHER_CALLS = [  # these look at the tensors' device first
    ("attention", "q", lambda x: x[:, :7]), ("attention", "k", lambda x: x.contiguous()), ("attention", "v", lambda x: x[:-1]),
    ("attention", "out", lambda x: x.float()), ("step", "pool", lambda x: x[:8]), ("step_append", "pool", lambda x: x[:, :1]),
    ("step_append", "k_new", lambda x: x[:, :1]),
]


@pytest.mark.parametrize("name,arg,bad", PAGE_CALLS)
def test_wrappers_refuse_tensors_that_the_descriptions_do_not_fit(name, arg, bad):
    t = tensors("cpu")
    t[arg] = bad(t[arg])
    with pytest.raises(ValueError, match=f"^{arg}\\b"):
        call(name, t)


def test_an_output_at_the_address_of_another_argument_is_refused():
    """(Stand-ins for addresses, never dereferenced: the call is refused before any device work.)"""
    lib, p, pr, f = pkv.load(), problem(), prompt(), ctypes.c_float(SCALE)
    a, b, c, d, e = (ctypes.c_void_p(i << 20) for i in range(1, 6))

    def step(out, q=a, k_new=b, v_new=c, pool=d):
        return lib.pkv_q4_decode_step_append(p, q, k_new, v_new, pool, a, a, f, 152, e, 1 << 30, out, None)

    for out in (a, b, c, d):
        assert step(out) == -1
    assert lib.pkv_q4_decode_step(p, a, b, a, a, f, 152, e, 1 << 30, b, None) == -1
    assert lib.pkv_prompt_append(p, pr, a, b, a, None, c, c, a, 152, e, 256, None) == -1
    for k_out, v_out in ((b, b), (a, b), (b, a)):
        assert lib.pkv_q4_read(p, pr, a, None, a, a, k_out, v_out, 152, e, 256, None) == -1


@pytest.mark.gpu
@pytest.mark.parametrize("name,arg,bad", PAGE_CALLS + OTHER_CALLS)
def test_wrappers_refuse_them_before_any_device_work(name, arg, bad):
    t = tensors("cuda")
    t[arg] = bad(t[arg])
    with pytest.raises(ValueError, match=f"^{arg}\\b"):
        call(name, t)


@pytest.mark.gpu
def test_wrappers_do_what_the_described_calls_do():
    import __graft_entry__

    __graft_entry__.build()
    a, b = tensors("cuda"), tensors("cuda")
    for name in ("attention", "append", "q4_append", "q4_read", "step", "step_append"):
        call(name, a)
        if name == "attention":
            pkv.prompt_attention(b["q"], b["k"], b["v"], b["cu_seqlens"], out=b["out"])
        elif name == "append":
            pkv.prompt_append(b["k"], b["v"], b["cu_seqlens"], b["k_pool"], b["v_pool"], b["block_table"])
        elif name == "q4_append":
            pkv.q4_prompt_append(b["k"], b["v"], b["cu_seqlens"], b["pool"], b["block_table"])
        elif name == "q4_read":
            pkv.q4_read(b["cu_seqlens"], b["pool"], b["block_table"], k_out=b["k_out"], v_out=b["v_out"])
        elif name == "step":
            pkv.q4_decode(b["qt"], b["pool"], b["block_table"], b["seq_lens"], out=b["out_t"])
        else:
            pkv.q4_decode(b["qt"], b["pool"], b["block_table"], b["seq_lens"], b["k_new"], b["v_new"], out=b["out_t"])
        torch.cuda.synchronize()
        for k in a:
            if a[k] is not None and not k.startswith("ws"):
                assert torch.equal(a[k], b[k]), (name, k)
    assert pkv.pkv_read_status(a["ws"]) == 0 and pkv.pkv_read_status(a["ws_t"]) == 0
    for k in ("out", "k_pool", "v_pool", "pool", "k_out", "v_out", "out_t"):
        assert (a[k] != 0).any(), k
