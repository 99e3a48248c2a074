"""pkv_chunk_attention on sequences of one tile of new tokens, many of them a CTA, one behind the other: what one tile's warps leave
for others has been read before the next tile's overwrite it."""

import ctypes
import math

import pytest
import torch

import prompt_reference as ref
import serving_paged_gqa_gb300 as pkv
from paged_reference import D, PS, Cache
from test_chunk_edges_gpu import check_not_finite, put

pytestmark = pytest.mark.gpu


def run_on(sms, c, q=None):
    """The call on a grid of `sms` CTAs."""
    lib, n = pkv.load(), ctypes.c_size_t()
    assert lib.pkv_chunk_workspace_bytes(sms, ctypes.byref(n)) == 0
    ws = pkv.alloc_workspace(n.value)
    t = c.q.shape[0]
    pr = pkv.make_problem(len(c.new), c.hq, c.hkv, D, PS, c.num_pages, c.bt.shape[1])
    pm = pkv.make_prompt(len(c.new), t, c.hq, c.hkv, D)
    q, out = (c.q if q is None else q).contiguous(), torch.full((t, c.hq, D), 7.0, dtype=torch.float16, device="cuda")
    rc = lib.pkv_chunk_attention(ctypes.byref(pr), ctypes.byref(pm), q.data_ptr(), c.k.data_ptr(), c.v.data_ptr(), c.cu.data_ptr(),
                                 c.st.data_ptr(), c.bt.data_ptr(), ctypes.c_float(c.scale), sms, ws.data_ptr(), ws.numel(),
                                 out.data_ptr(), torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert rc == 0 and pkv.pkv_read_status(ws) == 0
    assert (out[c.tokens:] == 7.0).all()
    return out[: c.tokens]


# At most 64 keys a sequence: rows of one half (64 and fewer) and of both, single keys, a tile that is full; longer ones among them.
SHORT = [([20], [10]), ([5], [30]), ([32], [32]), ([1], [0]), ([3, 20], [40, 3]), ([20, 5, 32], [70, 9, 1]), ([18, 20], [3000, 20])]


@pytest.mark.parametrize("sms", [1, 8, 152])
@pytest.mark.parametrize("new,start", SHORT)
def test_short_sequences_one_behind_the_other(sms, new, start):
    many = 12 if sms == 1 else 40
    c = Cache(new * many, start * many, 8, 2, seed=sum(new) + sms)
    want, bound = c.attend()
    ref.check(run_on(sms, c), want, bound)


@pytest.mark.parametrize("sms", [1, 8, 152])
@pytest.mark.parametrize("new,start", SHORT)
def test_short_sequences_with_values_that_are_not_finite(sms, new, start):
    """In dims of one half, of the other, or of both, from sequence to sequence; the last token's is seen by one token's rows and by no
    other, whose products with a weight of 0 are NaN all the same."""
    many = 12 if sms == 1 else 40
    c = Cache(new * many, start * many, 8, 2, seed=sum(new) + sms + 1)
    for s, (m, st) in enumerate(zip(c.new, c.start)):
        v = torch.randn((2, D), generator=torch.Generator(device="cuda").manual_seed(s), device="cuda").half()
        if s % 5 < 4:
            v[s % 2, (70, 5, 127, 64)[s % 5]] = (math.inf, -math.inf, math.nan, math.inf)[s % 4]
            if s % 5 == 3:
                v[0, 3] = math.nan
            put(c, s, st + m - 1 if s % 3 else max(0, st + m // 2 - 1), v=v)
    check_not_finite(c, run_on(sms, c))


@pytest.mark.parametrize("new,start", [([5], [40]), ([16], [300]), ([30], [20]), ([9], [5000])])
def test_rows_that_other_lanes_have_stored(new, start):
    """Values that are not finite in the dims that tile B's warps store, and finish by tile A's: the finite ones beside them stay, call
    after call."""
    c = Cache(new * 30, start * 30, 8, 2, seed=sum(new) + 2)
    for s, (m, st) in enumerate(zip(c.new, c.start)):
        v = torch.randn((2, D), generator=torch.Generator(device="cuda").manual_seed(s + 50), device="cuda").half()
        v[:, (32, 45, 63, 96, 127)[s % 5]] = math.inf
        v[0, 100] = -math.inf
        put(c, s, st + s % m, v=v)
    first = run_on(152, c)
    check_not_finite(c, first)
    for _ in range(20):
        assert torch.equal(run_on(152, c).view(torch.int16), first.view(torch.int16))


def test_a_warp_that_finishes_rows_of_a_long_context():
    """A CTA's first tile leaves the third and fourth warps of the second half many rows to be computed again from all keys (and the first
    and second none: NaN queries), while the first ones are at the next tile, of fewer than 64 keys, and wait for the others' part of it."""
    c = Cache([32, 5, 16, 3], [60000, 10, 4, 30], 4, 1, seed=31)
    q = c.q.clone()
    q[:16] = math.nan
    v = torch.zeros((1, D), dtype=torch.float16, device="cuda")
    put(c, 0, 60031, v=v)
    want, bound = c.attend()
    v[0, 100] = math.inf
    put(c, 0, 60031, v=v)
    got = run_on(1, c, q)
    assert torch.isnan(got[:16]).all()
    ref.check(got[16:31], want[16:31], bound[16:31])
    ref.check(got[32:], want[32:], bound[32:])
    assert (got[31, :, 100] == math.inf).all()
    rest = [d for d in range(D) if d != 100]
    ref.check(got[31:32, :, rest], want[31:32, :, rest], bound[31:32, :, rest])


@pytest.mark.parametrize("new,start", [([700, 3, 90, 1, 33], [3000, 20000, 100, 5, 900]), ([5], [9000]), ([600], [4000])])
def test_results_do_not_depend_on_timing(new, start):
    c = Cache(new, start, 8, 2, seed=sum(new) + 3)
    first = run_on(152, c)
    busy = torch.randn((2048, 2048), device="cuda")
    for i in range(10):
        if i % 2:
            busy = busy @ busy * 1e-3  # something before it on the stream
        assert torch.equal(run_on(152, c), first)
