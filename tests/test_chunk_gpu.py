"""pkv_chunk_attention against its definition in 64 bits."""

import math

import pytest
import torch

import prompt_reference as ref
import serving_paged_gqa_gb300 as pkv
from paged_reference import Cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ws():
    return pkv.alloc_workspace(pkv.pkv_chunk_workspace_bytes())


def run(c, ws, **kw):
    out = torch.full((c.q.shape[0] + 0, c.hq, 128), 7.0, dtype=torch.float16, device="cuda")
    kw = {"start": c.st, "out": out, "ws": ws, **kw}
    got = pkv.chunk_attention(c.q, c.k, c.v, c.cu, c.bt, **kw)
    return got


def check(c, ws, status=0, **kw):
    got = run(c, ws, **kw)
    torch.cuda.synchronize()
    assert pkv.pkv_read_status(ws) == status
    want, bound = c.attend()
    ref.check(got[: c.tokens], want, bound)
    assert (got[c.tokens:] == 7.0).all()
    return got


HEADS = [(1, 1), (2, 1), (4, 1), (8, 1), (16, 1), (32, 8), (32, 4), (6, 3), (20, 5), (14, 7), (24, 12)]


@pytest.mark.parametrize("hq,hkv", HEADS)
@pytest.mark.parametrize("new,start", [
    ([1], [0]), ([1], [700]), ([5], [123]), ([17, 0, 1, 200], [0, 9, 300, 55]), ([130], [1]), ([300], [5000]),
    ([2, 3, 1, 8], [2000, 17, 0, 4095]),
])
def test_shapes(ws, hq, hkv, new, start):
    check(Cache(new, start, hq, hkv, seed=len(new) + hq), ws)


@pytest.mark.parametrize("start", [0, 1, 15, 16, 63, 64, 65, 111, 112, 127, 128, 129, 255, 256, 257])
@pytest.mark.parametrize("n", [1, 31, 32, 33, 64, 128, 129])
def test_borders_of_steps_and_pages(ws, n, start):
    check(Cache([n], [start], 8, 2, seed=n + start), ws)


@pytest.mark.parametrize("hq,hkv", [(32, 8), (16, 1), (4, 4)])
def test_long_contexts_are_cut_into_pieces(ws, hq, hkv):
    check(Cache([3, 1, 40], [20000, 33001, 9000], hq, hkv, seed=3), ws)


@pytest.mark.parametrize("hq,hkv", [(32, 8), (8, 8), (16, 1)])
def test_long_chunks(ws, hq, hkv):
    check(Cache([1500, 700], [3000, 0], hq, hkv, seed=4, fused=True), ws)


def test_many_short_sequences(ws):
    g = torch.Generator().manual_seed(5)
    n = torch.randint(0, 4, (1300,), generator=g).tolist()
    st = torch.randint(0, 60, (1300,), generator=g).tolist()
    check(Cache(n, st, 8, 2, seed=6), ws)


def test_no_start_means_none(ws):
    c = Cache([40, 3], [0, 0], 8, 2, seed=7)
    got = check(c, ws, start=None)
    k, v = torch.cat([list(c.rows(s, n))[0] for s, n in enumerate(c.new)]), torch.cat([list(c.rows(s, n))[1] for s, n in enumerate(c.new)])
    own = pkv.prompt_attention(c.q[: c.tokens], k, v, c.cu)
    assert (own.float() - got[: c.tokens].float()).abs().max() < 4e-3


def test_strided_outputs(ws):
    c = Cache([33, 2], [100, 7], 16, 2, seed=8, fused=True)
    wide = torch.full((c.q.shape[0], 24, 128), 7.0, dtype=torch.float16, device="cuda")
    check(c, ws, out=wide[:, :16])
    assert (wide[:, 16:] == 7.0).all()


def test_same_results_whatever_ran_before(ws):
    c = Cache([9, 300, 1], [4000, 100, 31000], 32, 8, seed=9)
    first = run(c, ws).clone()
    check(Cache([100], [3000], 8, 8, seed=10), ws)
    for _ in range(5):
        assert torch.equal(run(c, ws), first)
