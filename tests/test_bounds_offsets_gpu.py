"""pkv_page_bounds of sequences that are a part of the packed rows."""

import math

import pytest
import torch

import serving_paged_gqa_gb300 as pkv
from paged_reference import D, Cache

pytestmark = pytest.mark.gpu


def bounds_of(c, ws, cu, first=0, last=None, status=0):
    rows = slice(first, last)
    got = torch.full((c.num_pages, c.hkv, 2, D), 7.0, dtype=torch.float16, device="cuda")
    pkv.page_bounds(c.k, cu, c.bt[rows], got, start=c.st[rows], ws=ws)
    torch.cuda.synchronize()
    assert pkv.pkv_read_status(ws) == status
    return got


@pytest.fixture(scope="module")
def ws():
    return pkv.alloc_workspace(pkv.PKV_PROMPT_WS_BYTES)


@pytest.mark.parametrize("new,start", [([5], [3]), ([40, 0, 9], [7, 12, 100]), ([1] * 35, list(range(35)))])
def test_packed_rows_before_the_sequences(ws, new, start):
    """Any first packed row, also behind the last token that the block table has room for."""
    c = Cache(new, start, 2, 2, seed=len(new))
    want = bounds_of(c, ws, c.cu)
    room = c.bt.numel() * 16
    for first in (1, room - c.tokens, room - c.tokens + 1, room, room + 12345, 2 ** 31 - 1 - c.tokens):
        assert torch.equal(bounds_of(c, ws, c.cu + first), want)


def test_a_part_of_the_batch(ws):
    """The last sequences of a batch, behind long ones: the append takes their packed rows where they are, and so do the bounds."""
    c = Cache([3000, 2000, 20, 1], [0, 5, 30, 15], 2, 2, seed=9)
    c.bt = c.bt.contiguous()
    part = c.bt[2:, :4].contiguous()  # a table with no more columns than these need
    want = bounds_of(c, ws, c.cu[2:], 2)
    got = torch.full_like(want, 7.0)
    pkv.page_bounds(c.k, c.cu[2:], part, got, start=c.st[2:], ws=ws)
    torch.cuda.synchronize()
    assert pkv.pkv_read_status(ws) == 0 and torch.equal(got, want)
    full = bounds_of(c, ws, c.cu)
    pages = part[part.ge(0) & part.lt(c.num_pages)].long()
    assert torch.equal(got[pages], full[pages]) and bool((got[pages] != 7.0).any())


def test_a_sequence_that_is_skipped_takes_none_behind_it_along(ws):
    """A row that would outgrow its table is skipped; the packed rows of those behind it begin where its own would end."""
    c = Cache([5, 40], [3, 7], 2, 2, seed=4)
    want = bounds_of(c, ws, c.cu)
    cu = torch.tensor([0, 1000000, 1000040], dtype=torch.int32, device="cuda")
    got = bounds_of(c, ws, cu, status=pkv.PKV_STATUS_BAD_LEN)
    mine = c.bt[1, :3].long()
    assert torch.equal(got[mine], want[mine])
    got[mine] = 7.0
    assert (got == 7.0).all()


def test_tables_without_columns_and_without_rows(ws):
    k = torch.zeros((4, 16, 2, D), dtype=torch.float16, device="cuda")
    got = torch.full((4, 2, 2, D), math.nan, dtype=torch.float16, device="cuda")
    for b in (0, 3):
        cu = torch.zeros(b + 1, dtype=torch.int32, device="cuda")
        pkv.page_bounds(k, cu, torch.zeros((b, 0), dtype=torch.int32, device="cuda"), got, ws=ws)
    torch.cuda.synchronize()
    assert torch.isnan(got).all() and pkv.pkv_read_status(ws) == 0
