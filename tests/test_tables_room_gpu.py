"""pkv_tables_grow with slots and positions that have no entries: no room, not no limit."""

import pytest
import torch

import serving_paged_gqa_gb300 as pkv

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("slots,positions", [(True, False), (False, True), (True, True)])
def test_no_room_for_any_token(slots, positions):
    ws = pkv.alloc_workspace(pkv.PKV_PROMPT_WS_BYTES)
    lens, table, free, count = i32([5, 0]), i32([[7, -1], [-1, -1]]), i32([3, 4, 5]), i32([3])
    kw = {}
    if slots:
        kw["slots"] = torch.empty(0, dtype=torch.int64, device="cuda")
    if positions:
        kw["positions"] = torch.full((4,), -9, dtype=torch.int32, device="cuda")[:0]
    cu, start = pkv.tables_grow(i32([2, 20]), lens, table, free, count, ws=ws, **kw)
    torch.cuda.synchronize()
    assert pkv.pkv_read_status(ws) == pkv.PKV_STATUS_NO_PAGES
    assert lens.tolist() == [5, 0] and count.tolist() == [3] and table.tolist() == [[7, -1], [-1, -1]]
    assert cu.tolist() == [0, 0, 0] and start.tolist() == [5, 0]
    # nothing to be placed: nothing is missing
    cu, start = pkv.tables_grow(i32([0, 0]), lens, table, free, count, ws=ws, **kw)
    torch.cuda.synchronize()
    assert pkv.pkv_read_status(ws) == 0 and cu.tolist() == [0, 0, 0] and start.tolist() == [5, 0]
    assert bool((ws == 0).all())
