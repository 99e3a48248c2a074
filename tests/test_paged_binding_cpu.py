"""What the binding of the calls over tables hands to the library, on the CPU: the library's call is replaced by a list."""

import pytest
import torch

from serving_paged_gqa_gb300 import paged


@pytest.fixture
def called(monkeypatch):
    calls = []
    monkeypatch.setattr(paged, "_call", lambda dev, name, *args: calls.append((name, args)))
    monkeypatch.setattr(paged, "_num_sms", lambda dev: 152)
    monkeypatch.setattr(paged, "_handle", lambda stream, dev: 0)
    return calls


def i32(*x):
    return torch.tensor(x, dtype=torch.int32)


@pytest.mark.parametrize("slots,positions", [(0, None), (None, 0), (0, 0), (None, None), (3, None), (None, 3), (3, 3)])
def test_slots_and_positions_without_entries_are_not_those_that_nobody_asks_for(called, slots, positions):
    to = None if slots is None else torch.empty(slots, dtype=torch.int64)
    pos = None if positions is None else torch.empty(positions, dtype=torch.int32)
    ws = torch.zeros(256, dtype=torch.uint8)
    lens, free, count = i32(5, 9), i32(0, 1, 2, 3), i32(4)
    paged._grow(-1, None, 2, 4, 8, i32(1, 2), lens, torch.zeros((2, 4), dtype=torch.int32), free, count, i32(0, 0, 0), i32(0, 0), to, pos,
                lens, count, ws, None)
    (name, args), = called
    assert name == "pkv_tables_grow"
    got_to, got_pos, cap = args[8:11]
    assert (got_to is None) == (slots is None) and (got_pos is None) == (positions is None)
    assert cap == (slots if slots is not None else positions or 0)
    at = [x for x in args[1:10] if x is not None]
    assert all(at) and len(set(at)) == len(at)  # addresses, each at its own place
    if slots is not None:
        assert got_to % 8 == 0
    if slots:
        assert got_to == to.data_ptr()
    if positions:
        assert got_pos == pos.data_ptr()


def test_numbers_of_slots_and_positions_differ(called):
    lens, count = i32(5), i32(1)
    with pytest.raises(ValueError, match="positions"):
        paged._grow(-1, None, 1, 1, 1, i32(1), lens, i32(0).view(1, 1), i32(0), count, i32(0, 0), i32(0), torch.empty(0, dtype=torch.int64),
                    i32(7), lens, count, torch.zeros(256, dtype=torch.uint8), None)
    assert not called
