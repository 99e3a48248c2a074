"""pkv_tables_grow and pkv_tables_release against tables that are kept row by row on the host."""

import random

import pytest
import torch

import serving_paged_gqa_gb300 as pkv

pytestmark = pytest.mark.gpu
PS = 16


def pages(n):
    return -(-n // PS)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.fixture(scope="module")
def ws():
    return pkv.alloc_workspace(pkv.PKV_PROMPT_WS_BYTES)


class Host:
    """Rows, their tables and the stack, by the definition."""

    def __init__(self, lens, num_pages, width, seed=0):
        r = random.Random(seed)
        order = list(range(num_pages))
        r.shuffle(order)
        self.lens, self.width, self.num_pages = list(lens), width, num_pages
        self.table = [[-1] * width for _ in lens]
        for b, n in enumerate(lens):
            for p in range(pages(n) if 0 <= n <= width * PS else 0):
                self.table[b][p] = order.pop()
        self.count = len(order)
        self.stack = order + [-1] * (num_pages - len(order))

    def grow(self, new, capacity=1 << 40):
        tokens = need = 0
        status, cu, start, slots, positions = 0, [0], list(self.lens), [], []
        taken = 0
        for b, (n, m) in enumerate(zip(self.lens, new)):
            if n < 0 or m < 0 or n + m > self.width * PS:
                status, m = status | pkv.PKV_STATUS_BAD_LEN, 0
            tokens += m
            more = pages(n + m) - pages(n) if m else 0
            need += more
            if m and (tokens > capacity or (more and need > self.count)):
                status, m, more = status | pkv.PKV_STATUS_NO_PAGES, 0, 0
            for p in range(more):
                self.table[b][pages(n) + p] = self.stack[self.count - 1 - taken]
                taken += 1
            for pos in range(n, n + m):
                slots.append(self.table[b][pos // PS] * PS + pos % PS)
                positions.append(pos)
            self.lens[b] = n + m
            cu.append(cu[-1] + m)
        self.count -= taken
        return status, cu, start, slots, positions

    def release(self, ended):
        given = [b for b, e in enumerate(ended) if e and 0 <= self.lens[b] <= self.width * PS]
        status = pkv.PKV_STATUS_BAD_LEN if any(e and b not in given for b, e in enumerate(ended)) else 0
        back = [self.table[b][p] for b in given for p in range(pages(self.lens[b]))]
        if self.count + len(back) > self.num_pages:
            return pkv.PKV_STATUS_BAD_LEN
        self.stack[self.count:self.count + len(back)] = back
        self.count += len(back)
        for b in given:
            self.lens[b] = 0
        return status


class Device:
    def __init__(self, h):
        self.lens, self.table = i32(h.lens), i32(h.table).view(len(h.lens), h.width)
        self.stack, self.count = i32(h.stack), i32([h.count])

    def same(self, h):
        torch.cuda.synchronize()
        assert self.lens.tolist() == h.lens
        assert self.count.tolist() == [h.count]
        assert self.stack.tolist() == h.stack
        assert self.table.tolist() == h.table


def grow(d, h, new, ws, capacity=None, spare=3, in_place=True):
    room = sum(max(x, 0) for x in new) if capacity is None else capacity
    slots = torch.full((room + (spare if capacity is None else 0),), -9, dtype=torch.int64, device="cuda")
    positions = torch.full((slots.numel(),), -9, dtype=torch.int32, device="cuda")
    outs = {} if in_place else dict(seq_lens_out=torch.empty_like(d.lens), free_count_out=torch.empty_like(d.count))
    lens, count = d.lens.clone(), d.count.clone()
    cu, start = pkv.tables_grow(i32(new), d.lens, d.table, d.stack, d.count, slots=slots, positions=positions, ws=ws, **outs)
    if outs:
        assert torch.equal(lens, d.lens) and torch.equal(count, d.count)
        d.lens, d.count = outs["seq_lens_out"], outs["free_count_out"]
    status, w_cu, w_start, w_slots, w_pos = h.grow(new, slots.numel())
    d.same(h)
    rest = slots.numel() - len(w_slots)
    assert cu.tolist() == w_cu and start.tolist() == w_start
    assert slots.tolist() == w_slots + [-9] * rest and positions.tolist() == w_pos + [-9] * rest
    assert pkv.pkv_read_status(ws) == status
    assert ws[:256].view(torch.int32)[[0, 3]].tolist() == [0, 0]  # the counters are back
    return status


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("lens,new", [
    ([0], [1]), ([0], [0]), ([15], [1]), ([16], [1]), ([17], [15]), ([0, 5, 16, 31], [16, 0, 17, 2]), ([7], [1000]),
    ([0] * 40, [1] * 40), ([33] * 33, list(range(33))),
])
def test_grow(ws, lens, new, in_place):
    h = Host(lens, 400, 80, seed=len(lens))
    assert grow(Device(h), h, new, ws, in_place=in_place) == 0


@pytest.mark.parametrize("rows,most", [(513, 40), (4096, 3), (1000, 1), (64, 4000), (3, 20000)])
def test_many_rows_and_tokens(ws, rows, most):
    r = random.Random(rows)
    lens, new = [r.randint(0, 70) for _ in range(rows)], [r.randint(0, most) for _ in range(rows)]
    h = Host(lens, sum(pages(a + b) for a, b in zip(lens, new)) + 5, pages(most + 70) + 1, seed=1)
    assert grow(Device(h), h, new, ws) == 0


def test_a_loop_of_steps(ws):
    r = random.Random(3)
    h = Host([0] * 24, 300, 40, seed=4)
    d = Device(h)
    for step in range(30):
        grow(d, h, [r.choice([0, 1, 1, 1, r.randint(2, 60)]) if h.lens[b] < 500 else 0 for b in range(24)], ws)
        ended = [int(h.lens[b] > 100 and r.random() < 0.3) for b in range(24)]
        pkv.tables_release(i32(ended), d.lens, d.table, d.stack, d.count, ws=ws)
        assert h.release(ended) == 0
        d.same(h)
        assert pkv.pkv_read_status(ws) == 0
        held = [h.table[b][p] for b in range(24) for p in range(pages(h.lens[b]))] + h.stack[: h.count]
        assert sorted(held) == list(range(300))  # every page in one place


def test_pages_run_out(ws):
    h = Host([10, 0, 20, 3], 9, 20, seed=5)  # 9 pages, of which 4 are held
    d = Device(h)
    # the second row takes 3 of 5, the third needs 4, the fourth fits the page that it has, the first, too
    assert grow(d, h, [5, 48, 70, 13], ws) == pkv.PKV_STATUS_NO_PAGES
    assert h.lens == [15, 48, 20, 16]


def test_slots_run_out(ws):
    h = Host([10, 0, 20, 3], 100, 20, seed=6)
    assert grow(Device(h), h, [5, 48, 0, 13], ws, capacity=53) == pkv.PKV_STATUS_NO_PAGES
    assert h.lens == [15, 48, 20, 3]


def test_no_slots_no_limit(ws):
    h = Host([10, 0], 100, 20, seed=6)
    d = Device(h)
    cu, start = pkv.tables_grow(i32([100, 200]), d.lens, d.table, d.stack, d.count, ws=ws)
    status, w_cu, w_start, _, _ = h.grow([100, 200])
    d.same(h)
    assert (cu.tolist(), start.tolist(), status) == (w_cu, w_start, 0)


def test_rows_out_of_order(ws):
    h = Host([10, -1, 0, 320, 5, 321], 100, 20, seed=7)
    assert grow(Device(h), h, [-3, 4, 30, 1, 2147483647, 0], ws, capacity=40) == pkv.PKV_STATUS_BAD_LEN


@pytest.mark.parametrize("in_place", [True, False])
def test_release(ws, in_place):
    h = Host([0, 1, 16, 17, 300, 5, 320], 100, 20, seed=8)
    d = Device(h)
    ended = [1, 0, 2, -1, 1, 0, 1]
    outs = {} if in_place else dict(seq_lens_out=torch.empty_like(d.lens), free_count_out=torch.empty_like(d.count))
    pkv.tables_release(i32(ended), d.lens, d.table, d.stack, d.count, ws=ws, **outs)
    if outs:
        d.lens, d.count = outs["seq_lens_out"], outs["free_count_out"]
    assert h.release(ended) == 0
    d.same(h)
    assert pkv.pkv_read_status(ws) == 0


def test_release_of_many_pages(ws):
    r = random.Random(9)
    lens = [r.randint(0, 9000) for _ in range(300)]
    h = Host(lens, sum(map(pages, lens)) + 3, pages(9000), seed=9)
    d = Device(h)
    ended = [r.randint(0, 1) for _ in lens]
    pkv.tables_release(i32(ended), d.lens, d.table, d.stack, d.count, ws=ws)
    assert h.release(ended) == 0
    d.same(h)


def test_release_refuses_what_is_not_in_order(ws):
    h = Host([16, -4, 500], 50, 20, seed=10)
    d = Device(h)
    pkv.tables_release(i32([1, 1, 1]), d.lens, d.table, d.stack, d.count, ws=ws)
    assert h.release([1, 1, 1]) == pkv.PKV_STATUS_BAD_LEN == pkv.pkv_read_status(ws)
    d.same(h)
    d.count.fill_(50)  # a stack that is full already
    h.count = 50
    d.lens.fill_(16)
    h.lens = [16] * 3
    pkv.tables_release(i32([1, 0, 0]), d.lens, d.table, d.stack, d.count, ws=ws)
    assert h.release([1, 0, 0]) == pkv.PKV_STATUS_BAD_LEN == pkv.pkv_read_status(ws)
    d.same(h)


def test_no_rows(ws):
    d = Device(Host([], 10, 4))
    cu, _ = pkv.tables_grow(i32([]), d.lens, d.table.view(0, 4), d.stack, d.count, ws=ws)
    torch.cuda.synchronize()
    assert cu.tolist() == [0] and d.count.tolist() == [10]


def test_captured_steps(ws):
    h = Host([5] * 8, 200, 20, seed=11)
    d = Device(h)
    new = i32([1] * 8)
    cu, start, slots = i32([0] * 9), i32([0] * 8), torch.zeros(8, dtype=torch.int64, device="cuda")
    def call():
        pkv.tables_grow(new, d.lens, d.table, d.stack, d.count, cu_seqlens=cu, start=start, slots=slots, ws=ws)
    call()
    h.grow([1] * 8)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for _ in range(30):
        g.replay()
        _, w_cu, w_start, w_slots, _ = h.grow([1] * 8)
        d.same(h)
        assert slots.tolist() == w_slots and start.tolist() == w_start and cu.tolist() == w_cu
