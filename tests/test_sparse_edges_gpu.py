"""pkv_select_pages and pkv_sparse_decode_step where they can go wrong: many pages next to the border, values that are not finite in
selected pages, captured steps, other streams, calls in a row, grids of any size."""

import math

import pytest
import torch

import prompt_reference as ref
import serving_paged_gqa_gb300 as pkv
from paged_reference import D, PS, Cache, chunk_bound
from test_sparse_gpu import Step, best_scores, want_bounds, want_pages

pytestmark = pytest.mark.gpu


# ---- many pages next to the border: ranked by exact sums that fp32 does not tell apart ------------------------------------------
@pytest.mark.parametrize("n", [270, 600, 8192, 9500])
@pytest.mark.parametrize("sign", ["above", "below", "both"])
def test_many_scores_that_fp32_does_not_tell_apart(n, sign):
    """A sum of large products, the same for every page (positive, negative, or 0), and a small one, a whole number of 2^-12: 64-bit sums
    are exact."""
    s = Step([n * PS], 4, 1, seed=n)
    page = s.c.bt[0, :n].long()
    g = torch.Generator().manual_seed(n)
    s.q[0] = 0
    s.q[0, :, 0], s.q[0, :, 1], s.q[0, :, 2] = {"above": (1024.0, 0.0, 2.0 ** -10), "below": (-1024.0, 0.0, 2.0 ** -10),
                                               "both": (1024.0, -1024.0, 2.0 ** -10)}[sign]
    s.bounds[page] = 0
    s.bounds[page, 0, :, 0] = 1000.0
    s.bounds[page, 0, :, 1] = 1000.0
    r = torch.randint(-2000, 2000, (n,), generator=g)  # many of them twice and more
    s.bounds[page, 0, :, 2] = (r.half() / 4)[:, None].cuda()
    bd = s.bounds[page, 0].double()
    score = best_scores(s.q[0], bd.half())
    assert torch.equal(score.cpu(), {"above": 1024000.0, "below": -1024000.0, "both": 0.0}[sign] + r.double() / 4096)
    for k in (2, 30, n // 2, n - 1):
        assert s.select(k).flatten().tolist() == want_pages(score.cpu(), k)


@pytest.mark.parametrize("n", [400, 9000])
def test_groups_of_scores_on_either_side_of_the_border(n):
    """A third of the pages far above, a third far below, a third next to the border whose last selected page is among equal ones."""
    s = Step([n * PS + 5], 8, 2, seed=n + 1)
    n += 1
    page = s.c.bt[0, :n].long()
    g = torch.Generator().manual_seed(n)
    s.q[0] = 0
    s.q[0, :, 0], s.q[0, :, 1] = 1024.0, 2.0 ** -10
    s.bounds[page] = 0
    level = torch.randint(-1, 2, (n,), generator=g)
    r = torch.randint(0, 7, (2, n), generator=g)  # equal ones by the dozen
    s.bounds[page, :, :, 0] = (1000.0 + 500 * level).half().cuda()[:, None, None]
    s.bounds[page, :, :, 1] = r.half().cuda().T[:, :, None]
    ups = int((level == 1).sum())
    for k in (ups // 2, ups + 2, ups + int((level == 0).sum()) // 2, n - int((level == -1).sum()) // 3):
        assert torch.equal(s.select(k).cpu(), s.want(k))


@pytest.mark.parametrize("first", [100, 8170, 8192, 9300])
def test_few_pages_at_the_border_of_a_long_row(first):
    """Forty that fp32 does not tell apart, of which some are selected, wherever they lie in a row of 9500 pages."""
    n = 9500
    s = Step([n * PS], 4, 1, seed=first)
    page = s.c.bt[0, :n].long()
    s.q[0] = 0
    s.q[0, :, 0], s.q[0, :, 1] = 1024.0, 2.0 ** -10
    s.bounds[page] = 0
    s.bounds[page, 0, :, 0] = 100.0
    s.bounds[page[7::50], 0, :, 0] = 1000.0
    ups = set(range(7, n, 50)) - set(range(first, first + 40))
    s.bounds[page[first:first + 40], 0, :, 0] = 500.0
    r = torch.randint(0, 30, (40,), generator=torch.Generator().manual_seed(first))
    s.bounds[page[first:first + 40], 0, :, 1] = (r.half() / 4)[:, None].cuda()
    for more in (1, 20, 39):
        k = len(ups) + more + 1
        got = s.select(k).cpu()
        assert torch.equal(got, s.want(k))
        assert ups < set(got.flatten().tolist())


@pytest.mark.parametrize("n,hq,hkv", [(300, 4, 2), (2000, 32, 8), (9000, 2, 1)])
def test_a_page_with_a_key_of_great_magnitude(n, hq, hkv):
    """Its bounds widen the error of every score of the row, so that all pages are next to the border."""
    s = Step([n * PS, 700], hq, hkv, seed=n + 2)
    s.bounds[s.c.bt[0, n // 3].long(), :, 1, 17] = 60000.0
    s.bounds[s.c.bt[0, n // 2].long(), :, 0, 90] = -60000.0
    for k in (2, 17, n // 2):
        assert torch.equal(s.select(k).cpu(), s.want(k))


def test_many_pages_whose_bounds_are_not_finite():
    """More than are selected, and than are ranked side by side: the lowest ones."""
    s = Step([5000 * PS], 4, 2, seed=3)
    page = s.c.bt[0, 100:4000].long()
    s.bounds[page, 0, 1, 5] = math.inf
    s.bounds[page, 1, 0, 9] = math.nan
    for k in (7, 1000, 4500):
        assert torch.equal(s.select(k).cpu(), s.want(k))


# ---- values that are not finite in selected pages ------------------------------------------------------------------------------
def check_row(s, b, pages, out):
    """Row b against the definition over the tokens of its pages, values that are not finite among them."""
    g, n = s.hq // s.hkv, s.lens[b]
    k, v = s.c.rows(b, n)
    for h in range(s.hkv):
        at = [p * PS + i for p in pages[b, h].tolist() if p >= 0 for i in range(PS) if p * PS + i < n]
        kk, vv, q = k[at, h:h + 1], v[at, h:h + 1], s.q[b:b + 1, h * g:(h + 1) * g]
        zk, zv = torch.where(torch.isfinite(kk), kk, 0), torch.where(torch.isfinite(vv), vv, 0)
        want, mag = ref.attend(q, zk, zv, s.c.scale, len(at) - 1)
        bound = chunk_bound(want, mag, len(at), q, zk, zv, s.c.scale)
        y = out[b:b + 1, h * g:(h + 1) * g].double()
        up, down = ((vv == x).any(0).expand(g, D)[None] for x in (math.inf, -math.inf))
        nan = torch.isnan(vv).any(0).expand(g, D)[None] | (up & down) | bool(torch.isnan(kk).any())
        assert torch.isnan(y[nan]).all()
        assert (y[up & ~nan] == math.inf).all() and (y[down & ~nan] == -math.inf).all()
        rest = ~(nan | up | down)
        assert torch.isfinite(y[rest]).all() and ((y - want).abs() <= bound)[rest].all()


@pytest.mark.parametrize("hq,hkv", [(8, 2), (4, 4), (16, 1), (32, 8)])
@pytest.mark.parametrize("lens,k", [([40], 3), ([300, 5, 700], 4), ([6000, 17, 9000], 200), ([500] * 40, 7)])
def test_values_that_are_not_finite(hq, hkv, lens, k):
    s = Step(lens, hq, hkv, seed=len(lens) + hq)
    pages = s.select(k).cpu()
    for b, n in enumerate(lens):
        for h in range(hkv):
            mine = [p for p in pages[b, h].tolist() if p >= 0]
            what = (b + h) % 4
            first, last = mine[0], mine[-1]
            if what != 3:
                s.c.v[int(s.c.bt[b, first]), 0, h, (5, 77, 127)[what]] = (math.inf, -math.inf, math.nan)[what]
            if what == 1:
                s.c.v[int(s.c.bt[b, last]), (n - 1) % PS, h, 77] = math.inf
            if what == 2 and len(mine) > 2:
                s.c.k[int(s.c.bt[b, mine[1]]), 3, h, 4] = math.nan
            # one that is not selected leaves no trace
            other = next((p for p in range(-(-n // PS)) if p not in mine), None)
            if other is not None:
                s.c.v[int(s.c.bt[b, other]), :, h] = math.nan
                s.c.k[int(s.c.bt[b, other]), :, h] = math.inf
    out = s.decode(pages.cuda())
    for b in range(len(lens)):
        check_row(s, b, pages, out)


@pytest.mark.parametrize("n,k", [(3, 1), (100, 7), (700, 44), (20000, 300)])
def test_scores_of_minus_infinity(n, k):
    """Keys whose scores are all -inf have no weight: NaN where a row has no other, and nothing where it has some."""
    s = Step([n, n], 4, 1, seed=n)
    pages = s.select(k).cpu()
    s.q[:, :, 0] = 1.0
    rows = [[p * PS + i for p in pages[b, 0].tolist() if p >= 0 for i in range(PS) if p * PS + i < n] for b in range(2)]
    keep = rows[1][len(rows[1]) // 2:]  # of row 1 the second half
    for b in range(2):
        for at in rows[b]:
            if b == 0 or at not in keep:
                s.c.k[int(s.c.bt[b, at // PS]), at % PS, 0, 0] = -math.inf
    out = s.decode(pages.cuda())
    assert torch.isnan(out[0]).all()
    kk, vv = (x[keep] for x in s.c.rows(1, n))
    want, mag = ref.attend(s.q[1:], kk, vv, s.c.scale, len(keep) - 1)
    ref.check(out[1:], want, chunk_bound(want, mag, len(keep), s.q[1:], kk, vv, s.c.scale))


# ---- steps in a row ------------------------------------------------------------------------------------------------------------
class Steps:
    """Steps of changing queries, lengths and tables over one set of buffers."""

    def __init__(self, hq, hkv, k, seed):
        self.k, self.hq, self.hkv = k, hq, hkv
        g = torch.Generator().manual_seed(seed)
        self.each = []
        base = Step([1500, 2500, 900], hq, hkv, seed=seed)
        self.c = base.c
        for i in range(8):
            lens = [int(torch.randint(0, x + 1, (1,), generator=g)) for x in (1500, 2500, 900)]
            q = torch.randn((3, hq, D), generator=g).half().cuda()
            bt = self.c.bt.clone()
            rows = torch.arange(3) if i % 2 else torch.tensor([2, 0, 1])  # another row's pages
            lens = [lens[j] for j in rows.tolist()]
            self.each.append((q, torch.tensor(lens, dtype=torch.int32, device="cuda"), bt[rows.cuda()].contiguous(), lens))
        self.bounds, self.ws = base.bounds, base.ws
        self.q, self.sl, self.bt = base.q.clone(), base.sl.clone(), self.c.bt.clone()
        self.pages = torch.empty((3, hkv, k), dtype=torch.int32, device="cuda")
        self.out = torch.empty((3, hq, D), dtype=torch.float16, device="cuda")

    def fill(self, i):
        q, sl, bt, _ = self.each[i]
        self.q.copy_(q), self.sl.copy_(sl), self.bt.copy_(bt)

    def call(self, **kw):
        pkv.select_pages(self.q, self.bounds, self.bt, self.sl, self.k, pages=self.pages, ws=self.ws, **kw)
        pkv.sparse_decode(self.q, self.c.k, self.c.v, self.bt, self.sl, self.pages, out=self.out, ws=self.ws, **kw)

    def check(self, i, pages, out):
        q, _, bt, lens = self.each[i]
        g = self.hq // self.hkv
        for b, n in enumerate(lens):
            if n == 0:
                assert (pages[b] == -1).all() and (out[b] == 0).all()
                continue
            at = bt[b, : -(-n // PS)].long()
            pos = torch.arange(n, device="cuda")
            k, v = (x[at[pos // PS], pos % PS] for x in (self.c.k, self.c.v))
            for h in range(self.hkv):
                qq = q[b:b + 1, h * g:(h + 1) * g]
                mine = want_pages(best_scores(qq[0], self.bounds[at, h]).cpu(), self.k)
                assert pages[b, h].tolist() == mine
                rows = [p * PS + j for p in mine if p >= 0 for j in range(PS) if p * PS + j < n]
                want, mag = ref.attend(qq, k[rows, h:h + 1], v[rows, h:h + 1], 1 / math.sqrt(D), len(rows) - 1)
                bound = chunk_bound(want, mag, len(rows), qq, k[rows, h:h + 1], v[rows, h:h + 1], 1 / math.sqrt(D))
                ref.check(out[b:b + 1, h * g:(h + 1) * g], want, bound)


@pytest.mark.parametrize("hq,hkv,k", [(8, 2, 9), (32, 8, 30), (4, 1, 200), (4, 4, 1)])
@pytest.mark.parametrize("how", ["calls", "graph", "stream"])
def test_steps_in_a_row(hq, hkv, k, how):
    """Nothing waits on the host between steps: each takes what the one before it on the stream left, and no more."""
    s = Steps(hq, hkv, k, seed=k)
    side = torch.cuda.Stream() if how == "stream" else torch.cuda.current_stream()
    s.fill(0)
    s.call()
    if how == "graph":
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            s.call()
    torch.cuda.synchronize()
    got = []
    for turn in range(3):
        for i in range(8):
            with torch.cuda.stream(side):
                s.fill(i)
                if how == "graph":
                    graph.replay()
                elif how == "calls":
                    s.call()
                else:
                    with torch.cuda.stream(torch.cuda.default_stream()):  # the argument says where, not the current stream
                        s.call(stream=side)
                got.append((i, s.pages.clone(), s.out.clone()))
    torch.cuda.synchronize()
    assert pkv.pkv_read_status(s.ws) == 0
    for i, pages, out in got[:8]:
        s.check(i, pages, out)
    for n, (i, pages, out) in enumerate(got[8:]):
        assert torch.equal(pages, got[n % 8][1]) and torch.equal(out, got[n % 8][2])


def test_two_graphs_on_one_workspace():
    a, b = Steps(8, 2, 9, seed=1), Steps(4, 1, 40, seed=2)
    ws = a.ws if a.ws.numel() >= b.ws.numel() else b.ws
    graphs = []
    for s in (a, b):
        s.ws = ws
        s.fill(3)
        s.call()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s.call()
        graphs.append(g)
    for x, i in ((0, 1), (1, 5), (1, 2), (0, 6), (1, 0), (0, 0)):
        s = (a, b)[x]
        s.fill(i)
        graphs[x].replay()
        s.check(i, s.pages, s.out)
    assert pkv.pkv_read_status(ws) == 0


# ---- grids of any size ---------------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("sms", [1, 3, 20, 151])
def test_grids_of_any_size(sms, monkeypatch):
    monkeypatch.setattr(pkv.paged, "_num_sms", lambda dev: sms)
    # tables and bounds
    c = Cache([5, 0, 300, 1], [13, 9, 100, 2000], 6, 3, seed=sms)
    ws = pkv.alloc_workspace(pkv.PKV_PROMPT_WS_BYTES)
    got = torch.full((c.num_pages, 3, 2, D), 7.0, dtype=torch.float16, device="cuda")
    want = got.clone()
    for s, (m, st) in enumerate(zip(c.new, c.start)):
        if m:
            b, first = want_bounds(c, s, st + m), st // PS
            want[c.bt[s, first:len(b)].long()] = b[first:]
    pkv.page_bounds(c.k, c.cu, c.bt, got, start=c.st, ws=ws)
    assert torch.equal(got, want)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    rows, width, pool = 700, 9, 4000
    lens, table, free, count = i32([0] * rows), i32([-1] * (rows * width)).view(rows, width), i32(list(range(pool))), i32([pool])
    new = i32([i % 90 for i in range(rows)])
    slots = torch.full((int(new.sum()) + 3,), -9, dtype=torch.int64, device="cuda")
    cu, _ = pkv.tables_grow(new, lens, table, free, count, slots=slots, ws=ws)
    assert torch.equal(lens, new) and cu[1:].tolist() == new.cumsum(0).tolist()
    pages = (new + PS - 1) // PS
    assert int(count) == pool - int(pages.sum())
    row = torch.repeat_interleave(torch.arange(rows, device="cuda"), new.long())
    pos = torch.arange(len(row), device="cuda") - cu[row]
    assert torch.equal(slots[:-3], table[row, pos // PS].long() * PS + pos % PS) and (slots[-3:] == -9).all()
    pkv.tables_release(i32([1] * rows), lens, table, free, count, ws=ws)
    assert (lens == 0).all() and int(count) == pool and sorted(free.tolist()) == list(range(pool))
    assert pkv.pkv_read_status(ws) == 0
    # selection and the step over its pages
    s = Step([1000, 33, 0, 5000, 300], 24, 12, seed=sms)
    pages = s.select(17)
    assert torch.equal(pages.cpu(), s.want(17))
    want, bound = s.attend(pages)
    ref.check(s.decode(pages), want, bound)
