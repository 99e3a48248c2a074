"""pkv_page_bounds, pkv_select_pages and pkv_sparse_decode_step against their definitions in 64 bits."""

import math
import random

import pytest
import torch

import prompt_reference as ref
import serving_paged_gqa_gb300 as pkv
from paged_reference import D, PS, Cache, chunk_bound

pytestmark = pytest.mark.gpu


def want_bounds(c, s, n):
    """Least and greatest key of each page of row s's first n tokens: [pages, Hkv, 2, d]."""
    k = next(iter(c.rows(s, n)))
    return torch.stack([torch.stack((x.amin(0), x.amax(0)), 1) for x in k.split(PS)])


def best_scores(q, bounds):
    """q [G, d], bounds [pages, 2, d]: the pages' scores in 64 bits."""
    q, b = q.double(), bounds.double()
    return torch.maximum(q[:, None] * b[None, :, 0], q[:, None] * b[None, :, 1]).sum(-1).amax(0)


def want_pages(score, select):
    """The selection among the scores of all pages of a row."""
    n = len(score)
    score = [math.inf if not math.isfinite(x) else x for x in score[:-1].tolist()]
    mine = sorted(sorted(range(n - 1), key=lambda p: (-score[p], p))[: select - 1]) + [n - 1]
    return mine + [-1] * (select - len(mine))


class Step:
    """One decode step: a row of lens[b] tokens each."""

    def __init__(self, lens, hq, hkv, seed=0, **kw):
        self.c = Cache([1 if n else 0 for n in lens], [max(n - 1, 0) for n in lens], hq, hkv, seed=seed, behind=0, **kw)
        g = torch.Generator(device="cuda").manual_seed(seed + 99)
        self.lens, self.hq, self.hkv = lens, hq, hkv
        self.q = torch.randn((len(lens), hq, D), generator=g, device="cuda").half()
        self.sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
        c = self.c
        self.bounds = torch.full((c.num_pages, hkv, 2, D), math.nan, dtype=torch.float16, device="cuda")
        for b, n in enumerate(lens):
            if n:
                self.bounds[c.bt[b, : -(-n // PS)].long()] = want_bounds(c, b, n)
        self.ws = pkv.alloc_workspace(pkv.pkv_sparse_workspace_bytes(pkv.sparse_problem(self.q, c.k, c.bt)))

    def select(self, k, status=0, **kw):
        got = pkv.select_pages(self.q, self.bounds, self.c.bt, self.sl, k, ws=self.ws, **kw)
        torch.cuda.synchronize()
        assert pkv.pkv_read_status(self.ws) == status
        return got

    def want(self, k):
        g, out = self.hq // self.hkv, []
        for b, n in enumerate(self.lens):
            for h in range(self.hkv):
                if n == 0:
                    out.append([-1] * k)
                    continue
                bd = self.bounds[self.c.bt[b, : -(-n // PS)].long(), h]
                score = best_scores(self.q[b, h * g:(h + 1) * g], bd)
                bad = ~(torch.isfinite(bd).all(-1).all(-1) & torch.isfinite(self.q[b, h * g:(h + 1) * g]).all())
                out.append(want_pages(torch.where(bad, math.inf, score), k))
        return torch.tensor(out, dtype=torch.int32).view(len(self.lens), self.hkv, k)

    def attend(self, pages):
        """out and the bound of its error for given pages."""
        c, g = self.c, self.hq // self.hkv
        out = torch.zeros((len(self.lens), self.hq, D), dtype=torch.float64, device="cuda")
        bound = torch.zeros_like(out)
        for b, n in enumerate(self.lens):
            if n == 0:
                continue
            k, v = c.rows(b, n)
            for h in range(self.hkv):
                at = [p * PS + i for p in pages[b, h].tolist() if p >= 0 for i in range(PS) if p * PS + i < n]
                kk, vv, q = k[at, h:h + 1], v[at, h:h + 1], self.q[b:b + 1, h * g:(h + 1) * g]
                o, mag = ref.attend(q, kk, vv, c.scale, len(at) - 1)
                out[b, h * g:(h + 1) * g] = o[0]
                bound[b, h * g:(h + 1) * g] = chunk_bound(o, mag, len(at), q, kk, vv, c.scale)[0]
        return out, bound

    def decode(self, pages, **kw):
        out = torch.full_like(self.q, 7.0)
        c = self.c
        pkv.sparse_decode(self.q, c.k, c.v, c.bt, self.sl, pages, ws=self.ws, out=out, **kw)
        torch.cuda.synchronize()
        assert pkv.pkv_read_status(self.ws) == 0
        return out


@pytest.mark.parametrize("hkv", [1, 2, 3, 8, 12])
@pytest.mark.parametrize("new,start", [([1], [0]), ([1], [16]), ([5, 0, 40], [13, 9, 100]), ([1] * 40, list(range(40))), ([700], [3])])
def test_bounds(hkv, new, start):
    c = Cache(new, start, hkv, hkv, seed=len(new) + hkv)
    got = torch.full((c.num_pages, hkv, 2, D), 7.0, dtype=torch.float16, device="cuda")
    want = got.clone()
    for s, (m, st) in enumerate(zip(new, start)):
        if m:
            b, first = want_bounds(c, s, st + m), st // PS
            want[c.bt[s, first:len(b)].long()] = b[first:]
    ws = pkv.alloc_workspace(pkv.PKV_PROMPT_WS_BYTES)
    pkv.page_bounds(c.k, c.cu, c.bt, got, start=c.st, ws=ws)
    torch.cuda.synchronize()
    assert pkv.pkv_read_status(ws) == 0
    assert torch.equal(got, want)


def test_bounds_of_nan_and_infinity():
    c = Cache([40], [0], 2, 2, seed=1)
    page = c.bt[0].long()
    c.k[page[0], 3, 1, 7] = math.nan
    c.k[page[1], 4, 0, 9] = math.inf
    c.k[page[2], 1, 0, 2] = -math.inf
    got = torch.zeros((c.num_pages, 2, 2, D), dtype=torch.float16, device="cuda")
    pkv.page_bounds(c.k, c.cu, c.bt, got, start=c.st)
    assert torch.isnan(got[page[0], 1, :, 7]).all() and int(torch.isnan(got).sum()) == 2
    assert got[page[1], 0, 1, 9] == math.inf and got[page[2], 0, 0, 2] == -math.inf and int(torch.isinf(got).sum()) == 2


HEADS = [(1, 1), (2, 1), (4, 2), (32, 8), (8, 1), (16, 1), (6, 3), (24, 12)]


@pytest.mark.parametrize("hq,hkv", HEADS)
@pytest.mark.parametrize("lens,k", [([1], 1), ([16], 3), ([17, 0, 400], 5), ([1000, 33, 5000], 17), ([300] * 5, 1), ([300] * 5, 2), ([700], 44)])
def test_selection(hq, hkv, lens, k):
    s = Step(lens, hq, hkv, seed=len(lens) + hq)
    assert torch.equal(s.select(k).cpu(), s.want(k))


@pytest.mark.parametrize("n,k", [(70000, 64), (140000, 500), (66000, 4000)])
def test_selection_of_long_rows(n, k):
    s = Step([n, 2000], 4, 2, seed=n)
    assert torch.equal(s.select(k).cpu(), s.want(k))


@pytest.mark.parametrize("lens", [[500], [6000], [70000]])
def test_equal_scores_go_to_the_lowest_pages(lens):
    s = Step(lens, 4, 2, seed=2)
    s.q[:, :2] = 0  # one KV head's queries: every page scores 0
    n = -(-lens[0] // PS)
    s.bounds[s.c.bt[0, 5:n // 2].long()] = s.bounds[s.c.bt[0, 5].long()].clone()  # and many pages like each other
    k = min(n - 1, 20)
    assert torch.equal(s.select(k).cpu(), s.want(k))


def test_scores_that_differ_less_than_fp32_has():
    s = Step([4000], 4, 1, seed=3)
    n = 250
    page = s.c.bt[0, :n].long()
    s.q[0, :, 1:] = 0
    s.q[0, :, 0], s.q[0, :, 1] = 1024.0, 2.0 ** -10  # sums of a large and a small product
    s.bounds[page] = 0
    s.bounds[page, 0, :, 0] = 1000.0
    r = torch.randperm(n, generator=torch.Generator().manual_seed(4)).to(page.device)
    s.bounds[page, 0, :, 1] = (r.half() / 4)[:, None]
    k = 60
    want = s.want(k)
    assert torch.equal(s.select(k).cpu(), want)
    top = set(torch.topk(r[: n - 1], k - 1).indices.tolist()) | {n - 1}
    assert set(want.flatten().tolist()) == top


def whole(x):
    """fp16 values as whole numbers of 2^-24."""
    return [int(y * 2 ** 24) for y in x.double().flatten().tolist()]


@pytest.mark.parametrize("seed", range(4))
def test_scores_of_all_exponents(seed):
    s = Step([1600], 4, 1, seed=8)
    n, g = 100, torch.Generator().manual_seed(seed)
    page = s.c.bt[0, :n].long()

    def magnitudes(*shape):  # every exponent alike, numbers below the least normal one among them
        return torch.randint(0, 0x7800, shape, generator=g, dtype=torch.int16)

    s.q[0] = (magnitudes(4, D).view(torch.float16) * (1 - 2 * torch.randint(0, 2, (4, D), generator=g))).half().cuda()
    bits = magnitudes(2, D).repeat(n, 1, 1)
    for p in range(n):  # a page is the same as the others but for a few steps in one dim
        bits[p, :, int(torch.randint(0, D, (1,), generator=g))] += int(torch.randint(0, 40, (1,), generator=g))
    b = bits.view(torch.float16)
    b = torch.stack((-b[:, 0], b[:, 1]), 1)
    s.bounds[page, 0] = b.cuda()
    heads = [whole(x) for x in s.q[0].cpu()]
    score = []
    for p in range(n):
        lo, hi = whole(b[p, 0]), whole(b[p, 1])
        score.append(max(sum(x * (h if x > 0 else l) for x, l, h in zip(q, lo, hi)) for q in heads))
    for k in (2, 13, 50, 90):
        want = sorted(sorted(range(n - 1), key=lambda p: (-score[p], p))[: k - 1]) + [n - 1]
        assert s.select(k).flatten().tolist() == want


def test_bounds_and_queries_that_are_not_finite():
    s = Step([2000, 900], 8, 2, seed=5)
    page = s.c.bt[0].long()
    s.bounds[page[7], 0, 0, 3] = math.nan
    s.bounds[page[90], 0, 1, 100] = math.inf
    s.bounds[page[91], 0, 0, 100] = -math.inf
    s.bounds[page[3], 1, 1, 0] = math.inf
    assert torch.equal(s.select(9).cpu(), s.want(9))
    s.q[1, 5, 77] = math.nan
    s.q[1, 1, 7] = -math.inf
    got = s.select(9).cpu()
    assert torch.equal(got, s.want(9))
    assert got[1, 0].tolist() == list(range(8)) + [56]


def test_bad_lengths_and_pages():
    s = Step([300, 500, 400], 4, 2, seed=6)
    s.sl[0] = -1
    got = s.select(4, status=pkv.PKV_STATUS_BAD_LEN)
    assert (got[0] == -1).all() and torch.equal(got[1:].cpu(), s.want(4)[1:])
    s.sl[0] = 300
    s.c.bt[1, 3] = s.c.num_pages
    got = s.select(4, status=pkv.PKV_STATUS_BAD_PAGE)
    zero = s.bounds[s.c.bt[1, :32].clamp(0, s.c.num_pages - 1).long()].clone()
    zero[3] = 0
    for h in range(2):
        assert got[1, h].tolist() == want_pages(best_scores(s.q[1, 2 * h:2 * h + 2], zero[:, h]), 4)


@pytest.mark.parametrize("hq,hkv", HEADS)
@pytest.mark.parametrize("lens,k", [([1], 1), ([16], 3), ([17, 0, 400], 5), ([1000, 33, 5000], 17), ([300] * 5, 1)])
def test_step(hq, hkv, lens, k):
    s = Step(lens, hq, hkv, seed=len(lens) + hq)
    pages = s.select(k)
    want, bound = s.attend(pages)
    ref.check(s.decode(pages), want, bound)


def test_step_of_a_batch_of_long_rows():
    r = random.Random(7)
    s = Step([r.randint(1, 20000) for _ in range(24)] + [0, 5], 32, 8, seed=8)
    pages = s.select(96)
    assert torch.equal(pages.cpu(), s.want(96))
    want, bound = s.attend(pages)
    ref.check(s.decode(pages), want, bound)


def test_step_over_all_pages_is_the_decode_step():
    s = Step([700, 64, 1], 32, 8, seed=9)
    c, pages = s.c, s.select(50)
    own = pkv.decode(s.q, c.k, c.v, c.bt, s.sl)
    assert (s.decode(pages).float() - own.float()).abs().max() < 4e-3


def test_pages_that_are_not_there():
    s = Step([400, 300], 4, 2, seed=10)
    c, pages = s.c, s.select(4)
    good = s.decode(pages)
    pages[0, 0, 1] = c.bt.shape[1]  # outside the table
    out = torch.empty_like(s.q)
    pkv.sparse_decode(s.q, c.k, c.v, c.bt, s.sl, pages, ws=s.ws, out=out)
    torch.cuda.synchronize()
    assert pkv.pkv_read_status(s.ws) == pkv.PKV_STATUS_BAD_PAGE
    assert torch.equal(out[0, 2:], good[0, 2:]) and torch.equal(out[1], good[1]) and torch.isfinite(out).all()
    assert not torch.equal(out[0, :2], good[0, :2])


def test_bad_lengths_of_the_step():
    s = Step([400, 300], 4, 2, seed=11)
    c, pages = s.c, s.select(4)
    good = s.decode(pages)
    s.sl[0] = -5
    out = torch.full_like(s.q, 7.0)
    pkv.sparse_decode(s.q, c.k, c.v, c.bt, s.sl, pages, ws=s.ws, out=out)
    torch.cuda.synchronize()
    assert pkv.pkv_read_status(s.ws) == pkv.PKV_STATUS_BAD_LEN
    assert (out[0] == 0).all() and torch.equal(out[1], good[1])
