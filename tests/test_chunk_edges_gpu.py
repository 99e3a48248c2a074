"""pkv_chunk_attention where it can go wrong: values that are not finite, scores far apart, bad pages and lengths, grids of any
size, captured calls, other streams, pools beyond 4 GB."""

import ctypes
import math

import pytest
import torch

import prompt_reference as ref
import serving_paged_gqa_gb300 as pkv
from paged_reference import D, PS, Cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ws():
    return pkv.alloc_workspace(pkv.pkv_chunk_workspace_bytes())


def run(c, ws, status=0, **kw):
    out = torch.full((c.q.shape[0], c.hq, D), 7.0, dtype=torch.float16, device="cuda")
    got = pkv.chunk_attention(c.q, c.k, c.v, c.cu, c.bt, **{"start": c.st, "out": out, "ws": ws, "scale": c.scale, **kw})
    torch.cuda.synchronize()
    assert pkv.pkv_read_status(ws) == status
    assert (got[c.tokens:] == 7.0).all()
    return got[: c.tokens]


def put(c, s, pos, k=None, v=None):
    page, slot = int(c.bt[s, pos // PS]), pos % PS
    if k is not None:
        c.k[page, slot] = k
    if v is not None:
        c.v[page, slot] = v


def check_not_finite(c, got):
    """Rows against the definition where V or K has infinities and NaN: a value that a row does not attend to leaves no trace."""
    at = 0
    for s, (m, st) in enumerate(zip(c.new, c.start)):
        k, v = c.rows(s, st + m)
        bad_k = ~torch.isfinite(k).all(-1)  # [n, Hkv]: NaN scores (their queries have both signs)
        for i in range(0, m, 256):
            r = min(256, m - i)
            n = st + i + r
            q = c.q[at + i:at + i + r]
            zk, zv = torch.where(torch.isfinite(k[:n]), k[:n], 0), torch.where(torch.isfinite(v[:n]), v[:n], 0)
            want, mag = ref.attend(q, zk, zv, c.scale, st + i)
            from paged_reference import chunk_bound

            bound = chunk_bound(want, mag, n, q, zk, zv, c.scale)
            seen = torch.arange(n, device=q.device)[None] <= st + i + torch.arange(r, device=q.device)[:, None]
            g = c.hq // c.hkv

            def any_seen(x):  # x [n, Hkv, ...] -> [r, Hq, ...]
                return (torch.einsum("rn,nhd->rhd", seen.double(), x.double()) > 0).repeat_interleave(g, 1)

            up, down, nan = any_seen(v[:n] == math.inf), any_seen(v[:n] == -math.inf), any_seen(torch.isnan(v[:n]))
            lost = any_seen(bad_k[:n, :, None]).expand_as(up)
            y = got[at + i:at + i + r].double()
            nan = nan | (up & down) | lost
            assert torch.isnan(y[nan]).all()
            assert (y[up & ~nan] == math.inf).all() and (y[down & ~nan] == -math.inf).all()
            rest = ~(nan | up | down)
            assert torch.isfinite(y[rest]).all()
            assert ((y - want).abs() <= bound)[rest].all()
        at += m


@pytest.mark.parametrize("hq,hkv", [(8, 2), (4, 4), (16, 1)])
@pytest.mark.parametrize("new,start", [([3], [20]), ([40, 5], [100, 4000]), ([300], [50]), ([260, 1], [9000, 3])])
def test_values_that_are_not_finite(ws, hq, hkv, new, start):
    c = Cache(new, start, hq, hkv, seed=sum(new))
    for s, (m, st) in enumerate(zip(new, start)):
        n = st + m
        x = torch.zeros((hkv, D), dtype=torch.float16, device="cuda")
        put(c, s, n - 1, v=x + math.nan)        # the last token: of the rows before it none
        if m > 2:
            y = x.clone()
            y[0, 5], y[0, 77], y[-1, 100] = math.inf, -math.inf, math.nan
            put(c, s, n - 2, v=y)
            z = x.clone()
            z[0, 5], z[0, 6] = -math.inf, math.inf
            put(c, s, st + m // 2, v=z)
    check_not_finite(c, run(c, ws))


@pytest.mark.parametrize("new,start", [([5], [700]), ([2], [9000]), ([200], [500])])
def test_an_infinity_in_the_context(ws, new, start):
    c = Cache(new, start, 8, 2, seed=4)
    x = torch.ones((2, D), dtype=torch.float16, device="cuda")
    x[1, 3] = math.inf
    put(c, 0, 7, v=x)
    put(c, 0, start[0] // 2, v=-x)
    check_not_finite(c, run(c, ws))


@pytest.mark.parametrize("new,start", [([6], [40]), ([6], [9000]), ([150], [400])])
def test_keys_that_are_nan(ws, new, start):
    c = Cache(new, start, 8, 2, seed=5)
    x = torch.ones((2, D), dtype=torch.float16, device="cuda")
    x[1, 3] = math.nan
    put(c, 0, start[0] + new[0] // 2, k=x)
    check_not_finite(c, run(c, ws))


@pytest.mark.parametrize("new,start", [([6], [300]), ([4], [9000]), ([200], [300]), ([70], [5000])])
@pytest.mark.parametrize("spread", [3.0, 12.0, 60.0])
def test_scores_far_apart(ws, new, start, spread):
    """Standard deviations of the scores of 3 to 60 nats, rising along the row in one of the sequences."""
    c = Cache(new, start, 8, 2, seed=6, spread=spread)
    for pos in range(0, start[0] + new[0], 3):  # larger keys later
        page, slot = int(c.bt[0, pos // PS]), pos % PS
        c.k[page, slot] *= pos / (start[0] + new[0])
    want, bound = c.attend()
    ref.check(run(c, ws), want, bound)


@pytest.mark.parametrize("new,start", [([3], [3000]), ([140], [3000])])
def test_scores_beyond_fp32s_fractions(ws, new, start):
    """Scores of about 2^27 and more: equal ones share the weight, others have none."""
    c = Cache(new, start, 4, 1, seed=7)
    n = start[0] + new[0]
    c.scale = 1e6
    c.q[: c.tokens] = 0
    c.q[: c.tokens, :, 0] = 1000.0
    k = torch.zeros((n, 1, D), dtype=torch.float16, device="cuda")
    k[:, 0, 0] = torch.randint(-3, 2, (n,), generator=torch.Generator().manual_seed(1)).half().cuda()
    k[5, 0, 0] = 1.0
    for pos in range(n):
        put(c, 0, pos, k=k[pos])
    _, v = c.rows(0, n)
    got = run(c, ws)
    for i in range(0, new[0], max(1, new[0] // 7)):
        top = (k[: start[0] + i + 1, 0, 0] == 1.0)
        x = v[: start[0] + i + 1, 0][top].double()
        want, mag = x.mean(0), x.abs().mean(0)
        assert ((got[i].double() - want[None]).abs() <= 2.0 ** -10 * mag + 2.0 ** -11 * want.abs() + 2.0 ** -24).all()


@pytest.mark.parametrize("new", [[2], [100]])
def test_a_first_token_that_takes_most_of_the_weight(ws, new):
    c = Cache(new, [6000], 4, 1, seed=8)
    c.q[: c.tokens] = 0.25
    first = torch.full((1, D), 0.25 * 16 / (D * 0.0625) * math.sqrt(D), dtype=torch.float16, device="cuda")  # 16 nats above
    for pos in range(6000 + new[0]):
        put(c, 0, pos, k=torch.zeros_like(first))
    put(c, 0, 0, k=first, v=torch.zeros_like(first))
    got, (want, bound) = run(c, ws).double(), c.attend()
    # The weights beside the first token's are e^-16 of it, so the outputs are about 6000 e^-16 / (1 + 6000 e^-16) * 6000^-0.5 = 1e-5:
    # subnormal in fp16, whose values are 2^-24 apart there, which a rounding is off by up to half of (2^-25), whatever the value.
    assert (got - want).norm() < 5e-4 * want.norm() + 2.0 ** -25 * math.sqrt(want.numel())
    ref.check(got, want, bound + 2.0 ** -11 * want.abs())


def test_equal_scores_and_zero_scale(ws):
    c = Cache([9, 120], [500, 77], 8, 2, seed=9)
    c.scale = 0.0
    want, bound = c.attend()
    ref.check(run(c, ws), want, bound)


def test_pages_outside_the_pool_are_zeros(ws):
    for new, start in (([4, 3], [100, 9000]), ([150], [300])):
        c = Cache(new, start, 8, 2, seed=10)
        c.bt[0, 2] = -1
        c.bt[0, 4] = c.num_pages
        c.bt[-1, 5] = 2 ** 31 - 1
        want, bound = c.attend()
        ref.check(run(c, ws, status=pkv.PKV_STATUS_BAD_PAGE), want, bound)


def test_sequences_out_of_order_are_skipped(ws):
    c = Cache([5, 6, 7, 130], [10, 20, 30, 40], 8, 2, seed=11)
    want, bound = c.attend()
    good = run(c, ws)
    for change in ("start", "long", "cu"):
        st, cu, skip = c.st.clone(), c.cu.clone(), slice(5, 11)
        if change == "start":
            st[1] = -1
        elif change == "long":
            st[1] = c.bt.shape[1] * PS - 5
        else:
            cu[2] = 4  # ends before it begins; the sequence behind it begins earlier
            skip = slice(4, 18)
        out = torch.full((c.q.shape[0], 8, D), 7.0, dtype=torch.float16, device="cuda")
        pkv.chunk_attention(c.q, c.k, c.v, cu, c.bt, start=st, out=out, ws=ws)
        torch.cuda.synchronize()
        assert pkv.pkv_read_status(ws) & pkv.PKV_STATUS_BAD_LEN
        if change != "cu":
            assert (out[skip] == 7.0).all()
        assert torch.equal(out[: skip.start], good[: skip.start]) and torch.equal(out[skip.stop:c.tokens], good[skip.stop:])


@pytest.mark.parametrize("new", [[3], [300], [3, 4], [3, 300], [1] * 40])
def test_no_sequence_in_order(ws, new):
    c = Cache(new, [10] * len(new), 8, 2, seed=13)
    out = torch.full((c.q.shape[0], 8, D), 7.0, dtype=torch.float16, device="cuda")
    pkv.chunk_attention(c.q, c.k, c.v, c.cu, c.bt, start=torch.full_like(c.st, -1), out=out, ws=ws)
    torch.cuda.synchronize()
    assert pkv.pkv_read_status(ws) == pkv.PKV_STATUS_BAD_LEN and (out == 7.0).all()


def test_rows_of_no_sequence(ws):
    c = Cache([5, 140], [10, 20], 8, 2, seed=12)
    q = torch.cat((torch.full((9, 8, D), math.nan, dtype=torch.float16, device="cuda"), c.q))
    out = torch.full_like(q, 7.0)
    pkv.chunk_attention(q, c.k, c.v, c.cu + 9, c.bt, start=c.st, out=out, ws=ws)
    want, bound = c.attend()
    ref.check(out[9:9 + c.tokens], want, bound)
    assert (out[:9] == 7.0).all() and (out[9 + c.tokens:] == 7.0).all()


@pytest.mark.parametrize("sms", [1, 2, 7, 20, 151, 152])
def test_grids_of_any_size(sms):
    c = Cache([3, 90, 0, 1, 200], [2000, 100, 5, 700, 1500], 24, 12, seed=13)
    want, bound = c.attend()
    lib, n = pkv.load(), ctypes.c_size_t()
    assert lib.pkv_chunk_workspace_bytes(sms, ctypes.byref(n)) == 0
    ws = pkv.alloc_workspace(n.value)
    t = c.q.shape[0]
    pr = pkv.make_problem(5, 24, 12, D, PS, c.num_pages, c.bt.shape[1])
    pm = pkv.make_prompt(5, t, 24, 12, D)
    out = torch.full((t, 24, D), 7.0, dtype=torch.float16, device="cuda")
    q = c.q.contiguous()
    rc = lib.pkv_chunk_attention(ctypes.byref(pr), ctypes.byref(pm), q.data_ptr(), c.k.data_ptr(), c.v.data_ptr(), c.cu.data_ptr(),
                                 c.st.data_ptr(), c.bt.data_ptr(), ctypes.c_float(c.scale), sms, ws.data_ptr(), ws.numel(),
                                 out.data_ptr(), torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert rc == 0 and pkv.pkv_read_status(ws) == 0
    ref.check(out[: c.tokens], want, bound)


def test_one_captured_graph_serves_other_lengths(ws):
    a = Cache([4, 60, 1], [300, 20, 5000], 8, 2, seed=14)
    b = Cache([30, 5, 30], [2, 9000, 0], 8, 2, seed=15)
    c = Cache([4, 60, 1], [300, 20, 5000], 8, 2, seed=14)
    width, pool = max(a.bt.shape[1], b.bt.shape[1]), max(a.num_pages, b.num_pages)
    q, cu, st = a.q.clone(), a.cu.clone(), a.st.clone()
    k, v = (torch.zeros((pool, PS, 2, D), dtype=torch.float16, device="cuda") for _ in range(2))
    bt = torch.full((3, width), -1, dtype=torch.int32, device="cuda")
    out = torch.zeros((q.shape[0], 8, D), dtype=torch.float16, device="cuda")
    pkv.chunk_attention(q, k, v, cu, bt, start=st, out=out, ws=ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pkv.chunk_attention(q, k, v, cu, bt, start=st, out=out, ws=ws)
    torch.cuda.synchronize()
    pkv.pkv_read_status(ws)
    for x in (a, b, c):
        assert x.q.shape == q.shape
        q.copy_(x.q), cu.copy_(x.cu), st.copy_(x.st)
        k[: x.num_pages], v[: x.num_pages] = x.k, x.v
        bt.fill_(-1)
        bt[:, : x.bt.shape[1]] = x.bt
        g.replay()
        torch.cuda.synchronize()
        assert pkv.pkv_read_status(ws) == 0
        want, bound = x.attend()
        ref.check(out[: x.tokens], want, bound)


def test_other_streams_and_no_workspace(ws):
    c = Cache([7, 100], [3000, 11], 8, 2, seed=16)
    want, bound = c.attend()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = [pkv.chunk_attention(c.q, c.k, c.v, c.cu, c.bt, start=c.st, stream=side) for _ in range(3)]
    outs.append(pkv.chunk_attention(c.q, c.k, c.v, c.cu, c.bt, start=c.st))
    with torch.cuda.stream(side):
        outs.append(pkv.chunk_attention(c.q, c.k, c.v, c.cu, c.bt, start=c.st))
    torch.cuda.synchronize()
    for y in outs:
        ref.check(y[: c.tokens], want, bound)


def test_two_graphs_on_one_workspace(ws):
    a, b = Cache([5], [8000], 8, 2, seed=17), Cache([150], [900], 16, 1, seed=18)
    outs, graphs = [], []
    for c in (a, b):
        out = torch.zeros((c.q.shape[0], c.hq, D), dtype=torch.float16, device="cuda")
        pkv.chunk_attention(c.q, c.k, c.v, c.cu, c.bt, start=c.st, out=out, ws=ws)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pkv.chunk_attention(c.q, c.k, c.v, c.cu, c.bt, start=c.st, out=out, ws=ws)
        outs.append(out), graphs.append(g)
    for i in (0, 1, 1, 0, 1, 0):
        outs[i].zero_()
        graphs[i].replay()
        want, bound = (a, b)[i].attend()
        ref.check(outs[i][: (a, b)[i].tokens], want, bound)


def test_pages_beyond_4_gb(ws):
    """Page numbers whose offsets need more than 32 bits, in elements and in bytes."""
    c = Cache([3, 70], [200, 40], 4, 1, seed=19)
    pool = (1 << 20) + 70000  # 4 KB a page: beyond 2^31 elements
    k, v = (torch.empty((pool, PS, 1, D), dtype=torch.float16, device="cuda") for _ in range(2))
    far = torch.tensor([pool - 1 - 37 * i for i in range(c.num_pages)], device="cuda")
    k[far], v[far] = c.k, c.v
    good = (c.bt >= 0) & (c.bt < c.num_pages)
    bt = torch.where(good, far[c.bt.clamp(0, c.num_pages - 1).long()].int(), c.bt)
    out = pkv.chunk_attention(c.q, k, v, c.cu, bt, start=c.st, ws=ws)
    want, bound = c.attend()
    torch.cuda.synchronize()
    assert pkv.pkv_read_status(ws) == 0
    ref.check(out[: c.tokens], want, bound)


def test_rows_that_share_a_prefix(ws):
    c = Cache([4, 90], [320, 320], 8, 2, seed=20)
    c.bt[1, :20] = c.bt[0, :20]
    want, bound = c.attend()
    ref.check(run(c, ws), want, bound)


def test_nothing_to_do(ws):
    c = Cache([0, 0], [5, 9], 8, 2, seed=21)
    assert (run(c, ws) == 7.0).all()
    empty = pkv.chunk_attention(c.q[:0], c.k, c.v, c.cu, c.bt, start=c.st, ws=ws)
    assert empty.shape == (0, 8, D)


def test_a_serving_loop(ws):
    """Tables, K and V, bounds, attention of chunks, selection and sparse steps together, against one growing cache."""
    hq, hkv, width, pool, b = 8, 2, 40, 120, 3
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(22)
    bt = torch.full((b, width), -1, dtype=torch.int32, device=dev)
    lens = torch.zeros(b, dtype=torch.int32, device=dev)
    free = torch.randperm(pool, generator=g, device=dev).int()
    count = torch.tensor([pool], dtype=torch.int32, device=dev)
    kp, vp = (torch.full((pool, PS, hkv, D), math.nan, dtype=torch.float16, device=dev) for _ in range(2))
    bounds = torch.full((pool, hkv, 2, D), math.nan, dtype=torch.float16, device=dev)
    held = [[torch.zeros((0, hkv, D), dtype=torch.float16, device=dev)] * 2 for _ in range(b)]
    for new in ([40, 7, 0], [3, 200, 90], [1, 1, 1], [0, 65, 1], [1, 1, 1]):
        t = sum(new)
        q = torch.randn((t, hq, D), generator=g, device=dev).half()
        k, v = (torch.randn((t, hkv, D), generator=g, device=dev).half() for _ in range(2))
        cu, start = pkv.tables_grow(torch.tensor(new, dtype=torch.int32, device=dev), lens, bt, free, count)
        pkv.prompt_append(k, v, cu, kp, vp, bt, start=start)
        pkv.page_bounds(kp, cu, bt, bounds, start=start)
        out = pkv.chunk_attention(q, kp, vp, cu, bt, start=start, ws=ws)
        at = 0
        for s, m in enumerate(new):
            held[s] = [torch.cat((x, y[at:at + m])) for x, y in zip(held[s], (k, v))]
            n = held[s][0].shape[0]
            if m:
                want, mag = ref.attend(q[at:at + m], *held[s], 1 / math.sqrt(D), n - m)
                ref.check(out[at:at + m], want, ref.prompt_bound(want, mag, n, q[at:at + m], *held[s], 1 / math.sqrt(D)) + 2.0 ** -14 * mag)
            at += m
        assert lens.tolist() == [h[0].shape[0] for h in held]
        q1 = torch.randn((b, hq, D), generator=g, device=dev).half()
        pages = pkv.select_pages(q1, bounds, bt, lens, 4)
        sparse = pkv.sparse_decode(q1, kp, vp, bt, lens, pages)
        for s in range(b):
            n = held[s][0].shape[0]
            for h in range(hkv):
                rows = [p * PS + i for p in pages[s, h].tolist() if p >= 0 for i in range(PS) if p * PS + i < n]
                if not rows:
                    continue
                kk, vv, qq = held[s][0][rows, h:h + 1], held[s][1][rows, h:h + 1], q1[s:s + 1, 4 * h:4 * h + 4]
                want, mag = ref.attend(qq, kk, vv, 1 / math.sqrt(D), len(rows) - 1)
                ref.check(sparse[s:s + 1, 4 * h:4 * h + 4], want, ref.prompt_bound(want, mag, len(rows), qq, kk, vv, 1 / math.sqrt(D)))
    pkv.tables_release(torch.tensor([1, 0, 1], dtype=torch.int32, device=dev), lens, bt, free, count)
    assert lens.tolist() == [0, held[1][0].shape[0], 0]
    assert sorted(free[: int(count)].tolist() + bt[1, : -(-int(lens[1]) // PS)].tolist()) == list(range(pool))
