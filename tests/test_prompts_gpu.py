"""The prompt and 4-bit-cache operators on the GPU against plain 64-bit forms (tests/prompt_reference.py)."""

import math

import pytest
import torch

import prompt_reference as ref
import serving_paged_gqa_gb300 as pkv

pytestmark = pytest.mark.gpu

D, PS = 128, 16
SCALE = 1.0 / math.sqrt(D)
HEADS = [(32, 8), (3, 3), (8, 4), (32, 4), (16, 1)]  # G = 4, 1, 2, 8, 16


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__

    __graft_entry__.build()
    torch.cuda.set_device(0)


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda").half()


def cu_of(lens, first=0):
    at = [first]
    for n in lens:
        at.append(at[-1] + n)
    return torch.tensor(at, dtype=torch.int32, device="cuda")


def packed(g, lens, hq, hkv, before=0, behind=0, fused=True):
    """q, k, v of packed sequences with rows that belong to none of them before and behind (NaN), and cu_seqlens."""
    t = before + sum(lens) + behind
    if fused:
        x = normal(g, t, hq + 2 * hkv, D)
        q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    else:
        q, k, v = normal(g, t, hq, D), normal(g, t, hkv, D), normal(g, t, hkv, D)
    for y in (q, k, v):
        y[:before] = math.nan
        y[before + sum(lens):] = math.nan
    return q, k, v, cu_of(lens, before)


def status(ws):
    torch.cuda.synchronize()
    return pkv.pkv_read_status(ws)


def new_ws(n=pkv.PKV_PROMPT_WS_BYTES):
    return pkv.alloc_workspace(n)


def check_prompt(q, k, v, cu, got, scale=SCALE, seqs=None, what=""):
    at = cu.tolist()
    for s in range(len(at) - 1) if seqs is None else seqs:
        a, b = at[s], at[s + 1]
        for i in range(a, b, 2048):
            e = min(b, i + 2048)
            out, mag = ref.attend(q[i:e], k[a:e], v[a:e], scale, i - a)
            bound = ref.prompt_bound(out, mag, e - a, q[i:e], k[a:e], v[a:e], scale)
            ref.check(got[i:e], out, bound, f"{what} sequence {s} rows {i - a}..")


# --------------------------------------------------------------------------------------------------- prompt attention
@pytest.mark.parametrize("hq,hkv", HEADS)
@pytest.mark.parametrize("lens", [[1], [17], [64, 0, 1, 130], [128], [5, 33, 129, 127, 16, 0], [300, 257]], ids=str)
def test_prompt_lengths_and_heads(lens, hq, hkv):
    g = gen(len(lens) * 100 + hq)
    q, k, v, cu = packed(g, lens, hq, hkv, before=3, behind=5, fused=hq != 8)
    out = torch.full((q.shape[0], hq, D), 7.0, dtype=torch.float16, device="cuda")
    ws = new_ws()
    for call in range(2):
        got = pkv.prompt_attention(q, k, v, cu, out=out, ws=ws)
        assert got is out and status(ws) == 0
        check_prompt(q, k, v, cu, out, what=f"call {call}")
        assert (out[:3] == 7).all() and (out[3 + sum(lens):] == 7).all()  # rows of no sequence are left as they were


@pytest.mark.parametrize("lens", [[4096], [1025, 2000, 513], [3000, 7, 3000]], ids=str)
def test_prompt_longer(lens):
    q, k, v, cu = packed(gen(5), lens, 8, 2)
    ws = new_ws()
    out = pkv.prompt_attention(q, k, v, cu, ws=ws)
    assert status(ws) == 0
    check_prompt(q, k, v, cu, out)


def test_prompt_of_a_long_sequence():
    lens = [12345]
    q, k, v, cu = packed(gen(6), lens, 4, 1, fused=False)
    ws = new_ws()
    out = pkv.prompt_attention(q, k, v, cu, ws=ws)
    assert status(ws) == 0
    for a in (0, 6000, 12345 - 130):  # rows in the beginning, the middle and the end
        w, mag = ref.attend(q[a:a + 130], k[:a + 130], v[:a + 130], SCALE, a)
        ref.check(out[a:a + 130], w, ref.prompt_bound(w, mag, a + 130, q, k, v, SCALE), f"rows {a}..")


@pytest.mark.parametrize("n", [300, 4096])
def test_prompt_of_many_short_sequences(n):
    lens = [(i * 7) % 4 for i in range(n)]  # 0 to 3 tokens, up to the largest number of sequences
    q, k, v, cu = packed(gen(7), lens, 8, 2)
    ws = new_ws()
    out = pkv.prompt_attention(q, k, v, cu, ws=ws)
    assert status(ws) == 0
    check_prompt(q, k, v, cu, out, seqs=list(range(0, 40)) + list(range(n - 40, n)))


@pytest.mark.parametrize("factor,scale", [(1.0, 0.0), (6.0, SCALE), (1.0, 3.0), (0.01, SCALE)])
def test_prompt_flat_and_sharp_softmax(factor, scale):
    q, k, v, cu = packed(gen(8), [200, 140], 8, 2)
    q = (q.float() * factor).half()
    ws = new_ws()
    out = pkv.prompt_attention(q, k, v, cu, scale=scale, ws=ws)
    assert status(ws) == 0
    check_prompt(q, k, v, cu, out, scale=scale)


@pytest.mark.parametrize("step", [0.02, 0.2, 1.0])
@pytest.mark.parametrize("shape", ["up", "down", "second half", "saw"])
def test_prompt_scores_that_grow_along_the_keys(step, shape):
    """Scores whose maximum moves by up to 1.4 in log2 from key to key, so that the running reference is raised in
    every step, in a step's first or second 64 keys, by some rows only, or never after the first."""
    n, g = 700, gen(77)
    q, k, v, cu = packed(g, [n], 8, 2)
    at = torch.arange(n, device="cuda", dtype=torch.float32)
    along = {"up": at, "down": -at, "second half": torch.where(at % 128 >= 64, at, at * 0), "saw": (at * 37) % 300}[shape]
    unit = torch.zeros(D, device="cuda")
    unit[5] = 8.0
    k = (k.float() * 0.1 + (along * step * math.sqrt(D) / 8.0)[:, None, None] * (unit / 8.0)).half()
    turn = torch.tensor([1.0, 1.0, 0.5, 0.0], device="cuda").repeat(2)  # rows of one tile that grow at different rates
    q = (q.float() * 0.1 + turn[None, :, None] * unit).half()
    ws = new_ws()
    out = pkv.prompt_attention(q, k, v, cu, ws=ws)
    assert status(ws) == 0
    check_prompt(q, k, v, cu, out)


@pytest.mark.parametrize("rise", [15.5, 20.0, 23.9, 25.0, 26.5, 29.0])
@pytest.mark.parametrize("first,second", [(130, 200), (200, 130), (150, 255), (70, 10)])
def test_prompt_a_step_whose_halves_rise_differently(rise, first, second):
    """Key `first` raises the running reference by `rise` (in log2), while key `second` of the same step's other half stays
    just below the 2^15 that lets its weight as it is; its V is large enough to be seen."""
    n, g = 300, gen(98)
    q, k, v, cu = packed(g, [n], 8, 1, fused=False)
    unit = 1.0 / (8.0 * SCALE * math.log2(math.e))  # of k's dim 0, for a score of 1 in log2
    q.zero_()
    k.zero_()
    q[:, :, 0] = 8.0
    k[first, :, 0], k[second, :, 0] = rise * unit, 14.9 * unit
    v[second] *= 2.0 ** max(0.0, rise - 14.9)
    ws = new_ws()
    out = pkv.prompt_attention(q, k, v, cu, ws=ws)
    assert status(ws) == 0
    check_prompt(q, k, v, cu, out)


def one_hot_levels(g, order, sign, n):
    """Levels between 16384 and 2^15 in steps of 64 (exact in fp16), and for each row the key of the greatest up to it."""
    at = torch.randperm(n, generator=g, device="cuda") if order == "random" else torch.arange(n, device="cuda")
    level = sign * (16384 + 64 * (at if order != "down" else n - 1 - at)).double()
    return level, torch.tensor([int(level[:i + 1].argmax()) for i in range(n)], device="cuda")


@pytest.mark.parametrize("size", [512.0, 4096.0, 32768.0])
@pytest.mark.parametrize("order,sign", [("up", 1), ("down", 1), ("random", 1), ("random", -1)])
def test_prompt_scores_of_which_fp32_has_no_fractions(size, order, sign):
    """Scores from 2^24 to 2^30 (in log2), exact in fp32 and thousands apart: all weights but the greatest key's are 0,
    and the output is its V (one rounding of the weight, one of the output)."""
    n, g = 250, gen(93)
    q, k, v, cu = packed(g, [n], 8, 2, fused=False)
    level, best = one_hot_levels(g, order, sign, n)
    q.zero_()
    q[:, :, 3:19] = size
    k.zero_()
    k[:, :, 3:19] = level.half()[:, None, None]
    ws = new_ws()
    out = pkv.prompt_attention(q, k, v, cu, ws=ws)
    assert status(ws) == 0
    want = v[best].repeat_interleave(4, 1).double()
    ref.check(out, want, (2 * ref.HALF_STEP + 2.0 ** -16) * want.abs() + ref.TINY)


def test_prompt_values_of_the_largest_magnitude():
    """All V at fp16's largest value, and weights that fp16 rounds up by most of half a step (2^-0.99922 = 0.50027 next to
    the first key's 1): the mean is that value, which a rounding of the numerator alone carries to infinity."""
    n, g = 200, gen(94)
    q, k, v, cu = packed(g, [n], 8, 2, fused=False)
    q.zero_()
    k.zero_()
    q[:, :, 0] = 1.0
    k[0, :, 0] = 7.8359375
    v.fill_(65504.0)
    v[:, :, 64:] = -65504.0
    for scale in (SCALE, 2 * SCALE, -0.0):
        ws = new_ws()
        out = pkv.prompt_attention(q, k, v, cu, scale=scale, ws=ws)
        assert status(ws) == 0
        # the row's rounding to fp16 steps of 32, and a step for the weights' rounding
        assert ((out.double() - v.double().repeat_interleave(4, 1)).abs() <= 65504 * 2.0 ** -10).all()


def test_prompt_infinities_of_values_add_up():
    """V's infinities reach every later row of their dim, however small their weights in fp16 are, and meet as a NaN; the
    rows' other dims and the rows before are as they are without them."""
    n, g = 400, gen(95)
    q, k, v, cu = packed(g, [n], 8, 2)
    k[300:] += 3.0 * (q[300:, :1] > 0)  # sharper towards the end
    vb = v.clone()
    vb[5, 0, 10], vb[130, 0, 10] = math.inf, -math.inf
    vb[131, 1, 70], vb[390, 1, 70] = -math.inf, -math.inf
    vb[256, 0, 127] = math.nan
    ws = new_ws()
    out = pkv.prompt_attention(q, k, vb, cu, ws=ws)
    assert status(ws) == 0
    w, mag = ref.attend(q, k, v, SCALE, 0)
    bound = ref.prompt_bound(w, mag, n, q, k, v, SCALE)
    want = w.clone()
    want[5:130, :4, 10], want[130:, :4, 10] = math.inf, math.nan
    want[131:, 4:, 70] = -math.inf
    want[256:, :4, 127] = math.nan
    fin = torch.isfinite(want)
    assert torch.equal(torch.isnan(out), torch.isnan(want))
    assert (out.double()[torch.isinf(want)] == want[torch.isinf(want)]).all()
    ref.check(torch.where(fin, out.double(), 0.0), torch.where(fin, want, 0.0), bound)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("which", ["k", "v", "kv"])
def test_prompt_masked_tokens_never_reach_a_row(bad, which):
    """An infinity or a NaN in a token reaches its own row and later ones of its sequence at most: earlier rows and
    other sequences are as they are without it."""
    lens = [70, 150, 40]
    q, k, v, cu = packed(gen(9), lens, 8, 2)
    hit = 70 + 75
    kb, vb = k.clone(), v.clone()
    if "k" in which:
        kb[hit] = bad
    if "v" in which:
        vb[hit] = bad
    ws = new_ws()
    out = pkv.prompt_attention(q, kb, vb, cu, ws=ws)
    assert status(ws) == 0
    check_prompt(q, k, v, cu, out, seqs=[0, 2])
    w, mag = ref.attend(q[70:hit], k[70:hit], v[70:hit], SCALE, 0)
    ref.check(out[70:hit], w, ref.prompt_bound(w, mag, 80, q[70:hit], k[70:hit], v[70:hit], SCALE), "rows before")
    want = ref.attend(q[hit:220], kb[70:220], vb[70:220], SCALE, 75)[0]
    got = out[hit:220].double()
    assert (torch.isnan(got) == torch.isnan(want)).all()
    assert (got[torch.isinf(want)] == want[torch.isinf(want)]).all()


def test_prompt_rows_of_no_sequence_may_hold_anything():
    """Packed rows behind and between the sequences: infinities and NaN there reach nothing (a tile's keys run past its
    sequence's end), and a NaN in a whole sequence's V leaves its neighbours as they are."""
    g = gen(91)
    lens, gap = [300, 1000, 5], 40
    at, rows = [], 0
    for n in lens:
        at.append((rows, rows + n))
        rows += n + gap
    x = normal(g, rows, 12, D)
    q, k, v = x[:, :8], x[:, 8:10], x[:, 10:]
    keep = torch.zeros(rows, dtype=torch.bool, device="cuda")
    for a, b in at:
        keep[a:b] = True
    x[~keep] = math.inf
    v[at[1][0]:at[1][1]] = math.nan
    # the gaps are sequences of their own for cu_seqlens, whose rows are not looked at
    cu = ints([y for pair in at for y in pair] + [rows])
    ws = new_ws()
    out = pkv.prompt_attention(q, k, v, cu, ws=ws)
    assert status(ws) == 0
    for a, b in (at[0], at[2]):
        w, mag = ref.attend(q[a:b], k[a:b], v[a:b], SCALE, 0)
        ref.check(out[a:b], w, ref.prompt_bound(w, mag, b - a, q[a:b], k[a:b], v[a:b], SCALE), "beside a sequence of NaN")
    assert torch.isnan(out[at[1][0]:at[1][1]]).all()


@pytest.mark.parametrize("num_sms", [1, 3, 1000])
def test_grids_of_any_size(num_sms):
    """The SM count sets the grids alone: results are right for one CTA that does everything and for more than fit."""
    g = gen(92)
    q, k, v, cu = packed(g, [333, 20, 129], 8, 2, fused=False)
    out = torch.full_like(q, math.nan)
    ws = new_ws()
    lib, p = pkv.load(), pkv.make_prompt(3, 482, 8, 2, D)
    stream = torch.cuda.current_stream().cuda_stream
    assert lib.pkv_prompt_attention(p, q.data_ptr(), k.data_ptr(), v.data_ptr(), cu.data_ptr(), SCALE, num_sms, ws.data_ptr(), 256,
                                    out.data_ptr(), stream) == 0
    assert status(ws) == 0
    check_prompt(q, k, v, cu, out)
    lens = [333, 20, 129]
    bt, pages = table(g, lens)
    pool = torch.zeros((pages, 2, ref.BLOCK), dtype=torch.uint8, device="cuda")
    want = pool.clone()
    for b in range(3):
        ref.put_tokens(want, bt[b], torch.arange(lens[b], device="cuda"), k[cu[b]:cu[b + 1]], v[cu[b]:cu[b + 1]])
    pr = pkv.make_problem(3, 8, 2, D, PS, pages, bt.shape[1])
    assert lib.pkv_q4_prompt_append(pr, p, k.data_ptr(), v.data_ptr(), cu.data_ptr(), None, pool.data_ptr(), bt.data_ptr(), num_sms,
                                    ws.data_ptr(), 256, stream) == 0
    assert status(ws) == 0 and torch.equal(pool, want)
    qd, n = normal(g, 3, 8, D), ints(lens)
    for call in range(2):
        out = torch.full_like(qd, math.nan)
        wd = new_ws(pkv.pkv_q4_workspace_bytes(pr, num_sms))
        assert lib.pkv_q4_decode_step(pr, qd.data_ptr(), pool.data_ptr(), bt.data_ptr(), n.data_ptr(), SCALE, num_sms, wd.data_ptr(),
                                      wd.numel(), out.data_ptr(), stream) == 0
        assert status(wd) == 0
        check_q4(qd, pool, bt, lens, out)


def test_prompt_query_of_nan_reaches_its_own_row_alone():
    q, k, v, cu = packed(gen(10), [90], 8, 2)
    qb = q.clone()
    qb[41, 3] = math.nan
    out = pkv.prompt_attention(qb, k, v, cu)
    torch.cuda.synchronize()
    assert torch.isnan(out[41, 3]).all()
    out[41, 3] = pkv.prompt_attention(q, k, v, cu)[41, 3]
    check_prompt(q, k, v, cu, out)


def test_prompt_bad_bounds_are_reported_and_skipped():
    q, k, v, _ = packed(gen(11), [100], 8, 2, fused=False)
    for bounds, good in (([0, 40, 20, 100], [(0, 40), (20, 100)]), ([-5, 30, 100], [(30, 100)]), ([0, 30, 101], [(0, 30)]),
                         ([0, 2 ** 31 - 1, 50], [])):
        cu = torch.tensor(bounds, dtype=torch.int32, device="cuda")
        out = torch.full((100, 8, D), 7.0, dtype=torch.float16, device="cuda")
        ws = new_ws()
        pkv.prompt_attention(q, k, v, cu, out=out, ws=ws)
        assert status(ws) == pkv.PKV_STATUS_BAD_LEN, bounds
        for a, b in good:
            w, mag = ref.attend(q[a:b], k[a:b], v[a:b], SCALE, 0)
            if bounds != [0, 40, 20, 100]:  # its two good sequences write the rows 20..39 both
                ref.check(out[a:b], w, ref.prompt_bound(w, mag, b - a, q, k, v, SCALE), str(bounds))


def test_prompt_on_another_stream_and_captured():
    q, k, v, cu = packed(gen(12), [130, 61], 32, 8)
    ws = new_ws()
    out = torch.empty((191, 32, D), dtype=torch.float16, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    pkv.prompt_attention(q, k, v, cu, out=out, ws=ws, stream=side)
    made = pkv.prompt_attention(q, k, v, cu, stream=side)  # output and workspace made by the call
    side.synchronize()
    check_prompt(q, k, v, cu, out)
    assert torch.equal(made, out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pkv.prompt_attention(q, k, v, cu, out=out, ws=ws)
    for i in range(3):  # replayed with other contents and other lengths
        q.copy_(normal(gen(20 + i), *q.shape))
        cu.copy_(cu_of([[100, 91], [191, 0], [1, 189]][i]))
        g.replay()
        torch.cuda.synchronize()
        check_prompt(q, k, v, cu, out)
    assert status(ws) == 0


def test_prompt_results_do_not_depend_on_the_order_of_work():
    q, k, v, cu = packed(gen(13), [700, 20, 345], 16, 4)
    a = pkv.prompt_attention(q, k, v, cu)
    for _ in range(3):
        assert torch.equal(a, pkv.prompt_attention(q, k, v, cu))


# ------------------------------------------------------------------------------------------------------------- pages
def table(g, lens, extra=3, more_cols=0):
    n = [(x + PS - 1) // PS for x in lens]
    total = sum(n)
    perm = torch.randperm(total + extra, generator=g, device="cuda").to(torch.int32)
    bt = torch.full((len(lens), max(max(n), 1) + more_cols), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, c in enumerate(n):
        bt[b, :c] = perm[at:at + c]
        at += c
    return bt, total + extra


@pytest.mark.parametrize("starts", [None, 0, 5])
@pytest.mark.parametrize("lens,hkv", [([1], 8), ([16], 1), ([40, 0, 3, 100], 3), ([257, 31], 8)], ids=str)
def test_appends_write_their_slots_and_no_others(lens, hkv, starts):
    g = gen(30)
    start = None if starts is None else torch.tensor([starts * (b + 1) for b in range(len(lens))], dtype=torch.int32, device="cuda")
    has = [0] * len(lens) if start is None else start.tolist()
    q, k, v, cu = packed(g, lens, hkv, hkv, before=2, behind=2)
    bt, pages = table(g, [n + h for n, h in zip(lens, has)], more_cols=2)
    ws = new_ws()
    kp, vp = normal(g, pages, PS, hkv, D), normal(g, pages, PS, hkv, D)
    pool = torch.randint(0, 256, (pages, hkv, ref.BLOCK), dtype=torch.uint8, device="cuda", generator=g)
    want_k, want_v, want = kp.clone(), vp.clone(), pool.clone()
    at = cu.tolist()
    for b, n in enumerate(lens):
        if n == 0:
            continue
        pos = torch.arange(n, device="cuda") + has[b]
        page = bt[b][pos // PS].long()
        want_k[page, pos % PS] = k[at[b]:at[b + 1]]
        want_v[page, pos % PS] = v[at[b]:at[b + 1]]
        ref.put_tokens(want, bt[b], pos, k[at[b]:at[b + 1]], v[at[b]:at[b + 1]])
    pkv.prompt_append(k, v, cu, kp, vp, bt, start=start, ws=ws)
    pkv.q4_prompt_append(k, v, cu, pool, bt, start=start, ws=ws)
    assert status(ws) == 0
    assert torch.equal(kp, want_k) and torch.equal(vp, want_v)
    assert torch.equal(pool, want)
    k_out = torch.full((q.shape[0], hkv, D), 7.0, dtype=torch.float16, device="cuda")
    v_out = torch.full((q.shape[0], hkv + 1, D), 7.0, dtype=torch.float16, device="cuda")[:, :hkv]  # strided rows
    pkv.q4_read(cu, pool, bt, start=start, k_out=k_out, v_out=v_out, ws=ws)
    assert status(ws) == 0
    lo, hi = at[0], at[-1]
    for x, y in ((k, k_out), (v, v_out)):
        # code * scale in fp32 is exact (15 bits); the sum is rounded to fp32 and to fp16
        w = ref.values(*ref.quantise(x[lo:hi]))
        ref.check(y[lo:hi], w, ref.HALF_STEP * w.abs() + 2.0 ** -23 * w.abs() + ref.TINY, "read")
        assert (y[:lo] == 7).all() and (y[hi:] == 7).all()


@pytest.mark.parametrize("make", ["equal", "tiny", "huge", "mixed", "nan", "inf"])
def test_q4_quantises_every_kind_of_group(make):
    g = gen(31)
    x = normal(g, 35, 2, D)
    if make == "equal":
        x[:] = -0.75
    elif make == "tiny":  # subnormal scales
        x = (x.float() * 2.0 ** -20).half()
    elif make == "huge":  # the difference is beyond fp16
        x = torch.where(x > 0, 65504.0, -65504.0).half()
    elif make == "mixed":
        x[:, :, 0] = 60000.0
    elif make == "nan":
        x[3, 1, 70] = math.nan
    else:
        x[3, 1, 7], x[9, 0, 100] = math.inf, -math.inf
    bt, pages = table(g, [35])
    pool = torch.zeros((pages, 2, ref.BLOCK), dtype=torch.uint8, device="cuda")
    want = pool.clone()
    ref.put_tokens(want, bt[0], torch.arange(35, device="cuda"), x, x.flip(0))
    cu = cu_of([35])
    pkv.q4_prompt_append(x, x.flip(0), cu, pool, bt)
    k, _ = pkv.q4_read(cu, pool, bt, total_tokens=35)
    torch.cuda.synchronize()
    w = ref.values(*ref.quantise(x))
    assert torch.equal(torch.isnan(k), torch.isnan(w))
    w = torch.nan_to_num(w)
    ref.check(torch.nan_to_num(k), w, ref.HALF_STEP * w.abs() * 1.01 + ref.TINY)
    if make not in ("nan", "inf"):  # a NaN has more than one bit pattern
        assert torch.equal(pool, want)


def test_q4_writers_agree_on_every_byte():
    """A token has one 4-bit form, whether the prompt append or a decode step writes it: also with infinities and NaN, whose
    groups have codes 0."""
    g = gen(99)
    x = normal(g, 6, 2, 3, D)  # [token, K or V, head, d]
    x[1, 0, 0, 5], x[1, 1, 2, 127] = math.nan, math.inf
    x[2, :, :, :64] = -math.inf
    x[3, 0, 1] = 0.0
    x[4, 0, 1, ::2], x[4, 0, 1, 1::2] = 0.0, -0.0
    x[5] *= 1e-6
    bt = torch.arange(6, dtype=torch.int32, device="cuda").view(6, 1)
    one = torch.zeros((6, 3, ref.BLOCK), dtype=torch.uint8, device="cuda")
    two = one.clone()
    ws = new_ws()
    pkv.q4_prompt_append(x[:, 0].contiguous(), x[:, 1].contiguous(), cu_of([1] * 6), one, bt, ws=ws)
    q = normal(g, 6, 12, D)
    wd = q4_ws(q, two, bt)
    pkv.q4_decode(q, two, bt, ints([1] * 6), x[:, 0].contiguous(), x[:, 1].contiguous(), ws=wd)
    assert status(ws) == 0 and status(wd) == 0
    assert torch.equal(one, two)
    (kc, ks, _), (vc, vs, _) = ref.get_tokens(one, bt[1], torch.tensor([0], device="cuda"))
    assert torch.isnan(ks[0, 0, 0]) and (kc[0, 0, :64] == 0).all()
    assert torch.isnan(vs[0, 2, 1]) and (vc[0, 2, 64:] == 0).all()


def test_appends_report_bad_pages_and_lengths():
    g = gen(32)
    _, k, v, cu = packed(g, [40, 20], 2, 2)
    bt, pages = table(g, [40, 20])
    good = bt.clone()
    for name in ("page", "negative", "grow", "start"):
        bt = good.clone()
        start = torch.zeros(2, dtype=torch.int32, device="cuda")
        if name == "page":
            bt[0, 1] = pages
        elif name == "negative":
            bt[0, 1] = -1
        elif name == "grow":
            start[0] = 9  # 49 tokens in 3 pages
        else:
            start[0] = -1
        want_status = pkv.PKV_STATUS_BAD_PAGE if name in ("page", "negative") else pkv.PKV_STATUS_BAD_LEN
        kp = torch.zeros((pages, PS, 2, D), dtype=torch.float16, device="cuda")
        vp = torch.zeros_like(kp)
        pool = torch.zeros((pages, 2, ref.BLOCK), dtype=torch.uint8, device="cuda")
        want_k, want = kp.clone(), pool.clone()
        keep = []
        if want_status == pkv.PKV_STATUS_BAD_PAGE:
            keep = [(0, torch.tensor([i for i in range(40) if i // PS != 1], device="cuda"))]
        keep.append((1, torch.arange(20, device="cuda")))
        for b, pos in keep:
            rows = pos + 40 * b
            want_k[good[b][pos // PS].long(), pos % PS] = k[rows]
            ref.put_tokens(want, good[b], pos, k[rows], v[rows])
        k_out = torch.full((60, 2, D), 7.0, dtype=torch.float16, device="cuda")
        v_out = k_out.clone()
        for call in ("append", "q4", "read"):
            ws = new_ws()
            if call == "append":
                pkv.prompt_append(k, v, cu, kp, vp, bt, start=start, ws=ws)
            elif call == "q4":
                pkv.q4_prompt_append(k, v, cu, pool, bt, start=start, ws=ws)
            else:
                pkv.q4_read(cu, pool, bt, start=start, k_out=k_out, v_out=v_out, ws=ws)
            assert status(ws) == want_status, (name, call)
        assert torch.equal(kp, want_k) and torch.equal(pool, want), name
        skipped = slice(16, 32) if want_status == pkv.PKV_STATUS_BAD_PAGE else slice(0, 40)
        assert (k_out[skipped] == 7).all() and (v_out[skipped] == 7).all()
        assert (k_out[40:] != 7).any()


# -------------------------------------------------------------------------------------------------------- 4-bit decode
def q4_cache(g, lens, hkv, kscale=1.0, vscale=1.0, extra=3):
    """A 4-bit pool whose rows hold random tokens; slots behind a row's end and unused pages hold NaN parameters."""
    bt, pages = table(g, lens, extra)
    pool = torch.full((pages, hkv, ref.BLOCK), 0xFF, dtype=torch.uint8, device="cuda")
    for b, n in enumerate(lens):
        if n:
            k = (torch.randn((n, hkv, D), generator=g, device="cuda") * kscale).half()
            v = (torch.randn((n, hkv, D), generator=g, device="cuda") * vscale).half()
            ref.put_tokens(pool, bt[b], torch.arange(n, device="cuda"), k, v)
    return bt, pool


def q4_ws(q, pool, bt):
    return new_ws(pkv.pkv_q4_workspace_bytes(pkv.q4_problem(q, pool, bt)))


def check_q4(q, pool, bt, lens, out, scale=SCALE, rows=None, what=""):
    for b in range(len(lens)) if rows is None else rows:
        w, bound = ref.q4_row(q[b], pool, bt[b], lens[b], scale)
        ref.check(out[b], w, bound, f"{what} row {b} of {lens[b]} tokens")


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("hq,hkv", HEADS + [(32, 2), (12, 12)])
@pytest.mark.parametrize("lens", [[1], [16], [17, 0, 64], [63, 65, 1, 128, 0, 129], [1000, 3], [4097]], ids=str)
def test_q4_decode_lengths_and_heads(lens, hq, hkv):
    g = gen(40 + hq + len(lens))
    bt, pool = q4_cache(g, lens, hkv)
    q = normal(g, len(lens), hq, D)
    ws = q4_ws(q, pool, bt)
    before = pool.clone()
    for call in range(2):
        out = torch.full_like(q, math.nan)
        pkv.q4_decode(q, pool, bt, ints(lens), out=out, ws=ws)
        assert status(ws) == 0
        check_q4(q, pool, bt, lens, out, what=f"call {call}")
    assert torch.equal(pool, before)


@pytest.mark.parametrize("kscale,vscale,scale", [(1.0, 1e-3, SCALE), (1.0, 3e-6, SCALE), (1.0, 8000.0, SCALE), (100.0, 1.0, SCALE),
                                                 (1.0, 1.0, 0.0), (1.0, 1.0, -0.2), (1.0, 1.0, 4.0)])
def test_q4_decode_ranges_of_values(kscale, vscale, scale):
    g = gen(50)
    lens = [300, 77]
    bt, pool = q4_cache(g, lens, 2, kscale, vscale)
    q = normal(g, 2, 8, D)
    ws = q4_ws(q, pool, bt)
    out = pkv.q4_decode(q, pool, bt, ints(lens), scale=scale, ws=ws)
    assert status(ws) == 0
    check_q4(q, pool, bt, lens, out, scale=scale)


def test_q4_decode_value_scales_that_grow_along_the_row():
    """V's magnitude grows by 2^20 along the row, and shrinks along another: the weights' common factor follows."""
    g = gen(51)
    n = 500
    bt, pool = q4_cache(g, [n, n], 2)
    grow = torch.exp2(torch.linspace(-10, 10, n, device="cuda"))[:, None, None]
    for b, f in ((0, grow), (1, grow.flip(0))):
        k, v = normal(g, n, 2, D), (torch.randn((n, 2, D), generator=g, device="cuda") * f).half()
        ref.put_tokens(pool, bt[b], torch.arange(n, device="cuda"), k, v)
    q = normal(g, 2, 8, D)
    out = pkv.q4_decode(q, pool, bt, ints([n, n]))
    check_q4(q, pool, bt, [n, n], out)


@pytest.mark.parametrize("hq,hkv", [(8, 2), (16, 1)])
@pytest.mark.parametrize("vscale", [1.0, 1e-3, 3e3])
@pytest.mark.parametrize("size", [64.0, 512.0, 8192.0])
@pytest.mark.parametrize("order,sign", [("up", 1), ("down", 1), ("random", -1)])
def test_q4_decode_scores_of_which_fp32_has_no_fractions(order, sign, size, vscale, hq, hkv):
    """Scores from 2^24 to 2^31 (in log2), thousands apart: the output is the value that the greatest key's V stands
    for, up to the fp32 sum of its parts and its own rounding."""
    n, g = 250, gen(96)
    lens = [n, 77, 1]
    bt, pool = q4_cache(g, lens, hkv)
    best = []
    for b, m in enumerate(lens):
        level, at = one_hot_levels(g, order, sign, m)
        k = level.half()[:, None, None].expand(m, hkv, D)  # groups of equal values: exact
        v = (torch.randn((m, hkv, D), generator=g, device="cuda") * vscale).half()
        ref.put_tokens(pool, bt[b], torch.arange(m, device="cuda"), k, v)
        best.append(int(at[-1]))
    q = torch.full((3, hq, D), size, dtype=torch.float16, device="cuda")
    ws = q4_ws(q, pool, bt)
    out = pkv.q4_decode(q, pool, bt, ints(lens), ws=ws)
    assert status(ws) == 0
    for b in range(3):
        _, (c, sc, off) = ref.get_tokens(pool, bt[b], torch.tensor([best[b]], device="cuda"))
        coded = ref.values(c, sc, torch.zeros_like(off))
        want = ref.values(c, sc, off)
        parts = coded.abs() + off.double().abs().repeat_interleave(64, -1)
        # two fp16 parts of the scale (2^-21), the codes' common offset of up to 128 steps in and out (2^-24 each)
        bound = ref.HALF_STEP * want.abs() + 2.0 ** -15 * parts + 128 * 2.0 ** -22 * sc.double().repeat_interleave(64, -1) + ref.TINY
        bound = bound + 15 * ref.TINY * 2.0 ** -7
        ref.check(out[b], want[0].repeat_interleave(hq // hkv, 0), bound[0].repeat_interleave(hq // hkv, 0), f"row {b}")


def test_q4_decode_small_values_beside_large_ones():
    """The weights lie on tokens whose V is 2^14 times smaller than that of their neighbours, which have none."""
    g = gen(97)
    n = 700
    bt, pool = q4_cache(g, [n], 2)
    q = normal(g, 1, 8, D)
    q[:, :, 0] = 8.0
    small = torch.rand(n, generator=g, device="cuda") < 0.3
    small[::16] = False  # a page's first token is a large one
    k = normal(g, n, 2, D)
    k[:, :, 0] = torch.where(small, 60.0, -60.0).half()[:, None]
    v = (torch.randn((n, 2, D), generator=g, device="cuda") * torch.where(small, 2.0 ** -4, 2.0 ** 10)[:, None, None]).half()
    ref.put_tokens(pool, bt[0], torch.arange(n, device="cuda"), k, v)
    out = pkv.q4_decode(q, pool, bt, ints([n]))
    w, bound = ref.q4_row(q[0], pool, bt[0], n, SCALE)
    # Without the term for weights * scale below fp16's least steps: the largest is 2^7 for the large tokens' scale, thus
    # at least 2^-8 for the small ones', of which the second part's half step, 2^-25, is 2^-17.
    scales = ref.get_tokens(pool, bt[0], torch.arange(n, device="cuda"))[1][1].double()
    bound = bound - 15 * n * ref.TINY * float(scales.max()) * 2.0 ** -7
    ref.check(out[0], w, bound)


@pytest.mark.parametrize("hq,hkv", [(32, 8), (16, 1), (3, 3)])
def test_q4_decode_appends_the_new_token(hq, hkv):
    g = gen(52)
    lens = [1, 16, 17, 0, 300, 1025]
    bt, pool = q4_cache(g, [max(n - 1, 0) for n in lens], hkv, extra=20)
    used = set(bt[bt >= 0].tolist())
    free = [p for p in range(pool.shape[0]) if p not in used]
    bt = torch.cat((bt, torch.full((6, 1), -1, dtype=torch.int32, device="cuda")), 1)
    for b, n in enumerate(lens):
        if n and (n - 1) % PS == 0:
            bt[b, (n - 1) // PS] = free.pop()
    q, kn, vn = normal(g, 6, hq, D), normal(g, 6, hkv, D), normal(g, 6, hkv, D)
    want = pool.clone()
    for b, n in enumerate(lens):
        if n:
            ref.put_tokens(want, bt[b], torch.tensor([n - 1], device="cuda"), kn[b:b + 1], vn[b:b + 1])
    ws = q4_ws(q, pool, bt)
    for call in range(2):  # the second call appends the same token again
        out = pkv.q4_decode(q, pool, bt, ints(lens), k_new=kn, v_new=vn, ws=ws)
        assert status(ws) == 0
        assert torch.equal(pool, want)
        check_q4(q, want, bt, lens, out, what=f"call {call}")


@pytest.mark.parametrize("batch", [257, 4096])
def test_q4_decode_of_many_rows(batch):
    g = gen(53)
    lens = [(i * 37) % 90 for i in range(batch)]
    lens[batch // 2] = 5000
    n = [(x + PS - 1) // PS for x in lens]
    pages = sum(n)
    perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    host = torch.full((batch, max(n)), -1, dtype=torch.int32)
    flat, at = perm.cpu(), 0
    for b, c in enumerate(n):
        host[b, :c] = flat[at:at + c]
        at += c
    bt = host.cuda()
    pool = torch.randint(0, 256, (pages, 2, ref.BLOCK), dtype=torch.uint8, device="cuda", generator=g)
    for at in (1024, 2176):  # random codes, ordinary parameters
        par = torch.stack((torch.rand((pages, 2, 32), generator=g, device="cuda") * 0.3, torch.randn((pages, 2, 32), generator=g, device="cuda")), -1)
        pool[:, :, at:at + 128] = par.half().flatten(-2).contiguous().view(torch.uint8)
    q = normal(g, batch, 8, D)
    ws = q4_ws(q, pool, bt)
    out = pkv.q4_decode(q, pool, bt, ints(lens), ws=ws)
    assert status(ws) == 0
    check_q4(q, pool, bt, lens, out, rows=sorted({0, 1, 2, 3, 100, batch // 2 - 1, batch // 2, batch // 2 + 1, batch - 2, batch - 1}))
    empty = [b for b in range(batch) if lens[b] == 0]
    assert (out[empty] == 0).all()


def test_q4_decode_long_rows():
    g = gen(54)
    lens = [40000, 9]
    bt, pool = q4_cache(g, lens, 2)
    q = normal(g, 2, 8, D)
    ws = q4_ws(q, pool, bt)
    out = pkv.q4_decode(q, pool, bt, ints(lens), ws=ws)
    assert status(ws) == 0
    check_q4(q, pool, bt, lens, out)


def test_q4_decode_offsets_past_32_bits():
    """A pool of 4.7 GB: blocks behind 2^32 bytes are read and written at their places."""
    g = gen(55)
    pages, hkv = 255000, 8
    pool = torch.zeros((pages, hkv, ref.BLOCK), dtype=torch.uint8, device="cuda")
    bt = ints([[pages - 1, 3, pages - 2, 120000]])
    n = 55
    cu = cu_of([n])
    _, k, v, _ = packed(g, [n], hkv, hkv)
    pkv.q4_prompt_append(k, v, cu, pool, bt)
    want = torch.zeros((4, hkv, ref.BLOCK), dtype=torch.uint8, device="cuda")
    ref.put_tokens(want, torch.arange(4, device="cuda"), torch.arange(n, device="cuda"), k, v)
    assert torch.equal(pool[bt[0].long()], want)
    q = normal(g, 1, 32, D)
    out = pkv.q4_decode(q, pool, bt, ints([n]))
    check_q4(q, pool, bt, [n], out)


def test_q4_decode_nan_reaches_its_row_alone():
    g = gen(56)
    lens = [100, 80]
    bt, pool = q4_cache(g, lens, 2)
    bad = normal(g, 1, 2, D)
    bad[0, 1, 5] = math.nan
    ref.put_tokens(pool, bt[0], torch.tensor([40], device="cuda"), normal(g, 1, 2, D), bad)
    q = normal(g, 2, 8, D)
    out = pkv.q4_decode(q, pool, bt, ints(lens))
    torch.cuda.synchronize()
    assert torch.isnan(out[0, 4:, :64]).all()  # KV head 1, the group of dims 0-63
    check_q4(q, pool, bt, lens, out, rows=[1])


def test_q4_decode_reports_bad_pages_and_lengths():
    g = gen(57)
    lens = [100, 80, 64]
    bt, pool = q4_cache(g, lens, 2)
    q = normal(g, 3, 8, D)
    ws = q4_ws(q, pool, bt)
    for entry in (pool.shape[0], -1, 2 ** 31 - 1):
        bad = bt.clone()
        bad[1, 2] = entry
        out = pkv.q4_decode(q, pool, bad, ints(lens), ws=ws)
        assert status(ws) == pkv.PKV_STATUS_BAD_PAGE
        check_q4(q, pool, bt, lens, out, rows=[0, 2])
        (kc, ks, ko), (vc, vs, vo) = ref.get_tokens(pool, bt[1], torch.tensor([i for i in range(80) if i // PS != 2], device="cuda"))
        w, _ = ref.attend(q[1:2], ref.values(kc, ks, ko), ref.values(vc, vs, vo), SCALE, 63)
        _, bound = ref.q4_row(q[1], pool, bt[1], 80, SCALE)
        ref.check(out[1], w[0], bound + ref.HALF_STEP * w[0].abs() + ref.HALF_STEP * 8, "the row without its bad page")
    for n in (-1, bt.shape[1] * PS + 1, 2 ** 31 - 1):
        out = torch.full_like(q, math.nan)
        pkv.q4_decode(q, pool, bt, ints([100, n, 64]), out=out, ws=ws)
        assert status(ws) == pkv.PKV_STATUS_BAD_LEN
        check_q4(q, pool, bt, [100, 0, 64], out)
    pkv.q4_decode(q, pool, bt, ints(lens), ws=ws)
    assert status(ws) == 0


def test_q4_decode_on_another_stream_and_captured():
    g = gen(58)
    lens = [900, 33, 512]
    bt, pool = q4_cache(g, lens, 8)
    q = normal(g, 3, 32, D)
    ws = q4_ws(q, pool, bt)
    n = ints(lens)
    out = torch.empty_like(q)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    pkv.q4_decode(q, pool, bt, n, out=out, ws=ws, stream=side)
    made = pkv.q4_decode(q, pool, bt, n, stream=side.cuda_stream)
    side.synchronize()
    check_q4(q, pool, bt, lens, out)
    assert torch.equal(made, out)
    graphs = []
    for _ in range(2):  # two graphs share the workspace
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            pkv.q4_decode(q, pool, bt, n, out=out, ws=ws)
        graphs.append(graph)
    for i, now in enumerate(([900, 33, 512], [1, 0, 500], [899, 20, 3], [0, 0, 0])):
        n.copy_(ints(now))
        q.copy_(normal(gen(60 + i), *q.shape))
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        check_q4(q, pool, bt, now, out)
    assert status(ws) == 0


def test_q4_decode_results_do_not_depend_on_the_order_of_work():
    g = gen(59)
    lens = [3000, 17, 700, 2000]
    bt, pool = q4_cache(g, lens, 4)
    q = normal(g, 4, 16, D)
    a = pkv.q4_decode(q, pool, bt, ints(lens))
    for _ in range(4):
        assert torch.equal(a, pkv.q4_decode(q, pool, bt, ints(lens)))


# -------------------------------------------------------------------------------------------------------- all together
def test_prompt_then_decode_over_both_caches():
    """A serving program's run: attention over the prompts, their K/V into FP16 pages and into 4-bit pages, then tokens
    one by one. The FP16 decode of a token is the last row of the attention over the longer prompt; the 4-bit decode is
    the attention over the quantised tokens."""
    g = gen(70)
    hq, hkv, lens, steps = 32, 8, [130, 16, 77], 3
    full = [n + steps for n in lens]
    q, k, v, cu_full = packed(g, full, hq, hkv)
    at = cu_full.tolist()
    keep = torch.cat([torch.arange(at[b], at[b] + lens[b], device="cuda") for b in range(3)])
    cu = cu_of(lens)
    ws = new_ws()
    whole = pkv.prompt_attention(q, k, v, cu_full, ws=ws)
    head = pkv.prompt_attention(q[keep], k[keep], v[keep], cu, ws=ws)
    check_prompt(q, k, v, cu_full, whole)
    check_prompt(q[keep], k[keep], v[keep], cu, head)
    bt, pages = table(g, full)
    kp = torch.zeros((pages, PS, hkv, D), dtype=torch.float16, device="cuda")
    vp = torch.zeros_like(kp)
    pool = torch.zeros((pages, hkv, pkv.PKV_Q4_BLOCK_BYTES), dtype=torch.uint8, device="cuda")
    pkv.prompt_append(k[keep], v[keep], cu, kp, vp, bt, ws=ws)
    pkv.q4_prompt_append(k[keep], v[keep], cu, pool, bt, ws=ws)
    assert status(ws) == 0
    dws = q4_ws(q[:3], pool, bt)
    for step in range(steps):
        now = [n + step + 1 for n in lens]
        rows = torch.tensor([at[b] + now[b] - 1 for b in range(3)], device="cuda")
        qt, kt, vt = q[rows].contiguous(), k[rows].contiguous(), v[rows].contiguous()
        problem = pkv.make_problem(3, hq, hkv, D, PS, pages, bt.shape[1])
        plan = pkv.pkv_plan(problem, now, torch.cuda.get_device_properties(0).multi_processor_count)
        out = torch.empty_like(qt)
        pkv.pkv_decode_step_append(plan, problem, qt, kt, vt, kp, vp, bt, ints(now), SCALE, pkv.alloc_workspace(plan.ws_bytes), out)
        for b in range(3):
            a = at[b]
            w, mag = ref.attend(qt[b:b + 1], k[a:a + now[b]], v[a:a + now[b]], SCALE, now[b] - 1)
            bound = ref.prompt_bound(w, mag, now[b], qt[b:b + 1], k[a:a + now[b]], v[a:a + now[b]], SCALE)
            ref.check(out[b:b + 1], w, bound, "fp16 decode")
            ref.check(whole[rows[b]:rows[b] + 1], w, bound, "the prompt's row")
        out4 = pkv.q4_decode(qt, pool, bt, ints(now), k_new=kt, v_new=vt, ws=dws)
        assert status(dws) == 0
        check_q4(qt, pool, bt, now, out4)
    n = [x for x in full]
    kr, vr = pkv.q4_read(cu_of(n), pool, bt, total_tokens=sum(n))
    for x, y in ((k, kr), (v, vr)):
        w = ref.values(*ref.quantise(x))
        ref.check(y, w, ref.HALF_STEP * 1.01 * w.abs() + ref.TINY)
