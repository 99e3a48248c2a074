"""The prompt and 4-bit-cache operators where one call's state meets another's, and where values or lengths are extreme,
against the plain 64-bit forms of tests/prompt_reference.py."""

import math
import random

import pytest
import torch

import prompt_reference as ref
import serving_paged_gqa_gb300 as pkv
from test_prompts_gpu import (D, PS, SCALE, check_prompt, check_q4, gen, ints, new_ws, normal, packed, q4_cache, status,
                              table)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__

    __graft_entry__.build()
    torch.cuda.set_device(0)


def q4_step(problem, q, pool, bt, lens, num_sms, ws, out):
    """The C call, for a GPU of num_sms SMs."""
    stream = torch.cuda.current_stream().cuda_stream
    rc = pkv.load().pkv_q4_decode_step(problem, q.data_ptr(), pool.data_ptr(), bt.data_ptr(), lens.data_ptr(), SCALE, num_sms,
                                       ws.data_ptr(), ws.numel(), out.data_ptr(), stream)
    assert rc == 0


# --------------------------------------------------------------------------------------------- one workspace, many calls
def test_q4_steps_of_different_heads_share_a_workspace():
    """Rows that are split over many CTAs, steps of G = 16, 4, 1 and 8 and grids of different sizes in turn, on one
    workspace that was zeroed once: every step finds its arrival counters at zero."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    steps = []
    for hq, hkv, lens in ((16, 1, [20000, 9]), (32, 8, [5000, 4990, 70, 5100, 4800]), (3, 3, [30000]), (16, 2, [9000, 9100])):
        g = gen(200 + hq)
        bt, pool = q4_cache(g, lens, hkv)
        steps.append((hq, hkv, lens, bt, pool, normal(g, len(lens), hq, D)))
    problems = [pkv.q4_problem(q, pool, bt) for _, _, _, bt, pool, q in steps]
    counts = (sms, 100, sms)
    ws = new_ws(max(pkv.pkv_q4_workspace_bytes(p, n) for p in problems for n in counts))
    for n in counts:
        for p, (hq, hkv, lens, bt, pool, q) in zip(problems, steps):
            out = torch.full_like(q, math.nan)
            q4_step(p, q, pool, bt, ints(lens), n, ws, out)
            assert status(ws) == 0
            check_q4(q, pool, bt, lens, out, what=f"{hq} heads on {n} SMs")


# ------------------------------------------------------------------------------------- tiles that end in a step's first half
@pytest.mark.parametrize("hq,hkv", [(8, 2), (3, 3), (16, 1)])
@pytest.mark.parametrize("num_sms", [1, 2, 7])
def test_prompt_many_tiles_that_end_in_a_first_half(num_sms, hq, hkv):
    """Sequences whose last step has 1 to 64 keys, among others, dozens of pairs of tiles one after the other in a CTA: the
    warps of the second 64 keys have nothing to do in those steps, and meet the next tile's in phase all the same."""
    lens = [40, 300, 1, 64, 65, 128, 190, 129, 20, 192, 257, 0, 60, 384 + 33, 5, 64] * 2
    q, k, v, cu = packed(gen(230 + hq), lens, hq, hkv, fused=False)
    out = torch.full_like(q, math.nan)
    ws = new_ws()
    p = pkv.make_prompt(len(lens), q.shape[0], hq, hkv, D)
    for call in range(3):
        rc = pkv.load().pkv_prompt_attention(p, q.data_ptr(), k.data_ptr(), v.data_ptr(), cu.data_ptr(), SCALE, num_sms, ws.data_ptr(),
                                             ws.numel(), out.data_ptr(), torch.cuda.current_stream().cuda_stream)
        assert rc == 0 and status(ws) == 0
        check_prompt(q, k, v, cu, out, what=f"call {call}")


@pytest.mark.parametrize("variant", [pkv.PKV_VARIANT_WORKQUEUE, pkv.PKV_VARIANT_SPLIT])
def test_prompt_calls_on_the_workspaces_of_decode_steps(variant):
    """The prompt calls use a workspace's header alone, and leave it as they found it: on the workspace of an FP16 step, and of
    a 4-bit one, between steps."""
    g, hq, hkv, lens = gen(205), 8, 2, [900, 40, 1300]
    q, k, v, cu = packed(g, lens, hq, hkv, fused=False)
    bt, pages = table(g, lens)
    kp, vp = (torch.zeros((pages, PS, hkv, D), dtype=torch.float16, device="cuda") for _ in range(2))
    pool = torch.zeros((pages, hkv, ref.BLOCK), dtype=torch.uint8, device="cuda")
    qt, n = normal(g, 3, hq, D), ints(lens)
    problem = pkv.make_problem(3, hq, hkv, D, PS, pages, bt.shape[1])
    plan = pkv.pkv_plan_fixed(problem, lens, torch.cuda.get_device_properties(0).multi_processor_count, variant, 8)
    wide, four = new_ws(plan.ws_bytes), new_ws(pkv.pkv_q4_workspace_bytes(problem))
    for call in range(3):
        for ws in (wide, four):
            out = pkv.prompt_attention(q, k, v, cu, ws=ws)
            check_prompt(q, k, v, cu, out, what=f"call {call}")
            pkv.prompt_append(k, v, cu, kp, vp, bt, ws=ws)
            pkv.q4_prompt_append(k, v, cu, pool, bt, ws=ws)
        out, out4 = torch.full_like(qt, math.nan), torch.full_like(qt, math.nan)
        pkv.pkv_decode_step(plan, problem, qt, kp, vp, bt, n, SCALE, wide, out)
        pkv.q4_decode(qt, pool, bt, n, out=out4, ws=four)
        assert status(wide) == 0 and status(four) == 0
        check_q4(qt, pool, bt, lens, out4, what=f"call {call}")
        at = cu.tolist()
        for b in range(3):
            rows = slice(at[b], at[b + 1])
            w, mag = ref.attend(qt[b:b + 1], k[rows], v[rows], SCALE, lens[b] - 1)
            ref.check(out[b:b + 1], w, ref.prompt_bound(w, mag, lens[b], qt[b:b + 1], k[rows], v[rows], SCALE), f"row {b}")


# ----------------------------------------------------------------------------------------------- small softmax weights
@pytest.mark.parametrize("n,hq,hkv", [(3000, 8, 2), (16384, 4, 4)])
@pytest.mark.parametrize("nats", [10.0, 14.0, 16.0, 18.0])
def test_prompt_small_weights_beside_a_large_one(nats, n, hq, hkv):
    """An attention sink: the first key's score is `nats` above the mean of the others, and its V is 0, so that the output
    is made of the small weights. Their numerator keeps what their sum counts."""
    g = gen(210)
    q, k, v, cu = packed(g, [n], hq, hkv, fused=False)
    q[:, :, 0] = 8.0
    k[:, :, 0] = 0.0
    k[0] = 0.0
    k[0, :, 0] = nats / (8.0 * SCALE)
    v = (v.float() * 0.5 + 1.0).half()
    v[0] = 0.0
    ws = new_ws()
    out = pkv.prompt_attention(q, k, v, cu, ws=ws)
    assert status(ws) == 0
    for a in (1, n // 2, n - 130):
        e = min(n, a + 130)
        w, mag = ref.attend(q[a:e], k[:e], v[:e], SCALE, a)
        # As ref.prompt_bound, but for weights below fp16's least normal one: the first key's weight is 2^5 (what a row's
        # first maximum gets), so half the least subnormal is 2^-30 of it; the sum of all weights is at least that.
        ds = ref.prompt_bound(w, mag, 0, q[a:e], k[:e], v[:e], SCALE)
        ref.check(out[a:e], w, ds + e * 2.0 ** -30 * float(v.abs().max()), f"rows {a}..")


@pytest.mark.parametrize("rise", [11.5, 16.9, 18.0, 19.9, 21.0, 25.0])
@pytest.mark.parametrize("first,second", [(130, 200), (200, 130), (150, 255), (70, 10)])
def test_prompt_a_step_whose_halves_rise_by_little(rise, first, second):
    """Key `first` raises the running reference by `rise` (in log2), while key `second` of the same step's other half stays
    just below the 2^16 that lets its weight as it is (the first keys have 2^5); its V is large enough to be seen."""
    n, g = 300, gen(240)
    q, k, v, cu = packed(g, [n], 8, 1, fused=False)
    unit = 1.0 / (8.0 * SCALE * math.log2(math.e))  # of k's dim 0, for a score of 1 in log2
    q.zero_()
    k.zero_()
    q[:, :, 0] = 8.0
    k[first, :, 0], k[second, :, 0] = rise * unit, 10.9 * unit
    v[second] *= 2.0 ** max(0.0, rise - 10.9)
    ws = new_ws()
    out = pkv.prompt_attention(q, k, v, cu, ws=ws)
    assert status(ws) == 0
    check_prompt(q, k, v, cu, out)


# ------------------------------------------------------------------------------------- infinities in recomputed rows
@pytest.mark.parametrize("far", [40.0, 400.0])
@pytest.mark.parametrize("hq,hkv", [(8, 2), (2, 2)])
def test_prompt_infinities_in_rows_that_are_computed_again(hq, hkv, far):
    """V has infinities in a token whose weight is 0 in fp32, before and after the row's greatest score, and a NaN that the
    row does not attend to, for which it is computed again: infinities still make their dims infinite, of both signs NaN."""
    n, hit, g = 200, 180, gen(220)
    q, k, v, cu = packed(g, [n], hq, hkv, fused=False)
    q[:, :, 0] = 8.0
    k[:, :, 0] = 0.0
    k[100, :, 0] = far / (8.0 * SCALE * math.log2(math.e))  # from here on the others' weights are about 2^-far
    vb = v.clone()
    vb[5, :, 10], vb[150, :, 11], vb[7, :, 12], vb[151, :, 12], vb[9, :, 13] = math.inf, -math.inf, math.inf, -math.inf, math.nan
    vb[hit, :, 20] = math.nan  # its tile's rows before it are computed again
    vb[hit, :, 100] = math.inf
    ws = new_ws()
    out = pkv.prompt_attention(q, k, vb, cu, ws=ws)
    assert status(ws) == 0
    v[[5, 150, 7, 151, 9, hit, hit], :, [10, 11, 12, 12, 13, 20, 100]] = 0.0
    w, mag = ref.attend(q, k, v, SCALE, 0)
    bound = ref.prompt_bound(w, mag, n, q, k, v, SCALE)
    want = w.clone()
    want[5:, :, 10], want[150:, :, 11], want[7:151, :, 12], want[151:, :, 12], want[9:, :, 13] = math.inf, -math.inf, math.inf, math.nan, math.nan
    want[hit:, :, 20], want[hit:, :, 100] = math.nan, math.inf
    fin = torch.isfinite(want)
    assert torch.equal(torch.isnan(out), torch.isnan(want))
    assert (out.double()[torch.isinf(want)] == want[torch.isinf(want)]).all()
    ref.check(torch.where(fin, out.double(), 0.0), torch.where(fin, want, 0.0), bound)


# ------------------------------------------------------------------------------------------------- rows without a finite score
def graph_us(call, reps=6, best_of=9):
    """Device time of a call: the shortest of several replays of a graph of `reps` calls."""
    for _ in range(3):
        call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(reps):
            call()
    times = []
    for _ in range(best_of + 1):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        graph.replay()
        b.record()
        torch.cuda.synchronize()
        times.append(a.elapsed_time(b) / reps * 1e3)
    return min(times[1:])


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_prompt_rows_of_nan_behind_the_end_cost_nothing(bad):
    """A padded batch's garbage: the queries behind a sequence share its last tile's warps, whose steps stay ordinary."""
    n = 2043
    q, k, v, cu = packed(gen(250), [n], 32, 8, behind=60, fused=False)
    out, ws = torch.empty_like(q), new_ws()
    took = []
    for x in (1.0, bad):
        q[n:] = x
        took.append(graph_us(lambda: pkv.prompt_attention(q, k, v, cu, out=out, ws=ws)))
        assert status(ws) == 0
    check_prompt(q, k, v, cu, out)
    assert took[1] < 1.5 * took[0], took


@pytest.mark.parametrize("hq,hkv", [(8, 2), (2, 2)])
def test_prompt_rows_whose_first_scores_are_minus_infinity(hq, hkv):
    """Keys of which every query makes -inf, at the beginning, in whole steps and in a step's second half: rows that attend
    to nothing else are NaN (a softmax of -inf alone), and the others are as if those keys were not there."""
    n, g = 420, gen(251)
    for hide in (list(range(0, 3)), list(range(0, 64)), list(range(0, 70)), list(range(0, 200)), list(range(0, 300)),
                 [*range(0, 64), *range(128, 192)], list(range(64, 128))):
        q, k, v, cu = packed(g, [n], hq, hkv, fused=False)
        q[:, :, 0] = 4.0
        k[:, :, 0] = 0.0
        kb = k.clone()
        kb[hide, :, 0] = -math.inf
        ws = new_ws()
        out = pkv.prompt_attention(q, kb, v, cu, ws=ws)
        assert status(ws) == 0
        keep = torch.tensor([i for i in range(n) if i not in set(hide)], device="cuda")
        first = int(keep[0])
        assert torch.isnan(out[:first]).all()
        for i in range(first, n, 29):
            seen = keep[keep <= i]
            w, mag = ref.attend(q[i:i + 1], k[seen], v[seen], SCALE, len(seen) - 1)
            ref.check(out[i:i + 1], w, ref.prompt_bound(w, mag, len(seen), q[i:i + 1], k[seen], v[seen], SCALE), f"{hide[-1]} row {i}")


def test_prompt_rows_computed_again_for_longer_than_a_wait_may_take():
    """A NaN in the last of half a million tokens: a warp computes 32 rows before it again from all their keys, which takes
    more than the 2 s after which a wait of the kernel's other warps gives up."""
    n = 1 << 19
    q, k, v, cu = packed(gen(260), [n], 1, 1, fused=False)
    v[n - 1, 0, 77] = math.nan
    ws = new_ws()
    out = torch.full_like(q, math.inf)
    pkv.prompt_attention(q, k, v, cu, out=out, ws=ws)
    assert status(ws) == 0
    assert torch.isnan(out[n - 1, 0, 77]) and int((~torch.isfinite(out)).sum()) == 1
    v[n - 1, 0, 77], out[n - 1, 0, 77] = 0.0, 0.0
    for a in (n - 128, n // 2):
        w, mag = ref.attend(q[a:a + 127], k[:a + 127], v[:a + 127], SCALE, a)
        ref.check(out[a:a + 127], w, ref.prompt_bound(w, mag, a + 127, q[a:a + 127], k[:a + 127], v[:a + 127], SCALE), f"rows {a}..")


@pytest.mark.parametrize("near,far", [(-125.5, -130.0), (-140.0, -145.0), (-125.0, -160.0), (-700.0, -701.0), (-3.0, -9.0)])
def test_prompt_scores_far_below_zero_behind_minus_infinity(near, far):
    """Behind first keys of -inf the first finite scores (in log2) are the row's reference, however far below 0 they are:
    2^x of them may be nothing in fp32."""
    n, first, then = 330, 64, 200
    q, k, v, cu = packed(gen(252), [n], 8, 2, fused=False)
    unit = 1.0 / (16.0 * SCALE * math.log2(math.e))
    q.zero_()
    k.zero_()
    q[:, :, 0] = 16.0
    k[first:then, :, 0], k[then:, :, 0] = far * unit, near * unit
    kb = k.clone()
    kb[:first, :, 0] = -math.inf
    ws = new_ws()
    out = pkv.prompt_attention(q, kb, v, cu, ws=ws)
    assert status(ws) == 0
    assert torch.isnan(out[:first]).all()
    k, v, q, out = k[first:], v[first:], q[first:], out[first:]
    w, mag = ref.attend(q, k, v, SCALE, 0)
    ref.check(out, w, ref.prompt_bound(w, mag, n - first, q, k, v, SCALE))


# -------------------------------------------------------------------------------------------- many sequences, other heads
def mixed(n, seed):
    """Lengths of n sequences, empty ones and of one to a dozen pairs of tiles (at 16 heads to a KV head, a hundred) among
    them, in no order."""
    r = random.Random(seed)
    lens = [r.choice([0, 1, 2, 40, 129, 300, 517, 1500]) for _ in range(n)]
    lens[r.randrange(n)] = 1777
    return lens


@pytest.mark.parametrize("hq,hkv", [(2, 2), (16, 1), (8, 2)])
@pytest.mark.parametrize("n", [32, 33, 80])
def test_prompt_more_sequences_than_a_warp_holds(n, hq, hkv):
    """Above 32 sequences the claims go by a sorted list: every row of every sequence, on whole and on small grids."""
    lens = mixed(n, 300 + n)
    q, k, v, cu = packed(gen(270 + n), lens, hq, hkv, before=1, behind=9)
    p = pkv.make_prompt(n, q.shape[0], hq, hkv, D, q.stride(0), k.stride(0), v.stride(0))
    ws = new_ws()
    whole = None
    for num_sms in (torch.cuda.get_device_properties(0).multi_processor_count, 5):
        out = torch.full((q.shape[0], hq, D), 7.0, dtype=torch.float16, device="cuda")
        rc = pkv.load().pkv_prompt_attention(p, q.data_ptr(), k.data_ptr(), v.data_ptr(), cu.data_ptr(), SCALE, num_sms, ws.data_ptr(),
                                             ws.numel(), out.data_ptr(), torch.cuda.current_stream().cuda_stream)
        assert rc == 0 and status(ws) == 0
        assert (out[:1] == 7).all() and (out[-9:] == 7).all()
        if whole is None:
            whole = out
            check_prompt(q, k, v, cu, out)
        else:
            assert torch.equal(out, whole)


@pytest.mark.parametrize("hq,hkv", [(2, 2), (4, 2), (16, 2), (16, 1)])
def test_prompt_longer_with_other_heads(hq, hkv):
    lens = [2500, 130, 1111]
    q, k, v, cu = packed(gen(280 + hq), lens, hq, hkv, behind=3)
    ws = new_ws()
    out = pkv.prompt_attention(q, k, v, cu, ws=ws)
    assert status(ws) == 0
    check_prompt(q, k, v, cu, out)


@pytest.mark.parametrize("starts", [False, True])
@pytest.mark.parametrize("n,hkv", [(33, 2), (70, 1), (70, 3)])
def test_page_calls_of_more_sequences_than_a_warp_holds(n, hkv, starts):
    """The warps' items run on from one block of 32 sequences to the next: every token of every sequence is written once, into
    its slot, and read back from there."""
    r, g = random.Random(n), gen(290 + n)
    lens = [r.choice([0, 0, 1, 15, 16, 17, 100, 333]) for _ in range(n)]
    has = [r.randrange(40) if starts else 0 for _ in range(n)]
    _, k, v, cu = packed(g, lens, hkv, hkv, before=2, behind=2)
    bt, pages = table(g, [a + b for a, b in zip(lens, has)])
    start = ints(has) if starts else None
    kp, vp = normal(g, pages, PS, hkv, D), normal(g, pages, PS, hkv, D)
    pool = torch.randint(0, 256, (pages, hkv, ref.BLOCK), dtype=torch.uint8, device="cuda", generator=g)
    want_k, want_v, want, at = kp.clone(), vp.clone(), pool.clone(), cu.tolist()
    for b in range(n):
        rows = slice(at[b], at[b + 1])
        if lens[b]:
            pos = torch.arange(lens[b], device="cuda") + has[b]
            page = bt[b][pos // PS].long()
            want_k[page, pos % PS], want_v[page, pos % PS] = k[rows], v[rows]
            ref.put_tokens(want, bt[b], pos, k[rows], v[rows])
    ws = new_ws()
    pkv.prompt_append(k, v, cu, kp, vp, bt, start=start, ws=ws)
    pkv.q4_prompt_append(k, v, cu, pool, bt, start=start, ws=ws)
    assert status(ws) == 0
    assert torch.equal(kp, want_k) and torch.equal(vp, want_v) and torch.equal(pool, want)
    k_out, v_out = (torch.full((k.shape[0], hkv, D), 7.0, dtype=torch.float16, device="cuda") for _ in range(2))
    pkv.q4_read(cu, pool, bt, start=start, k_out=k_out, v_out=v_out, ws=ws)
    assert status(ws) == 0
    for x, y in ((k, k_out), (v, v_out)):
        w = ref.values(*ref.quantise(x[at[0]:at[-1]]))
        ref.check(y[at[0]:at[-1]], w, ref.HALF_STEP * w.abs() + 2.0 ** -23 * w.abs() + ref.TINY, "read")
        assert (y[:at[0]] == 7).all() and (y[at[-1]:] == 7).all()
