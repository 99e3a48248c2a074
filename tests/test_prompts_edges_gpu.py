"""The prompt and 4-bit-cache operators where one call's state meets another's, and where values or lengths are extreme,
against the plain 64-bit forms of tests/prompt_reference.py."""

import math

import pytest
import torch

import serving_paged_gqa_gb300 as pkv
from test_prompts_gpu import D, SCALE, check_prompt, check_q4, gen, ints, new_ws, normal, packed, q4_cache, status

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
    counts = (sms, 100, 2 * sms)
    ws = new_ws(max(pkv.pkv_q4_workspace_bytes(p, n) for p in problems for n in counts))
    for n in (sms, sms, 100, 2 * sms, sms):
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
