"""Operators of a paged cache's serving loop as a user's program calls them, beside their plain forms.

``own`` False: every operator in elementary torch operations in 32 bits (page scores in 64, since pages next to the border
of a selection have to fall on the same side), rounded once at the end. ``own`` True: the calls of this repository's
library. ``exact`` gives the same outputs from the definitions in 64 bits.

Operators (``op`` of a case):
  chunk    causal grouped-query attention of a chunk of new tokens of each sequence over the FP16 pages that hold its earlier
           tokens and the chunk's own K/V
  tables   block tables, slots, positions and sequence bounds of a step from the rows' lengths and new tokens, pages taken
           from a stack of free ones (``kind`` grow), or the pages of finished rows put back on it (``kind`` release)
  bounds   the least and greatest key of each page, dim by dim, of the pages that new tokens went to
  sparse   one decode step over the pages whose bounds promise a KV head's queries the greatest scores: the selection, then
           attention over the selected pages
"""

import math
import random

import numpy as np
import torch

own = False

D, PS = 128, 16


# ------------------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # a few proposed tokens of one conversation are verified: the smallest call, latency counts
        dict(name="chunk verify one", op="chunk", seqs=1, lo=5, hi=5, slo=700, shi=700, lseed=0, hq=32, hkv=8, fused=False),
        # a serving batch verifies two to eight proposed tokens each behind long contexts
        dict(name="chunk verify batch", op="chunk", seqs=16, lo=2, hi=8, slo=1000, shi=32000, lseed=1, hq=32, hkv=8, fused=True),
        # an ordinary chunk of a document that is read piece by piece
        dict(name="chunk 512 behind 8192", op="chunk", seqs=1, lo=512, hi=512, slo=8192, shi=8192, lseed=0, hq=32, hkv=8, fused=True),
        # a step of prompts, continued prompts and short turns, eight heads to a KV head
        dict(name="chunk mixed batch", op="chunk", seqs=12, lo=1, hi=1024, slo=0, shi=16000, lseed=2, hq=32, hkv=4, fused=False),
        # the last chunk of a long document
        dict(name="chunk 4096 behind 28672", op="chunk", seqs=1, lo=4096, hi=4096, slo=28672, shi=28672, lseed=0, hq=32, hkv=8, fused=False),
        # every decode step of a large batch: one token a row
        dict(name="tables decode step", op="tables", kind="grow", seqs=256, lo=1, hi=1, slo=1, shi=32000, lseed=3),
        # new prompts of different lengths come in, some of them behind a cached prefix
        dict(name="tables prompts", op="tables", kind="grow", seqs=64, lo=1, hi=4096, slo=0, shi=2000, lseed=4),
        # half of a batch ends
        dict(name="tables release", op="tables", kind="release", seqs=256, lo=1, hi=1, slo=1, shi=32000, lseed=5),
        # the page of each row's newest token
        dict(name="bounds decode step", op="bounds", seqs=48, lo=1, hi=1, slo=500, shi=32000, lseed=6, hkv=8),
        # prompts that have just been written into the pages
        dict(name="bounds prompts", op="bounds", seqs=8, lo=200, hi=8192, slo=0, shi=0, lseed=7, hkv=8),
        # one long conversation
        dict(name="sparse one row", op="sparse", seqs=1, slo=32768, shi=32768, lseed=0, hq=32, hkv=8, select=64),
        # a serving batch of long conversations
        dict(name="sparse batch", op="sparse", seqs=32, slo=4000, shi=32768, lseed=8, hq=32, hkv=8, select=128),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["chunk", "chunk", "chunk", "tables", "bounds", "sparse", "sparse"])
    g = rng.choice([1, 2, 4, 8, 16])
    hkv = rng.choice([h for h in (1, 2, 4, 8) if h * g <= 32])
    lseed = rng.randrange(1 << 20)
    if op == "chunk":
        hi = _spread(rng, 1, 4096)
        shi = rng.choice([0, _spread(rng, 1, 28000), _spread(rng, 1, 28000)])
        most = max(1, min(32, 300000 // (shi + hi), (1 << 27) // (hi * (shi + hi))))
        return dict(op=op, seqs=_spread(rng, 1, most), lo=rng.randint(1, hi), hi=hi, slo=rng.randint(0, shi), shi=shi, lseed=lseed,
                    hq=hkv * g, hkv=hkv, fused=rng.random() < 0.5)
    if op == "tables":
        hi, shi = rng.choice([1, 1, _spread(rng, 1, 4096)]), _spread(rng, 1, 32000)
        return dict(op=op, kind=rng.choice(["grow", "grow", "release"]), seqs=_spread(rng, 1, 64 if hi > 1 else 512), lo=rng.randint(1, hi), hi=hi,
                    slo=rng.randint(0, shi), shi=shi, lseed=lseed)
    if op == "bounds":
        hi, shi = rng.choice([1, _spread(rng, 1, 8192)]), rng.choice([0, _spread(rng, 1, 8000)])
        return dict(op=op, seqs=_spread(rng, 1, max(1, min(48, 50000 // (hi + shi)))), lo=rng.randint(1, hi), hi=hi, slo=rng.randint(0, shi),
                    shi=shi, lseed=lseed, hkv=hkv)
    shi = _spread(rng, 16, 32768)
    return dict(op=op, seqs=_spread(rng, 1, max(1, min(32, 700000 // shi))), slo=rng.randint(1, shi), shi=shi, lseed=lseed, hq=hkv * g, hkv=hkv,
                select=_spread(rng, 2, 160))


def _lens(case):
    """New tokens of each sequence, and those that it holds before them (sparse: the row's tokens)."""
    r = random.Random(case["lseed"])
    n = [r.randint(case["lo"], case["hi"]) if "lo" in case else 1 for _ in range(case["seqs"])]
    return n, [r.randint(case["slo"], case["shi"]) for _ in n]


def _pages_of(tokens):
    return (tokens + PS - 1) // PS


def work(case):
    n, start = _lens(case)
    t = sum(n)
    if case["op"] == "chunk":
        seen = sum(m * s + m * (m + 1) // 2 for m, s in zip(n, start))
        return {"bytes": (t * 2 * case["hq"] + sum(m + s for m, s in zip(n, start)) * 2 * case["hkv"]) * D * 2, "flops": 4 * D * case["hq"] * seen}
    if case["op"] == "tables":
        b = len(n)
        if case["kind"] == "release":  # flags, lengths in and out, the entries of the ended rows read and written
            return {"bytes": 12 * b + 8 * sum(_pages_of(s) for s in start[::2]), "flops": 0}
        new = sum(_pages_of(s + m) - _pages_of(s) for m, s in zip(n, start))
        return {"bytes": 20 * b + 8 * new + 12 * t, "flops": 0}  # lengths and bounds; entries; slots and positions
    if case["op"] == "bounds":
        pages = sum(_pages_of(s + m) - s // PS for m, s in zip(n, start))
        held = sum(s + m - s // PS * PS for m, s in zip(n, start))
        return {"bytes": case["hkv"] * D * 2 * (held + 2 * pages), "flops": 2 * held * case["hkv"] * D}
    hq, hkv, k = case["hq"], case["hkv"], case["select"]
    pages = [_pages_of(s) for s in start]
    keys = sum(min(s, (min(k, p) - 1) * PS + (s - 1) % PS + 1) for s, p in zip(start, pages))
    return {"bytes": hkv * (sum(pages) * 2 * D * 2 + keys * 2 * D * 2 + sum(min(k, p) for p in pages) * 4) + len(n) * hq * D * 4,
            "flops": hq * (sum(pages) * 2 * D + keys * 4 * D)}


# ----------------------------------------------------------------------------------------------------------- inputs
def _table(tokens, gen, dev, spare=3):
    """A block table over a shuffled pool: row b's pages at random places, -1 behind them; and the pages left over."""
    n = [_pages_of(x) for x in tokens]
    perm = torch.randperm(sum(n) + spare, generator=gen, device=dev).to(torch.int32)
    bt = torch.full((len(n), max(max(n), 1)), -1, dtype=torch.int32, device=dev)
    row = torch.repeat_interleave(torch.arange(len(n), device=dev), torch.tensor(n, device=dev))
    first = torch.tensor(np.cumsum([0] + n[:-1]), device=dev)
    at = torch.arange(sum(n), device=dev)
    bt[row, at - first[row]] = perm[: sum(n)]
    return bt, perm[sum(n):]


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    new, start = _lens(case)
    op, b = case["op"], case["seqs"]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev).half()

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device=dev)

    s = {"case": case, "scale": 1.0 / math.sqrt(D)}
    if op == "tables":
        held = start if case["kind"] == "release" else [x + y for x, y in zip(start, new)]
        grown = sum(_pages_of(x) for x in held)
        spare = 37 + grown - sum(_pages_of(x) for x in start)
        bt, free = _table(start, gen, dev, spare)
        pages = grown + 37
        width = max(1, max(_pages_of(x) for x in held))
        s["bt"] = torch.full((b, width), -1, dtype=torch.int32, device=dev)
        s["bt"][:, : bt.shape[1]] = bt
        s["free"] = torch.full((pages,), -1, dtype=torch.int32, device=dev)
        s["free"][: free.numel()] = free
        s["count"], s["lens"], s["count_out"], s["lens_out"] = ints([free.numel()]), ints(start), ints([0]), torch.zeros_like(ints(start))
        if case["kind"] == "release":
            s["ended"] = (torch.arange(b, device=dev) % 2 == 0).to(torch.int32)
            return s
        t = sum(new)
        s["new"], s["cu"], s["start"] = ints(new), torch.zeros(b + 1, dtype=torch.int32, device=dev), torch.zeros_like(ints(start))
        s["slots"] = torch.full((t + 5,), -1, dtype=torch.int64, device=dev)
        s["positions"] = torch.full((t + 5,), -1, dtype=torch.int32, device=dev)
        return s
    hkv = case["hkv"]
    total = start if op == "sparse" else [x + y for x, y in zip(start, new)]
    s["bt"], free = _table(total, gen, dev)
    num_pages = sum(_pages_of(x) for x in total) + free.numel()
    s["k_pool"] = normal(num_pages, PS, hkv, D)
    if op == "sparse":
        hq = case["hq"]
        s.update(q=normal(b, hq, D), v_pool=normal(num_pages, PS, hkv, D), lens=ints(start), out=torch.empty((b, hq, D), dtype=torch.float16, device=dev),
                 pages=torch.empty((b, hkv, case["select"]), dtype=torch.int32, device=dev))
        k = s["k_pool"].clone()  # the bounds are of the tokens that the pages hold
        row = torch.arange(b, device=dev)
        last = s["bt"][row, ((s["lens"] - 1) // PS).long()].long()
        beyond = torch.arange(PS, device=dev)[None] > ((s["lens"] - 1) % PS)[:, None]
        k[last] = torch.where(beyond[:, :, None, None], k[last, :1], k[last])
        s["bounds"] = torch.stack((k.amin(1), k.amax(1)), 2).contiguous()  # [num_pages, hkv, 2, D]
        return s
    s["cu"], s["start"] = ints(np.cumsum([0] + new).tolist()), ints(start)
    if op == "bounds":
        s["bounds"] = torch.zeros((num_pages, hkv, 2, D), dtype=torch.float16, device=dev)
        return s
    t, hq = sum(new), case["hq"]
    s["v_pool"] = normal(num_pages, PS, hkv, D)
    # fused: the queries are a slice of one [tokens, (Hq + 2 Hkv) * d] projection
    s["q"] = normal(t, hq + 2 * hkv, D)[:, :hq] if case["fused"] else normal(t, hq, D)
    s["out"] = torch.empty((t, hq, D), dtype=torch.float16, device=dev)
    return s


# ------------------------------------------------------------------------------------------------------ plain forms
def _rows(cu, t):
    """(sequence, index in it) of every packed token."""
    at = torch.arange(t, device=cu.device)
    seq = torch.searchsorted(cu[1:].contiguous(), at.to(torch.int32), right=True)
    return seq, at - cu[seq]


def _plain_chunk(s):
    q, start, bt, case = s["q"], s["start"], s["bt"].clamp(min=0).long(), s["case"]
    new, before = _lens(case)
    t, hq, hkv = q.shape[0], q.shape[1], case["hkv"]
    b, m, n, g = case["seqs"], max(new), bt.shape[1] * PS, hq // hkv
    seq, i = _rows(s["cu"], t)
    qp = torch.zeros((b, m, hq, D), dtype=torch.float32, device=q.device)
    qp[seq, i] = q.float()
    qp = qp.transpose(1, 2).reshape(b, hkv, g * m, D)
    k = s["k_pool"][bt].float().view(b, n, hkv, D).permute(0, 2, 3, 1)
    x = torch.matmul(qp, k).view(b, hkv, g, m, n).mul_(s["scale"])
    del k
    pos = start.long()[:, None] + torch.arange(m, device=q.device)[None]
    x.masked_fill_((torch.arange(n, device=q.device)[None, None] > pos[:, :, None])[:, None, None], -math.inf)
    x.sub_(x.amax(-1, keepdim=True)).exp_()
    v = s["v_pool"][bt].float().view(b, n, hkv, D).transpose(1, 2)
    y = torch.matmul(x.view(b, hkv, g * m, n), v).view(b, hq, m, D) / x.sum(-1).view(b, hq, m, 1)
    return {"out": y.transpose(1, 2)[seq, i].half()}


def _plain_grow(s):
    dev = s["lens"].device
    new, lens, bt, free = s["new"].long(), s["lens"].long(), s["bt"], s["free"].long()
    held = (lens + PS - 1) // PS
    need = (lens + new + PS - 1) // PS - held
    before = need.cumsum(0) - need
    p = torch.arange(bt.shape[1], device=dev)[None] - held[:, None]  # index among the row's new pages
    taken = (p >= 0) & (p < need[:, None])
    at = (s["count"].long() - 1 - before[:, None] - p).clamp(0, free.numel() - 1)
    bt.copy_(torch.where(taken, free[at], bt.long()))
    s["cu"].copy_(torch.cat((torch.zeros(1, dtype=torch.long, device=dev), new.cumsum(0))))
    t = s["slots"].numel() - 5
    seq, i = _rows(s["cu"], t)
    pos = lens[seq] + i
    s["slots"][:t] = bt.long()[seq, pos // PS] * PS + pos % PS
    s["positions"][:t] = pos.to(torch.int32)
    s["start"].copy_(lens)
    s["lens_out"].copy_(lens + new)
    s["count_out"].copy_(s["count"] - need.sum())
    return {x: s[x] for x in ("bt", "cu", "start", "slots", "positions", "lens_out", "count_out")}


def _plain_release(s):
    lens, bt, free = s["lens"].long(), s["bt"], s["free"]
    pages = torch.where(s["ended"] != 0, (lens + PS - 1) // PS, 0)
    mine = torch.arange(bt.shape[1], device=lens.device)[None] < pages[:, None]
    back = bt[mine]  # row by row
    n = s["count"].long() + torch.arange(back.numel(), device=lens.device)
    free[n] = back
    s["lens_out"].copy_(torch.where(s["ended"] != 0, 0, lens))
    s["count_out"].copy_(s["count"] + pages.sum())
    return {x: s[x] for x in ("free", "lens_out", "count_out")}


def _plain_bounds(s):
    start, bt = s["start"].long(), s["bt"].long()
    total = start + (s["cu"][1:] - s["cu"][:-1])
    p = torch.arange(bt.shape[1], device=start.device)[None]
    row, p = torch.nonzero((p >= start[:, None] // PS) & (p < (total[:, None] + PS - 1) // PS), as_tuple=True)
    page = bt[row, p]
    k = s["k_pool"][page].float()
    out = (p[:, None] * PS + torch.arange(PS, device=p.device)[None] >= total[row][:, None])[:, :, None, None]
    low, top = k.masked_fill(out, math.inf).amin(1), k.masked_fill(out, -math.inf).amax(1)
    s["bounds"][page] = torch.stack((low, top), 2).half()
    return {"bounds": s["bounds"]}


def _plain_sparse(s):
    q, lens, case, pages = s["q"], s["lens"].long(), s["case"], s["bt"].shape[1]
    b, hq, hkv, k = q.shape[0], q.shape[1], case["hkv"], case["select"]
    g = hq // hkv
    bt = s["bt"].clamp(min=0).long()
    bd = s["bounds"][bt].double().permute(0, 2, 3, 4, 1)  # [b, hkv, 2, D, pages]
    qd = q.double().view(b, hkv, g, D)
    score = (torch.matmul(qd.clamp(max=0), bd[:, :, 0]) + torch.matmul(qd.clamp(min=0), bd[:, :, 1])).amax(2)  # [b, hkv, pages]
    del bd
    count = ((lens + PS - 1) // PS)[:, None, None]
    p = torch.arange(pages, device=q.device)[None, None]
    score = torch.where(p == count - 1, math.inf, torch.where(p < count, score, -math.inf))
    first = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :k]
    first = torch.where(torch.arange(first.shape[-1], device=q.device)[None, None] < count, first, pages)
    first = torch.sort(first, -1).values
    s["pages"].fill_(-1)
    s["pages"][..., : first.shape[-1]] = torch.where(first < pages, first, -1).to(torch.int32)
    phys = torch.gather(bt[:, None].expand(b, hkv, pages), 2, first.clamp(max=pages - 1))
    head = torch.arange(hkv, device=q.device)[None, :, None]
    kk = s["k_pool"][phys, :, head].float().view(b, hkv, -1, D)  # [b, hkv, selected * PS, D]
    vv = s["v_pool"][phys, :, head].float().view(b, hkv, -1, D)
    x = torch.matmul(q.float().view(b, hkv, g, D), kk.transpose(2, 3)).mul_(s["scale"])
    at = (first[..., None] * PS + torch.arange(PS, device=q.device)).view(b, hkv, 1, -1)
    x.masked_fill_(at >= lens[:, None, None, None], -math.inf)
    x.sub_(x.amax(-1, keepdim=True)).exp_()
    return {"pages": s["pages"], "out": (torch.matmul(x, vv) / x.sum(-1, keepdim=True)).view(b, hq, D).half()}


# -------------------------------------------------------------------------------------------------------------- run
def run(s):
    op = s["case"]["op"]
    if own:
        return _own(s, op)
    if op == "chunk":
        return _plain_chunk(s)
    if op == "tables":
        return _plain_grow(s) if s["case"]["kind"] == "grow" else _plain_release(s)
    return _plain_bounds(s) if op == "bounds" else _plain_sparse(s)


def _own(s, op):
    import serving_paged_gqa_gb300 as pkv

    ws = s.get("ws")
    if ws is None:  # a program allocates its workspace once
        need = pkv.PKV_PROMPT_WS_BYTES
        if op == "chunk":
            need = pkv.pkv_chunk_workspace_bytes()
        elif op == "sparse":
            need = pkv.pkv_sparse_workspace_bytes(pkv.sparse_problem(s["q"], s["k_pool"], s["bt"]))
        ws = s["ws"] = pkv.alloc_workspace(need)
    if op == "chunk":
        return {"out": pkv.chunk_attention(s["q"], s["k_pool"], s["v_pool"], s["cu"], s["bt"], start=s["start"], scale=s["scale"], out=s["out"], ws=ws)}
    if op == "tables" and s["case"]["kind"] == "grow":
        pkv.tables_grow(s["new"], s["lens"], s["bt"], s["free"], s["count"], cu_seqlens=s["cu"], start=s["start"], slots=s["slots"],
                        positions=s["positions"], seq_lens_out=s["lens_out"], free_count_out=s["count_out"], ws=ws)
        return {x: s[x] for x in ("bt", "cu", "start", "slots", "positions", "lens_out", "count_out")}
    if op == "tables":
        pkv.tables_release(s["ended"], s["lens"], s["bt"], s["free"], s["count"], seq_lens_out=s["lens_out"], free_count_out=s["count_out"], ws=ws)
        return {x: s[x] for x in ("free", "lens_out", "count_out")}
    if op == "bounds":
        return {"bounds": pkv.page_bounds(s["k_pool"], s["cu"], s["bt"], s["bounds"], start=s["start"], ws=ws)}
    pages = pkv.select_pages(s["q"], s["bounds"], s["bt"], s["lens"], s["case"]["select"], pages=s["pages"], ws=ws)
    out = pkv.sparse_decode(s["q"], s["k_pool"], s["v_pool"], s["bt"], s["lens"], pages, scale=s["scale"], out=s["out"], ws=ws)
    return {"pages": pages, "out": out}


# ---------------------------------------------------------------------------------------------------- 64-bit values
def _attend(q, k, v, scale, first):
    """q [m, hq, d] at positions first..first+m-1 over k, v [n, hkv, d], one query head at a time."""
    g = q.shape[1] // k.shape[1]
    out = torch.empty(q.shape, dtype=torch.float64, device=q.device)
    seen = torch.arange(k.shape[0], device=q.device)[None] <= first + torch.arange(q.shape[0], device=q.device)[:, None]
    for h in range(q.shape[1]):
        w = torch.softmax(((q[:, h].double() @ k[:, h // g].double().T) * scale).masked_fill(~seen, -math.inf), -1)
        out[:, h] = w @ v[:, h // g].double()
    return out


def _exact_tables(s, case, new, start):
    """Row after row, page after page, as a program on the host would keep its tables."""
    bt, free, count = s["bt"].cpu().tolist(), s["free"].cpu().tolist(), int(s["count"])
    i32, dev = torch.int32, s["bt"].device

    def whole(x, like):
        return torch.tensor(x, dtype=like.dtype).to(dev)

    if case["kind"] == "release":
        lens = list(start)
        for b in range(0, len(lens), 2):
            for p in range(_pages_of(lens[b])):
                free[count] = bt[b][p]
                count += 1
            lens[b] = 0
        return {"free": whole(free, s["free"]), "lens_out": whole(lens, s["lens"]), "count_out": whole([count], s["count"])}
    slots, positions, cu = [], [], [0]
    for b, (m, at) in enumerate(zip(new, start)):
        for pos in range(at, at + m):
            if bt[b][pos // PS] < 0:
                count -= 1
                bt[b][pos // PS] = free[count]
            slots.append(bt[b][pos // PS] * PS + pos % PS)
            positions.append(pos)
        cu.append(cu[-1] + m)
    rest = [-1] * 5
    return {"bt": whole(bt, s["bt"]), "cu": whole(cu, s["cu"]), "start": whole(start, s["start"]), "slots": whole(slots + rest, s["slots"]),
            "positions": whole(positions + rest, s["positions"]), "lens_out": torch.tensor([x + y for x, y in zip(new, start)], dtype=i32).to(dev),
            "count_out": whole([count], s["count"])}


def exact(case, seed):
    s = prepare(case, seed)
    (new, start), op = _lens(case), case["op"]
    if op == "tables":
        return _exact_tables(s, case, new, start)
    bt = s["bt"].long()
    if op == "bounds":
        out = s["bounds"].double()
        for b, (m, at) in enumerate(zip(new, start)):
            for p in range(at // PS, _pages_of(at + m)):
                page = s["k_pool"][bt[b, p], : min(PS, at + m - p * PS)].double()
                out[bt[b, p], :, 0], out[bt[b, p], :, 1] = page.min(0).values, page.max(0).values
        return {"bounds": out}
    if op == "chunk":
        out, row = [], 0
        for b, (m, at) in enumerate(zip(new, start)):
            pages = bt[b, : _pages_of(at + m)]
            k, v = (s[x][pages].flatten(0, 1)[: at + m] for x in ("k_pool", "v_pool"))
            for i in range(0, m, 2048):
                r = min(2048, m - i)
                out.append(_attend(s["q"][row + i:row + i + r], k[: at + i + r], v[: at + i + r], s["scale"], at + i))
            row += m
        return {"out": torch.cat(out)}
    hq, hkv, sel = case["hq"], case["hkv"], case["select"]
    g = hq // hkv
    pages = np.full((len(start), hkv, sel), -1, dtype=np.int32)
    out = torch.empty((len(start), hq, D), dtype=torch.float64, device=bt.device)
    for b, n in enumerate(start):
        count = _pages_of(n)
        for h in range(hkv):
            q = s["q"][b, h * g:(h + 1) * g].double()
            low, top = s["bounds"][bt[b, :count], h].double().unbind(1)  # [count, D] each
            best = torch.maximum(q[:, None] * low[None], q[:, None] * top[None]).sum(-1).amax(0).cpu().numpy()
            order = sorted(range(count - 1), key=lambda p: (-best[p], p))[: sel - 1]
            mine = sorted(order) + [count - 1]
            pages[b, h, : len(mine)] = mine
            keys = torch.tensor([p * PS + i for p in mine for i in range(PS) if p * PS + i < n], device=bt.device)
            k, v = (s[x][bt[b, keys // PS], keys % PS, h].double() for x in ("k_pool", "v_pool"))
            out[b, h * g:(h + 1) * g] = torch.softmax((q @ k.T) * s["scale"], -1) @ v
    return {"pages": torch.from_numpy(pages).to(bt.device), "out": out}
