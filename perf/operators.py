"""The prompt and 4-bit-cache operators as a user's program calls them, beside their plain forms.

``own`` False: every operator in elementary torch operations in 32 bits, rounded once at the end. ``own`` True: the
calls of this repository's library. ``exact`` gives the same outputs from the definitions in 64 bits.

Operators (``op`` of a case):
  prompt    causal grouped-query attention over packed prompts of different lengths
  pages     the packed prompts' K/V written into the FP16 page pools
  pages4    the packed prompts' K/V quantised into 4-bit pages and read back as the values they stand for
  decode4   one decode step over the 4-bit pages (with ``append``: the new token's K/V quantised into its slot first;
            the appended tokens are read back and returned too)

4-bit pages: for each (page, KV head) one block of 2304 bytes: K codes (1024), K scale / offset (16 tokens x 2 groups
of 64 dims x 2 fp16), V codes (1024), V scale / offset. A byte holds dim d in its low and dim d + 64 in its high 4 bits.
"""

import math
import random

import numpy as np
import torch

own = False

D, PS, BLOCK = 128, 16, 2304


# ------------------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # a chat turn of a few tokens: the smallest prompt, latency counts
        dict(name="prompt one short", op="prompt", seqs=1, lo=17, hi=17, lseed=0, hq=32, hkv=8, fused=False),
        # a batch of short, ragged prompts, q/k/v as slices of one fused projection, eight heads to a KV head
        dict(name="prompt short batch", op="prompt", seqs=16, lo=5, hi=300, lseed=1, hq=32, hkv=4, fused=True),
        # an ordinary document
        dict(name="prompt 2048", op="prompt", seqs=1, lo=2048, hi=2048, lseed=0, hq=32, hkv=8, fused=True),
        # a prefill batch of different lengths
        dict(name="prompt ragged batch", op="prompt", seqs=6, lo=500, hi=8192, lseed=2, hq=32, hkv=8, fused=False),
        # the longest prompt
        dict(name="prompt long", op="prompt", seqs=1, lo=16384, hi=16384, lseed=0, hq=32, hkv=8, fused=False),
        # prompts into the FP16 pages: a batch after its prefill
        dict(name="pages batch", op="pages", seqs=8, lo=200, hi=4096, lseed=3, hkv=8, start=0, fused=True),
        # a few tokens behind others that the cache holds already (an odd start inside a page), quantised
        dict(name="pages4 few behind others", op="pages4", seqs=3, lo=7, hi=40, lseed=4, hkv=8, start=37, fused=True),
        # long prompts into the 4-bit pages
        dict(name="pages4 long", op="pages4", seqs=4, lo=8000, hi=16384, lseed=5, hkv=8, start=0, fused=True),
        # the smallest decode step: one row of 512 tokens
        dict(name="decode4 one row short", op="decode4", batch=1, lo=512, hi=512, lseed=0, hq=32, hkv=8, append=False),
        # one long-context row, the new token appended in the step
        dict(name="decode4 one row long", op="decode4", batch=1, lo=32768, hi=32768, lseed=0, hq=32, hkv=8, append=True),
        # eight rows of mixed lengths
        dict(name="decode4 eight rows", op="decode4", batch=8, lo=1024, hi=32768, lseed=6, hq=32, hkv=8, append=False),
        # a full serving batch
        dict(name="decode4 many rows", op="decode4", batch=48, lo=900, hi=32768, lseed=7, hq=32, hkv=8, append=True),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "pages", "pages4", "decode4", "decode4"])
    g = rng.choice([1, 2, 4, 8, 16])
    hkv = rng.choice([h for h in (1, 2, 4, 8) if h * g <= 32])
    lseed = rng.randrange(1 << 20)
    if op == "decode4":
        hi = _spread(rng, 16, 32768)
        batch = _spread(rng, 1, min(48, 700000 // hi))
        return dict(op=op, batch=batch, lo=rng.randint(1, hi), hi=hi, lseed=lseed, hq=hkv * g, hkv=hkv, append=rng.random() < 0.5)
    if op == "prompt":
        hi = _spread(rng, 1, 16384)
        seqs = _spread(rng, 1, max(1, min(32, (1 << 28) // (hi * hi))))
        return dict(op=op, seqs=seqs, lo=rng.randint(1, hi), hi=hi, lseed=lseed, hq=hkv * g, hkv=hkv, fused=rng.random() < 0.5)
    hi = _spread(rng, 1, 16384)
    return dict(op=op, seqs=_spread(rng, 1, max(1, min(32, 49152 // hi))), lo=rng.randint(1, hi), hi=hi, lseed=lseed, hkv=hkv,
                start=rng.choice([0, 0, rng.randint(1, 100)]), fused=rng.random() < 0.5)


def _lens(case):
    r = random.Random(case["lseed"])
    return [r.randint(case["lo"], case["hi"]) for _ in range(case["batch"] if case["op"] == "decode4" else case["seqs"])]


def work(case):
    lens = _lens(case)
    t, hkv = sum(lens), case["hkv"]
    if case["op"] == "prompt":
        return {"bytes": t * (2 * case["hq"] + 2 * hkv) * D * 2, "flops": sum(4 * D * case["hq"] * n * (n + 1) // 2 for n in lens)}
    if case["op"] == "pages":
        return {"bytes": t * hkv * 2 * 512, "flops": 0}
    if case["op"] == "pages4":  # K/V read, the blocks' share of these tokens written, read and dequantised
        return {"bytes": t * hkv * (512 + 144 + 144 + 512), "flops": t * hkv * 256 * 6}
    b = len(lens)
    extra = b * hkv * (512 + 144 + 144 + 512) if case["append"] else 0
    return {"bytes": t * hkv * 144 + b * case["hq"] * D * 4 + extra, "flops": 4 * D * case["hq"] * t}


# ----------------------------------------------------------------------------------------------------------- inputs
def _pages(lens, gen, dev):
    """A block table over a shuffled pool: row b's pages at random places, -1 behind them."""
    n = [(x + PS - 1) // PS for x in lens]
    perm = torch.randperm(sum(n) + 3, generator=gen, device=dev).to(torch.int32)
    bt = torch.full((len(lens), max(max(n), 1)), -1, dtype=torch.int32, device=dev)
    row = torch.repeat_interleave(torch.arange(len(n), device=dev), torch.tensor(n, device=dev))
    first = torch.tensor([sum(n[:i]) for i in range(len(n))], device=dev)
    at = torch.arange(sum(n), device=dev)
    bt[row, at - first[row]] = perm[: sum(n)]
    return bt, sum(n) + 3


def _k_bytes(c):
    """Codes [..., 16 tokens, 128 dims] (uint8) -> the 1024 bytes of a block's K codes."""
    b = c[..., :64] | (c[..., 64:] << 4)
    lead = b.shape[:-2]
    return b.reshape(*lead, 16, 4, 2, 4, 2).movedim((-4, -3, -2, -1), (-3, -1, -4, -2)).reshape(*lead, 1024)


def _v_bytes(c):
    b = c[..., :64] | (c[..., 64:] << 4)
    lead = b.shape[:-2]
    return b.reshape(*lead, 2, 4, 2, 4, 2, 8).movedim((-6, -5, -4, -3, -2, -1), (-6, -4, -2, -3, -1, -5)).reshape(*lead, 1024)


def _quantise(x):
    """x [..., 128] -> codes (uint8), scale and offset [..., 2] (fp16)."""
    x = x.float().unflatten(-1, (2, 64))
    off, top = x.amin(-1), x.amax(-1)
    sc = ((top - off) / 15).half()
    s = sc.float()
    c = torch.where(s[..., None] > 0, torch.round((x - off[..., None]) / torch.where(s > 0, s, 1.0)[..., None]).clamp(0, 15), 0.0)
    return c.to(torch.uint8).flatten(-2), sc, off.half()


def _blocks(x, to_bytes):
    """x [pages, 16, Hkv, 128] -> [pages, Hkv, 1152]: one half (K or V) of the blocks."""
    c, sc, off = _quantise(x.transpose(1, 2))
    par = torch.stack((sc, off), -1).flatten(-3).view(torch.uint8)
    return torch.cat((to_bytes(c), par.reshape(*par.shape[:2], 128)), -1)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    lens = _lens(case)
    op, hkv = case["op"], case["hkv"]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev).half()

    s = {"case": case, "scale": 1.0 / math.sqrt(D)}
    if op == "decode4":
        b, hq = len(lens), case["hq"]
        bt, num_pages = _pages(lens, gen, dev)
        pool = torch.empty((num_pages, hkv, BLOCK), dtype=torch.uint8, device=dev)
        step = max(1, (1 << 28) // (PS * hkv * D))
        for p in range(0, num_pages, step):
            n = min(step, num_pages - p)
            pool[p:p + n, :, :1152] = _blocks(normal(n, PS, hkv, D), _k_bytes)
            pool[p:p + n, :, 1152:] = _blocks(normal(n, PS, hkv, D), _v_bytes)
        s.update(q=normal(b, hq, D), pool=pool, bt=bt, lens=torch.tensor(lens, dtype=torch.int32, device=dev),
                 out=torch.empty((b, hq, D), dtype=torch.float16, device=dev))
        if case["append"]:
            s.update(k_new=normal(b, hkv, D), v_new=normal(b, hkv, D), last=s["lens"] - 1,
                     cu=torch.arange(b + 1, dtype=torch.int32, device=dev),
                     k_back=torch.empty((b, hkv, D), dtype=torch.float16, device=dev),
                     v_back=torch.empty((b, hkv, D), dtype=torch.float16, device=dev))
        return s
    t = sum(lens)
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    s["cu"] = torch.tensor(cu, dtype=torch.int32, device=dev)
    hq = case.get("hq", 0)
    if case["fused"]:  # slices of one [tokens, (Hq + 2 Hkv) * d] projection
        x = normal(t, hq + 2 * hkv, D)
        s["q"], s["k"], s["v"] = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    else:
        s["q"], s["k"], s["v"] = normal(t, hq, D), normal(t, hkv, D), normal(t, hkv, D)
    if op == "prompt":
        s["out"] = torch.empty((t, hq, D), dtype=torch.float16, device=dev)
        return s
    start = case["start"]
    s["bt"], num_pages = _pages([n + start for n in lens], gen, dev)
    s["start"] = torch.full((len(lens),), start, dtype=torch.int32, device=dev)
    if op == "pages":
        s["k_pool"] = torch.zeros((num_pages, PS, hkv, D), dtype=torch.float16, device=dev)
        s["v_pool"] = torch.zeros((num_pages, PS, hkv, D), dtype=torch.float16, device=dev)
    else:
        s["pool"] = torch.zeros((num_pages, hkv, BLOCK), dtype=torch.uint8, device=dev)
        s["k_back"] = torch.empty((t, hkv, D), dtype=torch.float16, device=dev)
        s["v_back"] = torch.empty((t, hkv, D), dtype=torch.float16, device=dev)
    return s


# ------------------------------------------------------------------------------------------------------ plain forms
def _rows(cu, t):
    """(sequence, position) of every packed token."""
    at = torch.arange(t, device=cu.device)
    seq = torch.searchsorted(cu[1:].contiguous(), at.to(torch.int32), right=True)
    return seq, at - cu[seq]


def _plain_prompt(s):
    q, k, v, cu = s["q"], s["k"], s["v"], s["cu"]
    t, hq, hkv = q.shape[0], q.shape[1], k.shape[1]
    b, n = s["case"]["seqs"], max(_lens(s["case"]))
    seq, pos = _rows(cu, t)

    def padded(x):
        y = torch.zeros((b, n, x.shape[1], D), dtype=torch.float32, device=x.device)
        y[seq, pos] = x.float()
        return y.transpose(1, 2)  # [b, h, n, d]

    qp = padded(q).reshape(b, hkv, (hq // hkv) * n, D)
    x = torch.matmul(qp, padded(k).transpose(2, 3)).view(b, hkv, hq // hkv, n, n).mul_(s["scale"])
    at = torch.arange(n, device=q.device)
    x.masked_fill_(at[None, :] > at[:, None], -math.inf)
    x.sub_(x.amax(-1, keepdim=True)).exp_()
    y = torch.matmul(x.view(b, hkv, -1, n), padded(v)).view(b, hq, n, D) / x.sum(-1).view(b, hq, n, 1)
    return y.transpose(1, 2)[seq, pos].half()


def _plain_pages(s):
    seq, pos = _rows(s["cu"], s["k"].shape[0])
    pos = pos + s["start"][seq]
    page = s["bt"][seq, pos // PS].long()
    s["k_pool"][page, pos % PS] = s["k"]
    s["v_pool"][page, pos % PS] = s["v"]
    return {"k_pool": s["k_pool"], "v_pool": s["v_pool"]}


def _stands_for(x):
    """The values that the 4-bit form of x stands for, in 32 bits."""
    c, sc, off = _quantise(x)
    return (c.float().unflatten(-1, (2, 64)) * sc.float()[..., None] + off.float()[..., None]).flatten(-2)


def _plain_decode4(s):
    case, q, lens = s["case"], s["q"], s["lens"]
    b, hq, hkv = q.shape[0], q.shape[1], case["hkv"]
    blk = s["pool"][s["bt"].clamp(min=0).long()].transpose(1, 2)  # [b, hkv, pages, 2304]
    pages = blk.shape[2]

    def half(x, v):
        y = x[..., :1024]
        if v:
            y = y.unflatten(-1, (2, 8, 4, 4, 2, 2)).movedim((-6, -5, -4, -3, -2, -1), (-6, -1, -5, -3, -4, -2))
        else:
            y = y.unflatten(-1, (16, 4, 4, 2, 2)).movedim((-4, -3, -2, -1), (-2, -4, -1, -3))
        y = y.reshape(b, hkv, pages, PS, 64)
        c = torch.stack((y & 15, y >> 4), -2).float()  # [..., 16, 2 groups, 64]
        par = x[..., 1024:].contiguous().view(torch.float16).float().view(b, hkv, pages, PS, 2, 2)
        return c.mul_(par[..., :1]).add_(par[..., 1:]).reshape(b, hkv, pages * PS, D)

    k, v = half(blk[..., :1152], False), half(blk[..., 1152:], True)
    more = {}
    if case["append"]:
        kn, vn, row, last = _stands_for(s["k_new"]), _stands_for(s["v_new"]), torch.arange(b, device=q.device), s["last"].long()
        k[row, :, last], v[row, :, last] = kn, vn
        more = {"k_back": kn.half(), "v_back": vn.half()}
    x = torch.matmul(q.float().view(b, hkv, hq // hkv, D), k.transpose(2, 3)).mul_(s["scale"])
    x.masked_fill_((torch.arange(pages * PS, device=q.device)[None] >= lens[:, None])[:, None, None], -math.inf)
    x.sub_(x.amax(-1, keepdim=True)).exp_()
    y = torch.matmul(x, v) / x.sum(-1, keepdim=True)
    return {"out": y.view(b, hq, D).half(), **more}


# -------------------------------------------------------------------------------------------------------------- run
def run(s):
    op = s["case"]["op"]
    if own:
        return _own(s, op)
    if op == "prompt":
        return _plain_prompt(s)
    if op == "pages":
        return _plain_pages(s)
    if op == "pages4":
        return {"k": _stands_for(s["k"]).half(), "v": _stands_for(s["v"]).half()}
    return _plain_decode4(s)


def _own(s, op):
    import serving_paged_gqa_gb300 as pkv

    ws = s.get("ws")
    if ws is None:  # a program allocates its workspace once
        if op == "decode4":
            b, hq, _ = s["q"].shape
            ws = pkv.alloc_workspace(pkv.pkv_q4_workspace_bytes(pkv.q4_problem(s["q"], s["pool"], s["bt"])))
        else:
            ws = pkv.alloc_workspace(pkv.PKV_PROMPT_WS_BYTES)
        s["ws"] = ws
    if op == "prompt":
        return pkv.prompt_attention(s["q"], s["k"], s["v"], s["cu"], scale=s["scale"], out=s["out"], ws=ws)
    if op == "pages":
        pkv.prompt_append(s["k"], s["v"], s["cu"], s["k_pool"], s["v_pool"], s["bt"], start=s["start"], ws=ws)
        return {"k_pool": s["k_pool"], "v_pool": s["v_pool"]}
    if op == "pages4":
        pkv.q4_prompt_append(s["k"], s["v"], s["cu"], s["pool"], s["bt"], start=s["start"], ws=ws)
        k, v = pkv.q4_read(s["cu"], s["pool"], s["bt"], start=s["start"], k_out=s["k_back"], v_out=s["v_back"], ws=ws)
        return {"k": k, "v": v}
    if not s["case"]["append"]:
        return {"out": pkv.q4_decode(s["q"], s["pool"], s["bt"], s["lens"], scale=s["scale"], out=s["out"], ws=ws)}
    out = pkv.q4_decode(s["q"], s["pool"], s["bt"], s["lens"], k_new=s["k_new"], v_new=s["v_new"], scale=s["scale"], out=s["out"], ws=ws)
    k, v = pkv.q4_read(s["cu"], s["pool"], s["bt"], start=s["last"], k_out=s["k_back"], v_out=s["v_back"], ws=ws)
    return {"out": out, "k_back": k, "v_back": v}


# ---------------------------------------------------------------------------------------------------- 64-bit values
def _exact4(x):
    """[tokens, heads, 128] -> the 4-bit values in 64 bits, from the definition."""
    y = x.double().reshape(*x.shape[:-1], 2, 64)
    low = y.min(-1, keepdim=True).values
    step = ((y.max(-1, keepdim=True).values - low) / 15).half().double()
    c = torch.nan_to_num((y - low) / step, nan=0.0, posinf=0.0).round().clamp(0, 15)
    return (low + c * step).reshape(x.shape)


def _attend(q, k, v, scale, first):
    """q [m, hq, d] at positions first..first+m-1 over k, v [n, hkv, d], one KV head at a time."""
    g = q.shape[1] // k.shape[1]
    out = torch.empty(q.shape, dtype=torch.float64, device=q.device)
    seen = torch.arange(k.shape[0], device=q.device)[None] <= first + torch.arange(q.shape[0], device=q.device)[:, None]
    for h in range(q.shape[1]):
        w = torch.softmax(((q[:, h].double() @ k[:, h // g].double().T) * scale).masked_fill(~seen, -math.inf), -1)
        out[:, h] = w @ v[:, h // g].double()
    return out


def _exact_cache(blk, n):
    """One row's blocks [pages, hkv, 2304] -> k, v [n, hkv, 128] in 64 bits, byte by byte from the layout."""
    i = np.arange(1024)
    t, ks, j = (i // 16) % 4, (i // 4) % 4, i % 4
    k_tok, k_dim = i // 64, 16 * ks + 2 * t + 8 * (j % 2) + j // 2
    v_tok, v_dim = 8 * (i // 512) + 2 * t + j // 2, 16 * ks + (i // 64) % 8 + 8 * (j % 2)
    both = []
    for at, tok, dim in ((0, k_tok, k_dim), (1152, v_tok, v_dim)):
        par = blk[..., at + 1024:at + 1152].contiguous().view(torch.float16).double().view(*blk.shape[:2], PS, 2, 2)
        tok, dim = torch.from_numpy(tok).to(blk.device), torch.from_numpy(dim).to(blk.device)
        x = torch.empty((blk.shape[0], PS, blk.shape[1], D), dtype=torch.float64, device=blk.device)
        code = blk[..., at:at + 1024]
        x[:, tok, :, dim] = ((code & 15).double() * par[:, :, tok, 0, 0] + par[:, :, tok, 0, 1]).permute(2, 0, 1)
        x[:, tok, :, dim + 64] = ((code >> 4).double() * par[:, :, tok, 1, 0] + par[:, :, tok, 1, 1]).permute(2, 0, 1)
        both.append(x.flatten(0, 1)[:n])
    return both


def exact(case, seed):
    s = prepare(case, seed)
    lens, op = _lens(case), case["op"]
    if op == "pages":
        for b, n in enumerate(lens):
            at = np.arange(n) + case["start"]
            page, slot = s["bt"][b].cpu().numpy()[at // PS], at % PS
            first = int(s["cu"][b])
            for name in ("k", "v"):
                s[name + "_pool"].view(-1, *s[name].shape[1:])[torch.from_numpy(page.astype(np.int64) * PS + slot).to(s["k"].device)] = s[name][first:first + n]
        return {"k_pool": s["k_pool"].double(), "v_pool": s["v_pool"].double()}
    if op == "pages4":
        return {"k": _exact4(s["k"]), "v": _exact4(s["v"])}
    if op == "prompt":
        out, at = [], 0
        for n in lens:
            part = slice(at, at + n)
            for i in range(0, n, 4096):  # rows in pieces
                m = min(4096, n - i)
                out.append(_attend(s["q"][part][i:i + m], s["k"][part][:i + m], s["v"][part][:i + m], s["scale"], i))
            at += n
        return torch.cat(out)
    back = {}
    if case["append"]:
        back = {"k_back": _exact4(s["k_new"]), "v_back": _exact4(s["v_new"])}
    rows = []
    for b, n in enumerate(lens):
        k, v = _exact_cache(s["pool"][s["bt"][b, :(n + PS - 1) // PS].long()], n)
        if back:
            k[-1], v[-1] = back["k_back"][b], back["v_back"][b]
        rows.append(_attend(s["q"][b:b + 1], k, v, s["scale"], n - 1))
    return {"out": torch.cat(rows), **back}
