"""Plain 64-bit forms of the prompt and 4-bit-cache operators, on the tensors' device, with the error bounds that the
kernels' roundings allow."""

from __future__ import annotations

import math

import torch

D, PS, BLOCK = 128, 16, 2304
HALF_STEP = 2.0 ** -11  # fp16: a rounding is off by at most half a step, relative to the value
TINY = 2.0 ** -25       # ... and by half the least subnormal


def attend(q, k, v, scale, first):
    """q [m, Hq, d] at positions first.. over k, v [n, Hkv, d]: out and sum_j p_j |v_j|, both [m, Hq, d] in 64 bits."""
    m, hq, _ = q.shape
    n, hkv, _ = k.shape
    g = hq // hkv
    s = torch.einsum("mhgd,nhd->hgmn", q.double().view(m, hkv, g, D), k.double()) * scale
    hide = torch.arange(n, device=q.device)[None] > first + torch.arange(m, device=q.device)[:, None]
    s.masked_fill_(hide, -math.inf)
    p = torch.softmax(s, -1)
    out = torch.einsum("hgmn,nhd->mhgd", p, v.double()).reshape(m, hq, D)
    mag = torch.einsum("hgmn,nhd->mhgd", p, v.double().abs()).reshape(m, hq, D)
    return out, mag


def prompt_bound(out, mag, n, q, k, v, scale):
    """Of the kernel's |error|. Scores: 128 products added in fp32, off by at most 128 * 2^-24 of the sum of their
    magnitudes, <= 128 |q| |k| scale; twice that is the relative error of a weight (numerator and sum). Weights are
    rounded to fp16 (half a step, or half the least subnormal next to a largest weight of 1); the output once."""
    if out.numel() == 0:
        return out
    ds = 2.0 ** -17 * float((q.double().norm(dim=-1).max() * k.double().norm(dim=-1).max()) * abs(scale)) * 2
    return HALF_STEP * out.abs() + (HALF_STEP + 2.0 ** -16 + ds) * mag + n * TINY * float(v.abs().max()) + TINY


def quantise(x):
    """x [..., 128] fp16 -> codes (uint8) [..., 128], scale, offset fp16 [..., 2] by the definition of include/pkv.h."""
    g = x.float().unflatten(-1, (2, 64))
    low, top = g.amin(-1), g.amax(-1)
    bad = ~torch.isfinite(g).all(-1)
    sc = ((top - low) / 15).half()
    s = sc.float()[..., None]
    c = torch.where(s > 0, torch.round((g - low[..., None]) / torch.where(s > 0, s, 1.0)).clamp(0, 15), 0.0)
    c = torch.where(bad[..., None], 0.0, c)
    nan = torch.full_like(sc, math.nan)
    return c.to(torch.uint8).flatten(-2), torch.where(bad, nan, sc), torch.where(bad, nan, low.half())


def values(c, sc, off):
    """What codes stand for, in 64 bits (exact)."""
    return (c.double().unflatten(-1, (2, 64)) * sc.double()[..., None] + off.double()[..., None]).flatten(-2)


def _byte_maps(dev):
    r = torch.arange(PS, device=dev)[:, None]
    d = torch.arange(64, device=dev)[None]
    inner = (d // 16) * 4 + d // 8 % 2
    k = r * 64 + (d // 2 % 4) * 16 + inner + 2 * (d % 2)
    v = (r // 8) * 512 + (d % 8) * 64 + (r // 2 % 4) * 16 + inner + 2 * (r % 2)
    return k, v


def put_tokens(pool, bt_row, pos, k, v):
    """Writes tokens k, v [n, Hkv, 128] fp16 at positions pos [n] of one row into a 4-bit pool, byte by byte."""
    dev = pool.device
    hkv = pool.shape[1]
    page, slot = bt_row[pos // PS].long(), pos % PS
    maps = _byte_maps(dev)
    h = torch.arange(hkv, device=dev)
    for x, base, bytes_of in ((k, 0, maps[0]), (v, 1152, maps[1])):
        c, sc, off = quantise(x)
        packed = c[..., :64] | (c[..., 64:] << 4)  # [n, hkv, 64]
        pool[page[:, None, None], h[None, :, None], base + bytes_of[slot][:, None, :]] = packed
        par = torch.stack((sc, off), -1).flatten(-2).contiguous().view(torch.uint8).view(-1, hkv, 8)
        at = base + 1024 + slot[:, None] * 8 + torch.arange(8, device=dev)[None]
        pool[page[:, None, None], h[None, :, None], at[:, None, :]] = par


def get_tokens(pool, bt_row, pos):
    """Tokens at positions pos [n] of one row: (codes, scale, offset) of K and of V."""
    dev = pool.device
    h = torch.arange(pool.shape[1], device=dev)
    page, slot = bt_row[pos // PS].long(), pos % PS
    both = []
    for base, bytes_of in zip((0, 1152), _byte_maps(dev)):
        packed = pool[page[:, None, None], h[None, :, None], base + bytes_of[slot][:, None, :]]
        at = base + 1024 + slot[:, None] * 8 + torch.arange(8, device=dev)[None]
        par = pool[page[:, None, None], h[None, :, None], at[:, None, :]].contiguous().view(torch.float16)
        par = par.view(len(pos), pool.shape[1], 2, 2)
        both.append((torch.cat((packed & 15, packed >> 4), -1), par[..., 0], par[..., 1]))
    return both


def q4_row(q, pool, bt_row, n, scale):
    """Decode of one row of n tokens over a 4-bit pool: out [Hq, d] in 64 bits and the bound of the kernel's error."""
    hq = q.shape[0]
    if n == 0:
        z = torch.zeros((hq, D), dtype=torch.float64, device=q.device)
        return z, z
    (kc, ks, ko), (vc, vs, vo) = get_tokens(pool, bt_row, torch.arange(n, device=pool.device))
    k, v = values(kc, ks, ko), values(vc, vs, vo)
    out, _ = attend(q[None], k, v, scale, n - 1)
    # Scores: scale * code products and offset * sum(q), each summed in fp32: 2^-24 for each of at most 140 steps of the
    # sum of magnitudes. Weights times scale are two fp16 parts (2^-21, or half the least subnormal next to a largest of
    # 1); their products with the codes are added by the matrix instructions, 16 tokens a time, which may cut each sum
    # to 24 bits: 2^-23 of the running sum a time, at most n / 16 times; the offsets' part stays in fp32.
    parts = values(kc, ks, torch.zeros_like(ko)).abs() + ko.double().abs().repeat_interleave(64, -1)
    ds = 2 * 140 * 2.0 ** -24 * abs(scale) * float((q.double().abs().sum(-1)).max() * parts.max())
    _, coded = attend(q[None], k, values(vc, vs, torch.zeros_like(vo)), scale, n - 1)
    _, offs = attend(q[None], k, vo.double().repeat_interleave(64, -1), scale, n - 1)
    bound = HALF_STEP * out.abs() + (2.0 ** -15 + ds + (n // 16 + 1) * 2.0 ** -23) * (coded + offs)
    return out[0], (bound + 15 * n * TINY * float(vs.double().max()) * 2.0 ** -7 + TINY)[0]


def check(got, want, bound, what=""):
    got = got.double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert torch.isfinite(got).all(), f"{what}: non-finite output"
    over = (got - want).abs() - bound
    i = int(over.argmax())
    assert float(over.flatten()[i]) <= 0, (f"{what}: off by {float((got - want).abs().flatten()[i]):.3e} at {i} "
                                           f"(value {float(want.flatten()[i]):.4e}, bound {float(bound.flatten()[i]):.3e})")
