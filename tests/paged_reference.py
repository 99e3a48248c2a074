"""Sequences in paged caches for the tests, and what the calls over them should give, in 64 bits."""

from __future__ import annotations

import math

import torch

import prompt_reference as ref

D, PS = 128, 16


class Cache:
    """FP16 pools whose unused slots and pages are NaN, a block table whose unused entries are outside the pool, and packed
    queries of new tokens: sequence s holds start[s] tokens and gets new[s] more, which the pools hold already."""

    def __init__(self, new, start, hq, hkv, seed=0, dev="cuda", fused=False, spread=1.0, poison=math.nan, spare=5, behind=3):
        g = torch.Generator(device=dev).manual_seed(seed)
        self.new, self.start, self.hq, self.hkv = list(new), list(start), hq, hkv
        total = [a + b for a, b in zip(new, start)]
        n = [-(-x // PS) for x in total]
        self.num_pages = sum(n) + spare
        perm = torch.randperm(self.num_pages, generator=g, device=dev).to(torch.int32)
        self.bt = torch.full((len(new), max(n + [0]) + 1), -(1 << 30), dtype=torch.int32, device=dev)
        self.bt[:, -1] = 1 << 30
        self.k, self.v = (torch.full((self.num_pages, PS, hkv, D), poison, dtype=torch.float16, device=dev) for _ in range(2))
        at = 0
        for s, x in enumerate(total):
            self.bt[s, : n[s]] = perm[at:at + n[s]]
            at += n[s]
            pos = torch.arange(x, device=dev)
            page = self.bt[s, pos // PS].long()
            self.k[page, pos % PS] = (torch.randn((x, hkv, D), generator=g, device=dev) * spread).half()
            self.v[page, pos % PS] = torch.randn((x, hkv, D), generator=g, device=dev).half()
        self.tokens = sum(new)
        wide = torch.randn((self.tokens + behind, hq + (2 * hkv if fused else 0), D), generator=g, device=dev).half()
        wide[self.tokens:] = math.nan  # rows of no sequence
        self.q = wide[:, :hq]
        self.cu = torch.tensor([sum(new[:i]) for i in range(len(new) + 1)], dtype=torch.int32, device=dev)
        self.st = torch.tensor(start, dtype=torch.int32, device=dev)
        self.lens = torch.tensor(total, dtype=torch.int32, device=dev)
        self.scale = 1.0 / math.sqrt(D)

    def rows(self, s, n):
        """K and V of row s's first n tokens [n, Hkv, d]; tokens of pages outside the pool are 0."""
        pos = torch.arange(n, device=self.bt.device)
        page = self.bt[s, pos // PS].long()
        bad = (page < 0) | (page >= self.num_pages)
        page = page.clamp(0, self.num_pages - 1)
        return (torch.where(bad[:, None, None], torch.zeros_like(x[page, pos % PS]), x[page, pos % PS]) for x in (self.k, self.v))

    def attend(self):
        """out of every packed token and the bound of the kernel's error, in 64 bits."""
        outs, bounds = [], []
        for s, (m, st) in enumerate(zip(self.new, self.start)):
            if m == 0:
                continue
            k, v = self.rows(s, st + m)
            at = int(self.cu[s])
            for i in range(0, m, 512):
                r = min(512, m - i)
                q, n = self.q[at + i:at + i + r], st + i + r
                out, mag = ref.attend(q, k[:n], v[:n], self.scale, st + i)
                outs.append(out)
                bounds.append(chunk_bound(out, mag, n, q, k[:n], v[:n], self.scale))
        return torch.cat(outs), torch.cat(bounds)


def chunk_bound(out, mag, n, q, k, v, scale):
    """Of the kernel's |error|: as for prompts (prompt_reference.prompt_bound); the sums over n keys are made by matrix
    instructions, 16 keys a time, which may cut each sum to 24 bits: 2^-23 of the sum of magnitudes a time, twice that for the
    numerator and the rounding of the sum of weights; states of pieces are added with factors of a relative error of 2^-22."""
    return ref.prompt_bound(out, mag, n, q, k, v, scale) + ((n // 16 + 1) * 2.0 ** -22 + 2.0 ** -20) * mag
