"""Inputs and plain 64-bit results (torch on the host) for block-scaled E4M3 pools and for norms with the rotation."""
from __future__ import annotations

import math

import numpy as np
import torch

from spec_helpers import TYPES, rope_reference

TOP, EDGE, LEAST = 448.0, 464.0, 2.0 ** -126


def values(codes):
    return codes.view(torch.float8_e4m3fn).double()


def codes_of(x):
    """The nearest codes of f32 values: ties to even, saturating, NaN stays."""
    return x.clamp(-TOP, TOP).to(torch.float8_e4m3fn).view(torch.uint8)


class BlockPaged:
    """A shuffled paged cache of codes with block scales on the host; NaN codes and scales where no request has rows."""

    def __init__(self, kv, hk, d, page, block, new=None, seed=0, extra=3, magnitude=1.0):
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.kv, self.new, self.page, self.block = list(kv), list(new or [1] * len(kv)), page, block
        n = [-(-x // page) for x in kv]
        self.total = sum(n) + extra
        self.indices = rng.permutation(self.total)[:sum(n)].astype(np.int32)
        self.indptr = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        self.last = np.array([x - (m - 1) * page if m else 0 for x, m in zip(kv, n)], np.int32)
        self.new_indptr = np.concatenate([[0], np.cumsum(self.new)]).astype(np.int32)
        shape = (self.total, hk, page, d)
        self.k, self.v = (codes_of(torch.randn(shape, generator=g) * 60) for _ in range(2))
        self.k_scale, self.v_scale = (magnitude * torch.exp2(4 * torch.rand(self.total, hk, page // block, generator=g) - 8)
                                      for _ in range(2))
        rows = torch.zeros(self.total, page, dtype=torch.bool)
        for b in range(len(self.kv)):
            p, r = self.rows(b, np.arange(self.kv[b]))
            rows[p, r] = True
        dead = ~rows.view(self.total, page // block, block).any(-1)  # blocks without a row
        for x, s in ((self.k, self.k_scale), (self.v, self.v_scale)):
            x.permute(0, 2, 1, 3)[~rows] = 0x7F
            s.permute(0, 2, 1)[dead] = math.nan

    def rows(self, b, tokens):
        tokens = np.asarray(tokens, np.int64)
        return (torch.from_numpy(self.indices[self.indptr[b] + tokens // self.page].astype(np.int64)),
                torch.from_numpy(tokens % self.page))

    def held(self, b, tokens=None):
        """K, V [tokens, heads, dim] of request b, in 64 bits."""
        p, r = self.rows(b, np.arange(self.kv[b]) if tokens is None else tokens)
        return tuple(values(x[p, :, r]) * s[p, :, r // self.block].double()[..., None]
                     for x, s in ((self.k, self.k_scale), (self.v, self.v_scale)))

    def dense(self, b):
        return self.held(b)

    def table(self, device="cuda"):
        return tuple(torch.from_numpy(x).to(device) for x in (self.indices, self.indptr, self.last))

    def pools(self, device="cuda"):
        """k, v, k_scale, v_scale"""
        return tuple(x.to(device) for x in (self.k, self.v, self.k_scale, self.v_scale))


def norm_reference(x, weight, eps):
    y = x.double()
    y = y / (y.square().mean(-1, keepdim=True) + eps).sqrt()
    return y if weight is None else y * weight.double()


def norm_rope_reference(x, weight, eps, positions, inv_freq, layout, scale=1.0):
    y = norm_reference(x, weight, eps) if eps else x.double()
    return rope_reference(y, positions, inv_freq, layout, scale) if len(inv_freq) else y


def norm_rope_tolerance(ref, normed, dtype, scale=1.0):
    """Half a step of the type; and of each of a rotation's two products: the norm's sum of up to 256 squares (up to 20
    roundings one after another), reciprocal root (2^-22) and weight, 1.25 2^-20 in all, and the rotation's 1.5 2^-22."""
    half = torch.finfo(TYPES[dtype]).eps / 2 if dtype else 0.0
    return half * ref.abs() + 3.25 * 2.0 ** -20 * max(1.0, abs(scale)) * normed.abs().amax(-1, keepdim=True) + 1e-12


def append_reference(c, which, b, new, exact):
    """What request b's blocks hold after `new` [n, heads, dim] (64 bits) became its last rows.

    Returns (scales by block [blocks, heads] f32, first block's token, older rows' codes [lead, heads, dim]). exact: the
    scales are those of f32 values `new` (no tolerance needed).
    """
    n, block = new.shape[0], c.block
    ctx = c.kv[b] - n
    first = ctx // block * block
    lead = ctx - first
    pool, scale = getattr(c, which), getattr(c, which + "_scale")
    mags = torch.where(torch.isfinite(new), new.abs(), torch.zeros_like(new)).amax(-1)  # [n, heads]
    out, older = [], torch.empty(0)
    for t0 in range(first, c.kv[b], block):
        rows = mags[max(0, t0 - ctx):t0 + block - ctx]
        top = rows.amax(0)
        if t0 < ctx:
            p, r = c.rows(b, np.arange(t0, ctx))
            was = scale[p[0], :, r[0] // block].double().clamp(min=LEAST)
            up = torch.ceil(torch.log2(top / (EDGE * was))).clamp(min=0)
            older = codes_of((values(pool[p, :, r]) * torch.exp2(-up)[:, None]).float())
            out.append((was * torch.exp2(up)).float())
        else:
            out.append(torch.clamp((top.float() / np.float32(TOP)), min=LEAST))
    return torch.stack(out) if out else torch.empty(0), first, lead, older
