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


def attend_reference(c, q, masks, sm_scale, dtype):
    """(o, lse, tolerance of o, tolerance of lse) in 64 bits, from attended tokens alone. masks[b] [n, n] booleans; None: a
    chain.

    Tolerance of o, per output: half a step of the type for the result; of each weight, its two E4M3 parts (4 significant
    bits each: 2^-8) and its step through f16 (2^-11); 2^-14, half a step of a subnormal code of the second part, where the
    largest weight times V scale is 2^2.5 or more; and its score's error, in f32 sums and the
    exponential (1e-5) and where a small element of q falls between codes: 2^-10 of q's codes, whose largest is 128 or more.
    """
    total, hq, d = q.shape
    hk = c.k.shape[1]
    g = hq // hk
    half = torch.finfo(TYPES[dtype]).eps / 2
    o, tol = torch.zeros(total, hq, d, dtype=torch.float64), torch.zeros(total, hq, d, dtype=torch.float64)
    lse, tol_l = torch.full((total, hq), -math.inf, dtype=torch.float64), torch.zeros(total, hq, dtype=torch.float64)
    for b, n in enumerate(c.new):
        if n == 0 or c.kv[b] == 0:
            continue
        k, v = c.held(b)
        p, r = c.rows(b, np.arange(c.kv[b]))
        vs = c.v_scale[p, :, r // c.block].double()  # [tokens, heads]
        codes = values(c.v[p, :, r]).abs()
        ctx = c.kv[b] - n
        seen = torch.ones(n, c.kv[b], dtype=torch.bool)
        seen[:, ctx:] = torch.from_numpy(np.tril(np.ones((n, n), bool)) if masks is None else masks[b][:n, :n])
        t = slice(int(c.new_indptr[b]), int(c.new_indptr[b]) + n)
        for h in range(hk):
            hs = slice(h * g, (h + 1) * g)
            x = torch.einsum("ngd,td->ngt", q[t, hs].double(), k[:, h]) * sm_scale
            x = x.masked_fill(~seen[:, None], -math.inf)
            z = torch.logsumexp(x, -1, keepdim=True)
            w = torch.exp(x - torch.where(torch.isinf(z), torch.zeros_like(z), z))
            vh = torch.where(torch.isnan(v[:, h]), torch.zeros_like(v[:, h]), v[:, h])
            out = torch.einsum("ngt,td->ngd", w, vh)
            weight = torch.einsum("ngt,td->ngd", w, vh.abs())
            top = torch.nan_to_num((w * vs[:, h]).masked_fill(~seen[:, None], 0.0)).amax(-1, keepdim=True)
            ch = torch.where(torch.isnan(codes[:, h]), torch.zeros_like(codes[:, h]), codes[:, h]).clamp(max=448)
            floor = torch.einsum("nt,td->nd", seen.double(), ch)[:, None]
            score = 1e-5 + abs(sm_scale) * 2.0 ** -17 * q[t, hs].double().abs().amax(-1) * k[:, h].nan_to_num().abs().sum(-1).max()
            o[t, hs], lse[t, hs] = out, z[..., 0]
            tol[t, hs] = half * out.abs() + (2.0 ** -8 + 2.0 ** -11 + 2 * score[..., None]) * weight + 2.0 ** -16.5 * top * floor
            tol_l[t, hs] = score + 2.0 ** -20 * z[..., 0].abs().nan_to_num(posinf=0.0)
    return o, lse, tol + 1e-9, tol_l + 1e-5


def check_attention(o, lse, ref, what=""):
    ro, rl, tol, tol_l = ref
    o, lse = o.double().cpu(), lse.double().cpu()
    assert torch.equal(torch.isinf(rl), torch.isinf(lse)), what
    assert not torch.isnan(o).any() and not torch.isnan(lse).any(), what
    off = (o - ro).abs() - tol
    assert float(off.max() if off.numel() else 0.0) <= 0, (what, float(off.max()), float((o - ro).abs().max()))
    fine = ~torch.isinf(rl)
    if fine.any():
        assert float(((lse - rl).abs() - tol_l)[fine].max()) <= 0, (what, float((lse - rl)[fine].abs().max()))
    assert float(o[~fine].abs().max() if (~fine).any() else 0.0) == 0.0, what
