"""Inputs and plain 64-bit results (numpy / torch on the host) for the speculative-decoding calls."""
from __future__ import annotations

import math

import numpy as np
import torch

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


class Paged:
    """A shuffled paged cache on the host: values of valid rows, NaN everywhere else."""

    def __init__(self, kv, new, hk, d, page, dtype, seed=0, fp8=False, extra=3):
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.kv, self.new, self.page, self.fp8 = list(kv), list(new), page, fp8
        n = [-(-x // page) for x in kv]
        self.total = sum(n) + extra
        self.indices = rng.permutation(self.total)[:sum(n)].astype(np.int32)
        self.indptr = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        self.last = np.array([x - (m - 1) * page if m else 0 for x, m in zip(kv, n)], np.int32)
        self.new_indptr = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        shape = (self.total, hk, page, d)
        if fp8:
            self.k_scale = torch.rand(hk, generator=g) * 0.01 + 0.01
            self.v_scale = torch.rand(hk, generator=g) * 0.01 + 0.01
            self.k, self.v = ((torch.randn(shape, generator=g) * 60).clamp(-448, 448).to(torch.float8_e4m3fn)
                              .view(torch.uint8) for _ in range(2))
            poison = 0x7F
        else:
            self.k, self.v = (torch.randn(shape, generator=g).to(TYPES[dtype]) for _ in range(2))
            poison = math.nan
        used = torch.zeros(self.total, page, dtype=torch.bool)
        for b in range(len(self.kv)):
            p, r = self.rows(b, np.arange(self.kv[b]))
            used[p, r] = True
        for x in (self.k, self.v):
            x.permute(0, 2, 1, 3)[~used] = poison

    def rows(self, b, tokens):
        tokens = np.asarray(tokens, np.int64)
        return (torch.from_numpy(self.indices[self.indptr[b] + tokens // self.page].astype(np.int64)),
                torch.from_numpy(tokens % self.page))

    def value(self, pool, scale=None):
        if not self.fp8:
            return pool.double()
        return pool.view(torch.float8_e4m3fn).double() * (1.0 if scale is None else scale.double()[:, None])

    def dense(self, b):
        """K, V [tokens, heads, dim] of request b, in 64 bits."""
        p, r = self.rows(b, np.arange(self.kv[b]))
        return (self.value(self.k[p, :, r], self.k_scale if self.fp8 else None),
                self.value(self.v[p, :, r], self.v_scale if self.fp8 else None))

    def table(self, device="cuda"):
        return tuple(torch.from_numpy(x).to(device) for x in (self.indices, self.indptr, self.last, self.new_indptr))


def tree_bits(rng, n, kind="tree"):
    """[n, n] booleans: who attends whom among the nodes."""
    seen = np.zeros((n, n), bool)
    if kind == "chain":
        return np.tril(np.ones((n, n), bool))
    if kind == "random":
        return rng.random((n, n)) < 0.4
    if kind == "nothing":
        return seen
    for j in range(n):
        p = int(rng.integers(-1, j)) if j else -1
        if p >= 0:
            seen[j] = seen[p]
        seen[j, j] = True
    return seen


def pack(masks, words):
    """The requests' boolean masks as int32 words [total, words]."""
    out = np.zeros((sum(len(m) for m in masks), words), np.uint32)
    at = 0
    for m in masks:
        for j in range(len(m)):
            for i in np.nonzero(m[j])[0]:
                if i < 32 * words:
                    out[at, i // 32] |= np.uint32(1 << (i % 32))
            at += 1
    return torch.from_numpy(out.view(np.int32))


def tree_reference(c, q, masks, sm_scale):
    """(o, lse, sum of weight * |v|) in 64 bits. Only attended tokens take part."""
    total, hq, d = q.shape
    hk = c.k.shape[1]
    g = hq // hk
    o = torch.zeros(total, hq, d, dtype=torch.float64)
    mag = torch.zeros_like(o)
    lse = torch.full((total, hq), -math.inf, dtype=torch.float64)
    for b, n in enumerate(c.new):
        if n == 0:
            continue
        k, v = c.dense(b)
        ctx = c.kv[b] - n
        for j in range(n):
            seen = np.concatenate([np.ones(ctx, bool), masks[b][j]])
            at = torch.from_numpy(np.nonzero(seen)[0])
            if not len(at):
                continue
            t = int(c.new_indptr[b]) + j
            for h in range(hk):
                x = q[t, h * g:(h + 1) * g].double() @ k[at, h].T * sm_scale
                z = torch.logsumexp(x, -1)
                w = torch.exp(x - z[:, None])
                o[t, h * g:(h + 1) * g] = w @ v[at, h]
                mag[t, h * g:(h + 1) * g] = w @ v[at, h].abs()
                lse[t, h * g:(h + 1) * g] = z
    return o, lse, mag


def check_tree(o, lse, ref, dtype, what=""):
    """Half a step of the type for each weight (16-bit only) and for the result; f32 sums and exponentials beside it.

    Per weight: the score's f32 sum over up to 256 products of order 1 and the exponential, 1e-5 in all.
    """
    ro, rl, mag = ref
    half = torch.finfo(TYPES[dtype]).eps / 2
    tol = (1e-5 + (half if dtype != "f32" else 0.0)) * mag + half * ro.abs() + 1e-7
    o, lse = o.double().cpu(), lse.double().cpu()
    off = (o - ro).abs() - tol
    assert not torch.isnan(o).any(), what
    assert float(off.max()) <= 0, (what, float(off.max()), float((o - ro).abs().max()))
    assert torch.equal(torch.isinf(rl), torch.isinf(lse)), what
    fine = ~torch.isinf(rl)
    if fine.any():
        assert float((lse - rl)[fine].abs().max()) <= 1e-4, (what, float((lse - rl)[fine].abs().max()))
    assert float(o[~fine].abs().max() if (~fine).any() else 0.0) == 0.0


def rope_reference(x, positions, inv_freq, layout, scale=1.0):
    """x [..., tokens, heads, d] rotated in 64 bits; inv_freq in radians."""
    rot = 2 * len(inv_freq)
    a = positions.double()[:, None] * torch.as_tensor(inv_freq, dtype=torch.float64)
    c, s = (a.cos() * scale)[:, None], (a.sin() * scale)[:, None]
    y = x.double().clone()
    one, two = (slice(0, rot // 2), slice(rot // 2, rot)) if layout == 0 else (slice(0, rot, 2), slice(1, rot, 2))
    u, w = x.double()[..., one], x.double()[..., two]
    y[..., one], y[..., two] = u * c - w * s, w * c + u * s
    return y


def rope_tolerance(x, ref, dtype, scale=1.0, rot=None):
    """cos and sin each to 2^-22 absolutely (the phase's 24 bits and sincospi), two products and a sum in f32, half a
    step of the type for the result."""
    half = torch.finfo(TYPES[dtype]).eps / 2
    top = x.double().abs().amax(-1, keepdim=True)
    return half * ref.abs() + 2 * abs(scale) * top * (2.0 ** -22 + 2.0 ** -23) + 1e-12
