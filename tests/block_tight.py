"""Plain 64-bit attention over block-scaled pools with a bound on the error that depends on the output's type."""
from __future__ import annotations

import math

import numpy as np
import torch

from block_helpers import values
from spec_helpers import TYPES

LEAST_V = 2.0 ** -88  # smaller V scales count so for the maximum that weights are held against


def attend_tight(c, q, masks, sm_scale, dtype, keep=None):
    """(o, lse, tolerance of o, tolerance of lse) of attention over the BlockPaged c; masks[b] [n, n] booleans, None: a chain;
    keep[b] [tokens] booleans: tokens that count at all.

    Tolerance of o, per output, with S = sum of weight * |value|:
     - half a step of the type for the result;
     - of each weight, its step through f16 (2^-11 S), and for bf16 outputs three E5M2 parts of 3 significant bits (2^-9 S);
     - f32 sums of n terms, at most n / 8 of them one after another into the sum of the weights and n / 32 products into the
       output: n 2^-26 S;
     - the score's error twice (a weight, and the sum): parts of q (2^-21 of a row's largest element), f32 sums of products
       (2^-20 of the sum of their magnitudes), the exponent's f32 (2^-21 of its magnitude), the exponential (2^-20);
     - weights are held to 2^-23 absolutely where the largest weight times V scale is 2^7 or more: 2^-30 of that product for
       each code. V scales below 2^-88 count as that for it.
    """
    total, hq, d = q.shape
    hk = c.k.shape[1]
    g = hq // hk
    half = torch.finfo(TYPES[dtype]).eps / 2
    weights = 2.0 ** -11 + (2.0 ** -9 if dtype == "bf16" else 0.0)
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
        if keep is not None and keep[b] is not None:
            seen &= keep[b]
        some = seen.any(-1)
        t = slice(int(c.new_indptr[b]), int(c.new_indptr[b]) + n)
        for h in range(hk):
            hs = slice(h * g, (h + 1) * g)
            qh, kh = q[t, hs].double(), k[:, h]
            x = (torch.einsum("ngd,td->ngt", qh, kh) * sm_scale).masked_fill(~seen[:, None], -math.inf)
            z = torch.logsumexp(x, -1, keepdim=True)
            w = torch.exp(x - torch.where(torch.isinf(z), torch.zeros_like(z), z))
            vh = v[:, h]
            size = torch.einsum("ngd,td->ngt", qh.abs(), kh.abs()).masked_fill(~seen[:, None], 0.0).amax(-1) * abs(sm_scale)
            most = x.masked_fill(~seen[:, None], 0.0).abs().amax(-1)
            lv = torch.log2(vs[:, h].clamp(min=LEAST_V)).abs().amax()
            score = (2.0 ** -21 * qh.abs().amax(-1) * kh.abs().sum(-1).max() * abs(sm_scale) + 2.0 ** -20 * size
                     + 2.0 ** -21 * (1.45 * most + lv) + 2.0 ** -20)
            s = torch.einsum("ngt,td->ngd", w, vh.abs())
            top = (w * vs[:, h].clamp(min=LEAST_V)).masked_fill(~seen[:, None], 0.0).amax(-1, keepdim=True)
            floor = torch.einsum("nt,td->nd", seen.double(), codes[:, h])[:, None]
            out = torch.einsum("ngt,td->ngd", w, vh)
            sums = c.kv[b] * 2.0 ** -26
            o[t, hs] = out
            lse[t, hs] = torch.where(some[:, None], z[..., 0], torch.full_like(z[..., 0], -math.inf))
            tol[t, hs] = half * out.abs() + (weights + sums + 2 * score[..., None]) * s + 2.0 ** -30 * top * floor
            tol_l[t, hs] = score + sums + 2.0 ** -20 * torch.where(some[:, None], z[..., 0], torch.zeros_like(z[..., 0])).abs()
    tiny = 2.0 ** -25 if dtype == "f16" else 0.0  # half a step of a subnormal f16
    return o, lse, tol + tiny, tol_l
