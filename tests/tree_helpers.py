"""Tree decode calls whose tensors stay on the card, and their 64-bit form there."""
from __future__ import annotations

import math

import numpy as np
import torch

from tests.spec_helpers import TYPES, Paged, check_tree, pack, tree_bits

CODES = {"f32": 0, "f16": 1, "bf16": 2}


def reference(c, q, masks, sm_scale, absent=None):
    """(o, lse, sum of weight * |v|) in 64 bits on the card; nobody attends tokens first .. last - 1 of request b for
    b: (first, last) in `absent`."""
    total, hq, d = q.shape
    hk = c.k.shape[1]
    o = torch.zeros(total, hq, d, dtype=torch.float64)
    mag, lse = torch.zeros_like(o), torch.full((total, hq), -math.inf, dtype=torch.float64)
    for b, n in enumerate(c.new):
        if n == 0:
            continue
        rows = slice(int(c.new_indptr[b]), int(c.new_indptr[b + 1]))
        k, v = (x.cuda() for x in c.dense(b))
        seen = np.concatenate([np.ones((n, c.kv[b] - n), bool), masks[b]], 1)
        if absent and b in absent:
            seen[:, absent[b][0]:absent[b][1]] = False
        x = torch.einsum("nhgd,thd->nhgt", q[rows].double().cuda().view(n, hk, hq // hk, d), k) * sm_scale
        x.masked_fill_(~torch.from_numpy(seen).cuda()[:, None, None], -math.inf)
        z = torch.logsumexp(x, -1)
        w = torch.exp(x - z[..., None]).nan_to_num(0.0)
        o[rows] = torch.einsum("nhgt,thd->nhgd", w, v).reshape(n, hq, d).cpu()
        mag[rows] = torch.einsum("nhgt,thd->nhgd", w, v.abs()).reshape(n, hq, d).cpu()
        lse[rows] = z.reshape(n, hq).cpu()
    return o, lse, mag


class Call:
    """One decode whose inputs and workspace stay on the card."""

    def __init__(self, kv, new, hq, hk, d, page, dtype, fp8, seed=0, kind="tree"):
        import paged_kv_gqa_13_gb300 as pd

        self.c = Paged(kv, new, hk, d, page, dtype, seed, fp8)
        rng = np.random.default_rng(seed + 7)
        self.q = torch.randn(sum(new), hq, d, generator=torch.Generator().manual_seed(seed + 3)).to(TYPES[dtype])
        self.masks = [tree_bits(rng, n, kind) for n in new]
        self.dtype, self.scale = dtype, 1 / math.sqrt(d)
        words = max(1, -(-max(new) // 32))
        self.mask = None if kind == "chain" else pack(self.masks, words).cuda()
        self.dev = [x.cuda() for x in (self.q, self.c.k, self.c.v)]
        self.scales = (self.c.k_scale.cuda(), self.c.v_scale.cuda()) if fp8 else ()
        self.table = self.c.table()
        self.ws = pd.alloc_workspace(pd.pd_paged_tree_decode_workspace_bytes(hq, hk, d, CODES[dtype]))
        self.o = torch.empty_like(self.dev[0])
        self.lse = torch.empty(self.q.shape[:2], device="cuda")
        self.fn = pd.pd_paged_tree_decode_fp8 if fp8 else pd.pd_paged_tree_decode

    def run(self):
        self.o.fill_(math.nan)
        self.lse.fill_(math.nan)
        self.launch()
        torch.cuda.synchronize()
        return self.o.clone(), self.lse.clone()

    def launch(self):
        self.fn(*self.dev, *self.scales, *self.table, self.mask, self.o, self.lse, self.scale, self.ws)

    def flags(self):
        import paged_kv_gqa_13_gb300 as pd

        return pd.pd_read_device_flags(self.ws)

    def line(self):
        """(total, share, tail) in units."""
        return tuple(int(x) for x in self.ws[256:280].view(torch.int64))

    def check(self, what=""):
        o, lse = self.run()
        assert self.flags() == 0
        check_tree(o, lse, reference(self.c, self.q, self.masks, self.scale), self.dtype, what)
        return o, lse
