"""Keeping the accepted nodes of a tree in a block-scaled pool: they are appended again at their places."""
import math

import numpy as np
import pytest
import torch

from block_helpers import values
from spec_helpers import TYPES, pack, tree_bits

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("block,hq,hk,d", [(16, 8, 2, 128), (1, 8, 2, 64), (4, 4, 4, 256)])
def test_accepted_nodes_appended_again(dtype, block, hq, hk, d):
    """Steps of: append a tree, attend, append the accepted nodes' rows again over the shortened request, attend them all."""
    import paged_kv_gqa_13_gb300 as pd

    page, kv = 16, [30, 17]
    rng = np.random.default_rng(block)
    g = torch.Generator().manual_seed(block)
    freqs, _ = pd.pd_rope_frequencies(d, 10000.0)
    k, v = (torch.zeros(20, hk, page, d, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros(20, hk, page // block, device="cuda") for _ in range(2))
    pages = [torch.arange(20, dtype=torch.int32)[b::2] for b in range(2)]
    code = pd.PD_F16 if dtype == "f16" else pd.PD_BF16
    ws = pd.alloc_workspace(pd.pd_paged_tree_decode_fp8_blocks_workspace_bytes(hq, hk, d, code))
    rows = [torch.randn(n, hq + 2 * hk, d, generator=g).to(TYPES[dtype]) for n in kv]  # what each request's tokens came as

    def table(lens):
        n = [-(-x // page) for x in lens]
        return tuple(torch.tensor(x, dtype=torch.int32, device="cuda") for x in (
            torch.cat([p[:m] for p, m in zip(pages, n)]).tolist(), [0, n[0], n[0] + n[1]], [x - (m - 1) * page for x, m in zip(lens, n)]))

    def append(lens, new, positions=None):
        """The last rows `new` of requests of `lens` tokens; the rotated q rows."""
        x = torch.cat(new).cuda()
        q = torch.empty(x.shape[0], hq, d, dtype=x.dtype, device="cuda")
        nptr = torch.tensor([0, len(new[0]), len(x)], dtype=torch.int32, device="cuda")
        pd.pd_paged_rope_append_fp8_blocks(x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:], positions, freqs, q, ks, vs, k, v, *table(lens),
                                           nptr, ws)
        return q, nptr

    def attend(lens, q, nptr, masks):
        o, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
        mask = None if masks is None else pack(masks, 1).cuda()
        pd.pd_paged_tree_decode_fp8_blocks(q, k, v, ks, vs, *table(lens), nptr, mask, o, lse, 1 / math.sqrt(d), ws)
        return o, lse

    def check(lens, q, masks, new, o):
        """o against attention over what the pools hold, and the pools against the rows that came."""
        at = 0
        for b, n in enumerate(new):
            t = torch.arange(lens[b])
            p, r = pages[b][t // page].long(), t % page
            held = [values(x.cpu()[p, :, r]) * s.cpu()[p, :, r // block].double()[..., None] for x, s in ((k, ks), (v, vs))]
            scale = vs.cpu()[p, :, r // block].double()[..., None]
            want = rows[b][:, hq + hk:].double()
            # half a step of a code, and of subnormal ones at each scale that the block has had: 2^-10 s + 2^-10 s / 2 + ...
            assert bool(((held[1] - want).abs() <= 2.0 ** -4 * want.abs() + 2 * 2.0 ** -10 * scale).all()), b
            seen = torch.ones(n, lens[b], dtype=torch.bool)
            seen[:, lens[b] - n:] = torch.from_numpy(np.tril(np.ones((n, n), bool)) if masks is None else masks[b])
            x = torch.einsum("ngd,tgd->ngt", q[at:at + n].double().cpu(), held[0].repeat_interleave(hq // hk, 1)) / math.sqrt(d)
            w = x.masked_fill(~seen[:, None], -math.inf).softmax(-1)
            vh = held[1].repeat_interleave(hq // hk, 1)
            ref, size = torch.einsum("ngt,tgd->ngd", w, vh), torch.einsum("ngt,tgd->ngd", w, vh.abs())
            # half a step of the output; of each weight 2^-9 and f16's 2^-11; scores to 1e-4
            tol = torch.finfo(TYPES[dtype]).eps / 2 * ref.abs() + (2.0 ** -9 + 2.0 ** -11 + 2e-4) * size
            assert bool(((o[at:at + n].double().cpu() - ref).abs() <= tol).all()), b
            at += n

    append(kv, rows)
    for step in range(4):
        sizes = [7, 12]
        trees = [torch.randn(n, hq + 2 * hk, d, generator=g).to(TYPES[dtype]) for n in sizes]
        trees[0][3] *= 4  # (a node that makes its block's scale grow, accepted or not)
        masks = [tree_bits(rng, n) for n in sizes]
        depth = [m.sum(1) - 1 for m in masks]
        positions = torch.tensor(np.concatenate([x + y for x, y in zip(kv, depth)]), dtype=torch.int32, device="cuda")
        before, lens = [r.clone() for r in rows], [x + n for x, n in zip(kv, sizes)]
        rows = [torch.cat(x) for x in zip(rows, trees)]
        q, nptr = append(lens, trees, positions)
        o, _ = attend(lens, q, nptr, masks)
        check(lens, q, masks, sizes, o)
        # keep the path to one node of each tree: its rows again, as a chain behind the context
        path = [np.nonzero(m[int(rng.integers(n))])[0] for m, n in zip(masks, sizes)]
        kept = [t[p] for t, p in zip(trees, path)]
        kv = [x + len(p) for x, p in zip(kv, path)]
        rows = [torch.cat(x) for x in zip(before, kept)]
        q, nptr = append(kv, kept)
        o, _ = attend(kv, q, nptr, None)
        check(kv, q, None, [len(p) for p in path], o)
    assert pd.pd_read_device_flags(ws) == 0
