"""Attention over block-scaled E4M3 pools: scores that are not a number, on each of the kernels."""
import math

import pytest
import torch

from block_helpers import BlockPaged
from test_gpu_blocks_attention import _q, _run
from test_gpu_blocks_scales import FORMS

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("hq,hk,d,block,new", FORMS)
def test_scores_of_nan_make_their_rows_nan(dtype, hq, hk, d, block, new):
    """A NaN code of K for every row of its head; a NaN of q for its row; in contexts that are cut and in short ones."""
    c = BlockPaged([200, 70, 9000, 20000], hk, d, 16, block, new, seed=2)
    for b, t in ((0, 17), (2, 8900)):
        p, r = c.rows(b, [t])
        c.k[p, 0, r, 5] = 0x7F
    q = _q(sum(c.new), hq, d, dtype, spread=1.0)
    bad = torch.zeros(q.shape[:2], dtype=torch.bool)
    g, starts = hq // hk, c.new_indptr
    for b in (0, 2):
        bad[starts[b]:starts[b + 1], :g] = True
    for row, head in ((int(starts[1]), 1), (int(starts[3]), hq - 1)):
        q[row, head, 3] = math.nan
        bad[row, head] = True
    _, o, lse = _run(c, q, single=new is None)
    o, lse = o.cpu(), lse.cpu()
    assert torch.equal(torch.isnan(o).all(-1), bad) and torch.equal(torch.isnan(o).any(-1), bad)
    assert torch.equal(torch.isnan(lse), bad)
