"""Attention over block-scaled E4M3 pools: rows that attend nothing of the first tiles of their context."""
import math

import numpy as np
import pytest
import torch

from block_helpers import BlockPaged, check_attention, codes_of
from block_tight import attend_tight
from spec_helpers import TYPES
from test_gpu_blocks_attention import _run

pytestmark = pytest.mark.gpu


def _set_scores(c, q, level, small):
    """K with a score of about level[t] (natural logarithms, for q's first element of sqrt(d)) on top of a random part; V
    scales `small`."""
    d = q.shape[-1]
    g = torch.Generator().manual_seed(7)
    q[:, :, 0] = math.sqrt(d)
    for b, n in enumerate(c.kv):
        p, r = c.rows(b, np.arange(n))
        k = torch.randn(n, c.k.shape[1], d, generator=g) * 8
        k[:, :, 0] = torch.as_tensor(level[:n], dtype=torch.float32)[:, None] * 16
        c.k[p, :, r] = codes_of(k)
    c.k_scale[:], c.v_scale[:] = 2.0 ** -4, small
    return q


@pytest.mark.parametrize("dtype,small", [("bf16", 2.0 ** -40), ("f16", 2.0 ** -14)])
@pytest.mark.parametrize("hq,hk,d,block,mean", [(1, 1, 128, 16, "few"), (2, 2, 64, 4, "few"), (1, 1, 256, 1, "few"), (4, 1, 128, 16, "many"),
                                                (2, 1, 64, 8, "many")])
@pytest.mark.parametrize("climb", [False, True])
def test_trees_whose_rows_skip_whole_tiles(dtype, small, hq, hk, d, block, mean, climb):
    """One tree of 400 nodes without context among many single nodes (or alone: the form for many rows). From node 128 on nobody
    attends the first 128 nodes, from node 256 on only every third row attends the second 128."""
    n = 400
    new = [n] + [1] * 60 if mean == "few" else [n]
    c = BlockPaged(new, hk, d, 16, block, new, seed=d)
    rng = np.random.default_rng(4)
    seen = rng.random((n, n)) < 0.3
    seen[128:, :128] = False
    seen[256:, 128:256] &= (np.arange(256, n) % 3 == 0)[:, None]
    seen[300:340] = False  # rows of nothing
    level = np.full(n, -14.0)
    if climb:
        level[:128], level[128:256], level[256:] = 8.0, -9.0, 9.0
    g = torch.Generator().manual_seed(d)
    q = _set_scores(c, torch.randn(sum(new), hq, d, generator=g).to(TYPES[dtype]), level, small)
    masks = [seen] + [np.ones((1, 1), bool)] * (len(new) - 1)
    flags, o, lse = _run(c, q, masks)
    assert flags == 0
    check_attention(o, lse, attend_tight(c, q, masks, 1 / math.sqrt(d), dtype))


@pytest.mark.parametrize("dtype,small", [("bf16", 2.0 ** -40), ("f16", 2.0 ** -14)])
@pytest.mark.parametrize("hq,hk,d,block,new", [(2, 1, 128, 16, 1), (8, 1, 64, 4, 1), (4, 1, 128, 16, 1), (8, 1, 256, 1, 1), (4, 1, 128, 16, 50),
                                               (4, 1, 64, 2, 50)])
def test_a_context_whose_first_pages_are_bad(dtype, small, hq, hk, d, block, new):
    import paged_kv_gqa_13_gb300 as pd

    kv = [500, 300]
    c = BlockPaged(kv, hk, d, 16, block, [new] * 2, seed=d)
    g = torch.Generator().manual_seed(d)
    q = _set_scores(c, torch.randn(2 * new, hq, d, generator=g).to(TYPES[dtype]), np.full(500, -14.0), small)
    keep = torch.ones(500, dtype=torch.bool)
    keep[:16 * 17] = False
    ref = attend_tight(c, q, None, 1 / math.sqrt(d), dtype, [keep, None])
    ind, ptr, last = c.table()
    ind[:17] = c.total + 5
    flags, o, lse = _run(c, q, single=new == 1, table=(ind, ptr, last))
    assert flags == pd.PD_FLAG_BAD_PAGE_ID
    check_attention(o, lse, ref)
