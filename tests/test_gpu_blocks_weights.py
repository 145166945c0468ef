"""Attention over block-scaled E4M3 pools: the mass of many small weights, and errors bounded by the output's type."""
import math

import numpy as np
import pytest
import torch

from block_helpers import BlockPaged, check_attention, codes_of
from block_tight import attend_tight
from spec_helpers import TYPES, tree_bits
from test_gpu_blocks_attention import _q, _run

pytestmark = pytest.mark.gpu


def _shared(c, batch):
    """c's one request `batch` times, over the same pages."""
    many = BlockPaged([1], 1, 64, 16, 16)
    many.__dict__.update(c.__dict__)
    many.kv, many.new = c.kv * batch, c.new * batch
    many.indices, many.last = np.tile(c.indices, batch), np.tile(c.last, batch)
    many.indptr = (np.arange(batch + 1) * len(c.indices)).astype(np.int32)
    many.new_indptr = (np.arange(batch + 1) * c.new[0]).astype(np.int32)
    return many


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("hq,hk,d,block,new,batch", [
    (2, 2, 128, 16, 1, 160), (4, 2, 64, 16, 1, 160), (16, 1, 128, 1, 1, 320), (16, 1, 256, 16, 1, 160), (8, 1, 64, 4, 1, 3),
    (24, 1, 128, 16, 1, 320), (4, 1, 64, 16, 4, 320), (4, 1, 128, 16, 1, 310), (8, 1, 256, 16, 1, 160), (4, 1, 128, 16, 40, 160),
    (4, 1, 64, 2, 40, 160), (24, 1, 128, 1, 1, 320), (24, 1, 128, 16, 1, 600), (32, 1, 64, 4, 1, 600),
])
@pytest.mark.parametrize("n,ahead,where", [(4096, 12.0, 0), (16384, 12.0, 0), (16384, 14.0, 16000), (65536, 16.0, 100)])
def test_a_long_tail_beside_one_dominant_key(dtype, hq, hk, d, block, new, batch, n, ahead, where):
    """One key whose score is `ahead` above the mean of the rest and whose V is 0; V of the rest is 1: the output is the tail's
    share of the weights. With many requests a segment is a whole context."""
    c = BlockPaged([n], hk, d, 16, block, [new], seed=int(ahead))
    p, r = c.rows(0, np.arange(n))
    g = torch.Generator().manual_seed(d)
    k = torch.randn(n, hk, d, generator=g) * 8
    k[:, :, 0] = 0
    k[where], k[where, :, 0] = 0, 16 * ahead
    c.k[p, :, r], c.k_scale[:] = codes_of(k), 2.0 ** -4
    v = torch.full((n, hk, d), 64.0)
    v[where] = 0
    c.v[p, :, r], c.v_scale[:] = codes_of(v), 2.0 ** -6
    q = torch.randn(new, hq, d, generator=g).to(TYPES[dtype])
    q[:, :, 0] = math.sqrt(d)
    ref = attend_tight(c, q, None, 1 / math.sqrt(d), dtype)
    flags, o, lse = _run(_shared(c, batch), q.repeat(batch, 1, 1), single=new == 1)
    assert flags == 0
    check_attention(o, lse, tuple(x.repeat(batch, *[1] * (x.dim() - 1)) for x in ref))


FORMS = [  # hq, hk, d, page, block, new tokens of each request (None: one, by the decode)
    (8, 2, 128, 16, 16, None), (12, 2, 256, 16, 1, None), (4, 2, 128, 16, 16, None), (8, 1, 64, 16, 4, None),
    (32, 2, 256, 64, 32, None), (16, 1, 128, 20, 5, None), (8, 2, 128, 16, 16, [40, 33, 50, 64, 41, 70]),
    (8, 1, 64, 16, 4, [40, 33, 50, 64, 41, 70]), (4, 1, 256, 32, 32, [40, 33, 50, 64, 41, 70]), (4, 2, 256, 7, 7, [40, 33, 50, 64, 41, 70]),
]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("hq,hk,d,page,block,new", FORMS)
def test_few_and_many_tokens_within_the_types_rounding(dtype, hq, hk, d, page, block, new):
    kv = [1, 2, 3, 40, 129, 1000] if new is None else [n + x for n, x in zip(new, [0, 1, 2, 100, 300, 900])]
    c = BlockPaged(kv, hk, d, page, block, new, seed=hq + d)
    q = _q(sum(c.new), hq, d, dtype, spread=1.0)
    flags, o, lse = _run(c, q, single=new is None)
    assert flags == 0
    check_attention(o, lse, attend_tight(c, q, None, 1 / math.sqrt(d), dtype))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("kind", ["tree", "random"])
def test_requests_of_very_different_numbers_of_rows(dtype, kind):
    """Single tokens beside one prompt piece or tree of many nodes: the form goes by the mean, the results by nothing."""
    new = [1] * 40 + [300] + [1] * 30
    rng = np.random.default_rng(3)
    kv = [n + int(x) for n, x in zip(new, rng.integers(0, 200, len(new)))]
    c = BlockPaged(kv, 1, 128, 16, 16, new, seed=9)
    masks = [tree_bits(rng, n, kind) for n in new]
    q = _q(sum(new), 2, 128, dtype, spread=1.0)
    flags, o, lse = _run(c, q, masks)
    assert flags == 0
    check_attention(o, lse, attend_tight(c, q, masks, 1 / math.sqrt(128), dtype))


@pytest.mark.parametrize("d,block", [(64, 16), (64, 2), (128, 16), (128, 1), (256, 16)])
def test_many_requests_of_17_to_32_rows(d, block):
    rng = np.random.default_rng(d)
    kv = [3000, 0, 1, 31] + rng.integers(1, 200, 68).tolist()
    c = BlockPaged(kv, 8, d, 16, block, seed=d)
    q = _q(len(kv), 8 * 24, d, "bf16", spread=1.0)
    flags, o, lse = _run(c, q, single=True)
    assert flags == 0
    check_attention(o, lse, attend_tight(c, q, None, 1 / math.sqrt(d), "bf16"))
