"""Attention over block-scaled E4M3 pools: scales of every size, on each of the kernels."""
import math

import numpy as np
import pytest
import torch

from block_helpers import BlockPaged, check_attention
from block_tight import attend_tight
from spec_helpers import TYPES
from test_gpu_blocks_attention import _q, _run

pytestmark = pytest.mark.gpu

MANY = [40, 33, 50, 64]
FORMS = [  # hq, hk, d, block, new tokens of each request (None: one, by the decode)
    (8, 2, 128, 16, None), (8, 2, 256, 4, None), (4, 2, 128, 16, None), (8, 2, 64, 1, None), (32, 2, 256, 16, None),
    (8, 2, 128, 16, MANY), (8, 2, 64, 4, MANY), (4, 2, 256, 16, MANY), (4, 2, 128, 2, MANY),
]


def _case(hq, hk, d, block, new, seed=3):
    kv = [700, 900, 33, 129] if new is None else [700, 900, 50, 129]
    return BlockPaged(kv, hk, d, 16, block, new, seed=seed)


@pytest.mark.parametrize("magnitude", [2.0 ** -20, 2.0 ** -100, 2.0 ** -112])
@pytest.mark.parametrize("hq,hk,d,block,new", FORMS)
def test_small_v_scales(hq, hk, d, block, new, magnitude):
    """Every value times `magnitude`: the same rounding, the same output times it (V scales from 2^-8 to 2^-4 times that)."""
    c = _case(hq, hk, d, block, new)
    c.v_scale *= magnitude
    q = _q(sum(c.new), hq, d, "bf16", spread=1.0)
    flags, o, lse = _run(c, q, single=new is None)
    assert flags == 0
    ref = attend_tight(c, q, None, 1 / math.sqrt(d), "bf16")
    check_attention(o, lse, ref)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("hq,hk,d,block,new", FORMS)
def test_scales_of_very_different_magnitude(dtype, hq, hk, d, block, new):
    """K and V scales over 40 octaves, blocks of zeros, q rows of 2^-20 to 2^7 and with one large element."""
    c = _case(hq, hk, d, block, new)
    g = torch.Generator().manual_seed(1)
    for s in (c.k_scale, c.v_scale):
        fine = ~torch.isnan(s)
        s[fine] = torch.exp2(torch.randint(-40, 1, (int(fine.sum()),), generator=g).float() - 8)
    for b in range(2):
        p, r = c.rows(b, np.arange(0, 32))
        c.v[p, :, r] = 0
        c.v_scale[p, :, r // block] = 2.0 ** -126
    q = _q(sum(c.new), hq, d, "f16").float()
    q *= torch.exp2(torch.randint(-20, 8, (sum(c.new), hq, 1), generator=g).float())
    q[:, :, 5] *= 64
    q = (q * (1.0 if dtype == "bf16" else 0.01)).to(TYPES[dtype])
    flags, o, lse = _run(c, q, single=new is None)
    assert flags == 0
    check_attention(o, lse, attend_tight(c, q, None, 1 / math.sqrt(d), dtype))


@pytest.mark.parametrize("hq,hk,d,block,new", FORMS)
def test_v_scales_of_zero_and_v_of_zeros(hq, hk, d, block, new):
    c = _case(hq, hk, d, block, new)
    q = _q(sum(c.new), hq, d, "bf16", spread=1.0)
    half = [c.rows(b, np.arange(0, n // 2 // 16 * 16)) for b, n in enumerate(c.kv)]
    for p, r in half:
        c.v_scale[p, :, r // block] = 0.0  # (over codes that are not 0)
    flags, o, lse = _run(c, q, single=new is None)
    assert flags == 0
    check_attention(o, lse, attend_tight(c, q, None, 1 / math.sqrt(d), "bf16"))
    c.v_scale[:] = 0.0
    flags, o, lse = _run(c, q, single=new is None)
    assert flags == 0 and not o.any()
    check_attention(o, lse, attend_tight(c, q, None, 1 / math.sqrt(d), "bf16"))
    c.v[:], c.v_scale[:] = 0, 2.0 ** -126
    flags, o, lse2 = _run(c, q, single=new is None)
    assert flags == 0 and not o.any()
    check_attention(o, lse2, attend_tight(c, q, None, 1 / math.sqrt(d), "bf16"))


@pytest.mark.parametrize("hq,hk,d,block,new", FORMS)
def test_negative_and_zero_score_scale(hq, hk, d, block, new):
    c = _case(hq, hk, d, block, new)
    q = _q(sum(c.new), hq, d, "bf16", spread=1.0)
    for scale in (-0.07, 0.0):
        flags, o, lse = _run(c, q, sm_scale=scale, single=new is None)
        assert flags == 0
        check_attention(o, lse, attend_tight(c, q, None, scale, "bf16"))
