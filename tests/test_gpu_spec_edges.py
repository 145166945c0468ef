"""Edges of the speculative-decoding calls: rows in place, empty tables, NaN, bits of copied rows."""

import numpy as np
import pytest
import torch

from tests.spec_helpers import TYPES, Paged, rope_reference, rope_tolerance

pytestmark = pytest.mark.gpu


def _inv(rot, theta=10000.0):
    return theta ** (-2.0 * np.arange(rot // 2) / rot)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("tokens,wide", [(9, False), (1, True)])
def test_append_rotates_q_in_place(dtype, tokens, wide):
    """q laid out as q_out, and one token's q as a view of its fused projection."""
    import paged_kv_gqa_13_gb300 as pd

    hq, hk, d = 4, 2, 128
    c = Paged([tokens + 5], [tokens], hk, d, 16, dtype)
    x = torch.randn(tokens, hq + 2 * hk, d).to(TYPES[dtype])
    dev = x.cuda()
    q = dev[:, :hq] if wide else dev[:, :hq].contiguous()
    pos = torch.arange(tokens, dtype=torch.int32) * 91
    freqs, _ = pd.pd_rope_frequencies(d)
    k, v, ws = c.k.cuda(), c.v.cuda(), pd.alloc_workspace(256)
    pd.pd_paged_rope_append(q, dev[:, hq:hq + hk], dev[:, hq + hk:], pos.cuda(), freqs, q, k, v, *c.table(), ws)
    assert pd.pd_read_device_flags(ws) == 0
    ref = rope_reference(x[:, :hq], pos, _inv(d), 0)
    assert bool(((q.double().cpu() - ref).abs() <= rope_tolerance(x[:, :hq], ref, dtype)).all())
    assert torch.equal(dev[:, hq:].cpu(), x[:, hq:])
