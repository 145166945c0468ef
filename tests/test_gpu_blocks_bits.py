"""The append into block-scaled pools without norms: q elements past rot_dim keep every bit, as in the other appends."""
import numpy as np
import pytest
import torch

from block_helpers import BlockPaged
from spec_helpers import TYPES
from test_gpu_blocks import _append

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("rot", [0, 128, 130])
def test_elements_that_are_not_rotated_keep_every_bit(dtype, layout, rot):
    """Every 16-bit pattern, NaNs of every payload and sign among them; 16-byte accesses, and single elements (rot_dim 130)."""
    import paged_kv_gqa_13_gb300 as pd

    n, hq, d = 512, 1, 256
    c = BlockPaged([n], 1, d, 16, 16, [n])
    x = torch.zeros(n, hq + 2, d, dtype=torch.int16)
    bits = torch.from_numpy(np.arange(n * 128, dtype=np.uint16).view(np.int16)).view(n, 1, 128)
    x[:, :hq, 128:] = bits
    if rot == 0:
        x[:, :hq, :128] = bits.flip(0)
    freqs = pd.pd_rope_frequencies(rot)[0] if rot else None
    flags, _, q = _append(c, x.view(TYPES[dtype]), hq, freqs, layout=layout)
    assert flags == 0
    assert torch.equal(q.cpu().view(torch.int16)[..., rot:], x[:, :hq, rot:])
