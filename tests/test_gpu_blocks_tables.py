"""Block-scaled E4M3 pools: tables of new and of read rows that leave rows out, or name them twice, are flagged."""
import numpy as np
import pytest
import torch

from block_helpers import BlockPaged
from test_gpu_blocks import _append

pytestmark = pytest.mark.gpu


def _device(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("hq", [0, 2])
@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("table", [[0, 9, 12, 31], [1, 9, 12, 32], [0, 9, 12, 12], [0, 0, 0, 0], [5, 5, 5, 5], [0, 9, 12, 33], [0, 9, 8, 32],
                                   [-1, 9, 12, 32], [32, 32, 32, 32]])
def test_append_flags_rows_of_no_request(hq, given, table):
    import paged_kv_gqa_13_gb300 as pd

    c = BlockPaged([40, 21, 37], 2, 64, 16, 8, [9, 3, 20], seed=5)
    x = torch.randn(32, hq + 4, 64, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16)
    positions = torch.arange(32, dtype=torch.int32, device="cuda") if given else None
    flags, _, _ = _append(c, x, hq, positions=positions, table=(*c.table(), _device(table)))
    assert flags & pd.PD_FLAG_BAD_NEW_ROWS
    flags, _, _ = _append(c, x, hq, positions=positions)
    assert flags == 0


@pytest.mark.parametrize("hq", [0, 1])
def test_append_flags_a_request_that_ends_before_it_starts(hq):
    """The next request's rows then belong to two."""
    import paged_kv_gqa_13_gb300 as pd

    c = BlockPaged([100, 16, 32], 1, 64, 16, 16, [100, 0, 0], seed=5)
    x = torch.randn(100, hq + 2, 64).to(torch.bfloat16)
    flags, _, _ = _append(c, x, hq, positions=torch.arange(100, dtype=torch.int32, device="cuda"), table=(*c.table(), _device([0, 100, 68, 100])))
    assert flags & pd.PD_FLAG_BAD_NEW_ROWS


def test_append_of_many_requests_checks_each():
    import paged_kv_gqa_13_gb300 as pd

    n = 500
    c = BlockPaged([3] * n, 1, 64, 16, 16, [1] * n, seed=1)
    x = torch.randn(n, 2, 64).to(torch.bfloat16)
    assert _append(c, x, 0)[0] == 0
    for at in (1, 77, n - 1, n):
        table = c.new_indptr.copy()
        table[at] -= 2
        assert _append(c, x, 0, table=(*c.table(), _device(table.tolist())))[0] & pd.PD_FLAG_BAD_NEW_ROWS


@pytest.mark.parametrize("table,bad", [([0, 100, 90, 100], True), ([0, 20, 19, 30], True), ([-1, 20, 30, 40], True), ([0, 20, 30, 101], True),
                                       ([0, 20, 30, 40], False), ([7, 20, 30, 40], False), ([0, 0, 0, 0], False), ([100, 100, 100, 100], False)])
def test_read_flags_malformed_tables_and_leaves_other_rows(table, bad):
    """Rows before the first request's and behind the last one's stay as they were."""
    import paged_kv_gqa_13_gb300 as pd

    c = BlockPaged([120, 30, 64], 2, 64, 16, 16)
    out = [torch.full((100, 2, 64), 7.0, device="cuda") for _ in range(2)]
    ws = pd.alloc_workspace(256)
    pd.pd_paged_read_fp8_blocks(*c.pools(), *c.table(), _device(table), None, *out, ws)
    flags = pd.pd_read_device_flags(ws)
    if bad:
        assert flags & pd.PD_FLAG_BAD_NEW_ROWS
        return
    assert flags == 0
    for y, which in ((out[0], 0), (out[1], 1)):
        assert bool((y[:table[0]] == 7).all()) and bool((y[table[-1]:] == 7).all())
        for b in range(3):
            n = table[b + 1] - table[b]
            if n:
                want = c.held(b, np.arange(n))[which].float()
                assert torch.equal(y[table[b]:table[b + 1]].cpu(), want)
