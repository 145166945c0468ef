"""Tree decode over lines long enough for tails: ranges that go to whichever worker asks first."""
import math

import numpy as np
import pytest
import torch

from tests.tree_helpers import Call

pytestmark = pytest.mark.gpu

# dtype, E4M3 pools, q heads, kv heads, head_dim, requests, nodes up to: the narrow and the wide form, one line, CUDA cores
FORMS = [("bf16", False, 32, 16, 64, 64, 3), ("f16", False, 32, 16, 128, 48, 3), ("bf16", False, 16, 16, 256, 40, 3),
         ("f16", True, 32, 16, 64, 64, 3), ("bf16", True, 128, 16, 64, 64, 16), ("bf16", True, 64, 8, 128, 80, 16),
         ("f16", True, 16, 16, 256, 40, 3), ("f32", False, 32, 16, 64, 64, 3), ("f32", False, 32, 16, 128, 48, 3)]


def _lengths(requests, nodes, seed):
    rng = np.random.default_rng(seed)
    new = [int(x) for x in rng.integers(max(1, nodes - 6), nodes + 1, requests)]
    return [int(x) for x in rng.integers(1000, 2400, requests)], new


@pytest.mark.parametrize("dtype,fp8,hq,hk,d,requests,nodes", FORMS)
def test_tails_are_right_and_repeat_bit_for_bit(dtype, fp8, hq, hk, d, requests, nodes):
    call = Call(*_lengths(requests, nodes, d), hq, hk, d, 16, dtype, fp8, seed=1)
    first = call.check((dtype, fp8, d))
    total, share, tail = call.line()
    assert share >= 48 and tail == share // 8 and total > share
    assert int(call.ws[128:132].view(torch.int32)) == 0  # set back by the merge
    for _ in range(4):
        again = call.run()
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call.launch()
    for _ in range(3):
        call.o.fill_(math.nan)
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(first[0], call.o) and torch.equal(first[1], call.lse)
    assert call.flags() == 0


@pytest.mark.parametrize("before", ["bytes", "another call"])
@pytest.mark.parametrize("dtype,fp8,hq,hk,d,requests,nodes", [FORMS[0], FORMS[2], FORMS[4], FORMS[7]])
def test_tails_that_nobody_runs_leave_the_merge_in_bounds(dtype, fp8, hq, hk, d, requests, nodes, before):
    """As after a call whose every worker gave up: no tail is run, and the descriptors of tails are those that the
    workspace held. The rows that need a tail are undefined; nothing else is touched, and the next call is right."""
    import paged_kv_gqa_13_gb300 as pd

    call = Call(*_lengths(requests, nodes, d), hq, hk, d, 16, dtype, fp8, seed=2)
    if before == "bytes":
        call.ws.fill_(0x7F)
        pd.pd_workspace_init(call.ws)
    else:  # more rows than this call has, descriptors of rows past its last one among them
        more = Call([1800] * (2 * requests), [nodes + 3] * (2 * requests), hq, hk, d, 16, dtype, fp8, seed=3)
        more.run()
        assert more.line()[2] > 0
        call.ws = more.ws
    # rows of the outputs' surroundings must stay as they are
    guard = torch.full((call.o.numel() + 4096,), 7.0, dtype=call.o.dtype, device="cuda")
    call.o = guard[2048:2048 + call.o.numel()].view(call.o.shape)
    guard_lse = torch.full((call.lse.numel() + 4096,), 7.0, device="cuda")
    call.lse = guard_lse[2048:2048 + call.lse.numel()].view(call.lse.shape)
    call.ws[128:132].view(torch.int32).fill_(1 << 20)  # every tail has been asked for
    call.run()
    assert call.line()[2] > 0
    for whole in (guard, guard_lse):
        assert bool((whole[:2048] == 7).all()) and bool((whole[-2048:] == 7).all())
    call.check()
