"""Further refusals and empty calls of the speculative-decoding calls, without a GPU."""
from tests.test_spec_abi import APPEND, ROPE, TREE, _call


def test_append_refuses_q_in_place_at_another_stride():
    """q_out is [total_new, Hq, D]: a wider q there would be overwritten by other tokens' rows before it is read."""
    import paged_kv_gqa_13_gb300 as pd

    assert APPEND["q"] == APPEND["q_out"]
    for dtype in (0, 1, 2):
        assert _call("pd_paged_rope_append", APPEND, qs=1024 + 256, dtype=dtype) == pd.PD_ERR_INVALID
    assert "q_out" in pd.pd_last_error_string()
    d = {}
    for k, v in APPEND.items():
        d[k] = v
        if k == "q_out":
            d["k_scale"] = d["v_scale"] = v
    assert _call("pd_paged_rope_append_fp8", d, qs=1024 + 256) == pd.PD_ERR_INVALID


def test_calls_without_a_token_need_no_rows():
    """No new token anywhere: tensors of no elements, whose pointers are null, are not refused."""
    assert _call("pd_rope", ROPE, tokens=0, x=None, out=None, positions=None) == 0
    assert _call("pd_paged_rope_append", APPEND, total=0, q=None, k=None, v=None, q_out=None, positions=None) == 0
    d = {}
    for k, v in APPEND.items():
        d[k] = v
        if k == "q_out":
            d["k_scale"] = d["v_scale"] = v
    assert _call("pd_paged_rope_append_fp8", d, total=0, q=None, k=None, v=None, q_out=None, positions=None) == 0
    # what is no row is still asked for
    assert _call("pd_paged_rope_append", APPEND, total=0, kd=None) == 1
    assert _call("pd_rope", ROPE, tokens=0, freqs=None) == 1


def test_empty_tensors_through_the_wrappers():
    import torch

    import paged_kv_gqa_13_gb300 as pd

    i32 = lambda *v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    x, f = torch.zeros(0, 2, 128), torch.zeros(64, dtype=torch.int64)
    pd.pd_rope(x, i32(), f, torch.zeros(0, 2, 128), stream=0)
    pool = torch.zeros(3, 2, 16, 128)
    raw = torch.zeros(4096 + 256, dtype=torch.uint8)
    ws = raw[-raw.data_ptr() % 256:][:4096]
    table = (i32(0, 1), i32(0, 1, 2), i32(4, 4), i32(0, 0, 0))
    for q, pos in ((None, None), (x, i32())):
        pd.pd_paged_rope_append(q, x, x, pos, f, torch.zeros(0, 2, 128), pool, pool, *table, ws, stream=0)


def test_tree_decode_without_a_node_needs_no_mask_rows():
    """A mask of no rows has a null pointer and its words."""
    import paged_kv_gqa_13_gb300 as pd

    rows = dict(total=0, q=None, o=None, lse=None)
    status = _call("pd_paged_tree_decode", TREE, mask=None, words=2, **rows)
    assert status in (pd.PD_OK, pd.PD_ERR_CUDA), pd.pd_last_error_string()  # PD_ERR_CUDA: no device here
    assert _call("pd_paged_tree_decode", TREE, mask=None, words=-1, **rows) == pd.PD_ERR_INVALID
    assert _call("pd_paged_tree_decode", TREE, mask=None, words=2) == pd.PD_ERR_INVALID


def test_wrapper_refuses_a_mask_without_words():
    """Its pointer would be null, which is the chain."""
    import pytest
    import torch

    import paged_kv_gqa_13_gb300 as pd

    i32 = lambda *v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    pool, q, lse = torch.zeros(3, 2, 16, 128), torch.zeros(4, 2, 128), torch.zeros(4, 2)
    ws = torch.zeros(4096, dtype=torch.uint8)
    with pytest.raises(pd.PagedecodeError) as e:
        pd.pd_paged_tree_decode(q, pool, pool, i32(0), i32(0, 1), i32(4), i32(0, 4), torch.zeros(4, 0, dtype=torch.int32),
                                torch.zeros_like(q), lse, 0.1, ws, stream=0)
    assert e.value.status == pd.PD_ERR_INVALID and "words" in str(e.value)
    codes = torch.zeros(3, 2, 16, 128, dtype=torch.uint8)
    s = torch.ones(2)
    with pytest.raises(pd.PagedecodeError, match="words"):
        pd.pd_paged_tree_decode_fp8(q.half(), codes, codes, s, s, i32(0), i32(0, 1), i32(4), i32(0, 4),
                                    torch.zeros(4, 0, dtype=torch.int32), q.half(), lse, 0.1, ws, stream=0)
