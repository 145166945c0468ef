"""Further refusals and empty calls of the speculative-decoding calls, without a GPU."""

from tests.test_spec_abi import APPEND, _call


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
