"""Tree decode where head tiles, pages and row tiles do not fit each other, in every form."""
import pytest

from tests.spec_helpers import check_tree
from tests.tree_helpers import Call, reference

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,fp8", [("f16", False), ("bf16", False), ("f16", True), ("bf16", True), ("f32", False)])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("hq,hk", [(129, 1), (160, 1), (320, 2)])
def test_groups_above_a_row_tile(dtype, fp8, d, hq, hk):
    """More than 128 q heads to a kv head: CUDA cores, the heads cut into tiles."""
    Call([70, 1, 0, 333, 40], [5, 1, 0, 2, 33], hq, hk, d, 16, dtype, fp8, seed=d).check((dtype, fp8, d, hq, hk))
    Call([5000, 9], [3, 2], hq, hk, d, 16, dtype, fp8, seed=d + 1, kind="chain").check((dtype, fp8, d, hq, hk, "cut"))


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("hq,hk", [(33, 1), (40, 1), (9, 1), (34, 2), (63, 1)])
@pytest.mark.parametrize("kv,new", [([900, 40], [1, 1]), ([700, 33, 0, 9], [6, 33, 0, 1])])
def test_head_tiles_in_f32(d, hq, hk, kv, new):
    """Groups that are cut into tiles of 8, 16 and 32 rows, the last of them smaller."""
    Call(kv, new, hq, hk, d, 16, "f32", False, seed=hq).check((d, hq, hk))


@pytest.mark.parametrize("dtype,fp8", [("f16", False), ("bf16", False)])
@pytest.mark.parametrize("hq,hk", [(128, 1), (127, 1), (65, 1), (100, 2), (43, 1), (86, 2)])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_groups_up_to_a_row_tile(dtype, fp8, hq, hk, d):
    """One node, or a few, fill a row tile of the tensor cores; some of its rows stay unused."""
    Call([300, 5, 77], [1, 1, 1], hq, hk, d, 16, dtype, fp8, seed=hq).check((dtype, hq, d, "one"))
    Call([2000, 44, 77], [9, 4, 20], hq, hk, d, 16, dtype, fp8, seed=hq).check((dtype, hq, d, "trees"))


PAGES = [1, 5, 8, 9, 24, 40, 100, 200]


@pytest.mark.parametrize("dtype,fp8", [("f16", False), ("bf16", True), ("f16", True)])
@pytest.mark.parametrize("page", PAGES)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("hq,new", [(4, [12, 5, 7, 1]), (16, [40, 20, 7, 33])])
def test_page_sizes(dtype, fp8, page, d, hq, new):
    """Pages that are whole slots, and pages that end inside one, few rows and many to a request."""
    kv = [129, 400, 7, 150]
    for kind in ("tree", "chain"):
        Call(kv, new, hq, 2, d, page, dtype, fp8, seed=page, kind=kind).check((dtype, fp8, page, d, hq, kind))


@pytest.mark.parametrize("dtype,fp8", [("f16", False), ("bf16", True)])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("page", [5, 24])
def test_pages_that_end_inside_a_slot_over_long_caches(dtype, fp8, d, page):
    Call([6000, 700, 2], [70, 9, 2], 8, 1, d, page, dtype, fp8, seed=page).check((dtype, fp8, d, page))


@pytest.mark.parametrize("dtype,fp8", [("f16", False), ("bf16", False), ("f16", True), ("bf16", True)])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("hq,nodes", [(4, 6), (16, 40)])
@pytest.mark.parametrize("page,at", [(16, 3), (8, 5), (5, 4), (128, 0), (16, -1)])
def test_a_bad_page(dtype, fp8, d, hq, nodes, page, at):
    """Its tokens count as absent; every other request, and every other page, as before."""
    import paged_kv_gqa_13_gb300 as pd

    call = Call([190, 333, nodes], [nodes] * 3, hq, 2, d, page, dtype, fp8, seed=9)
    c = call.c
    at = at if at >= 0 else int(c.indptr[2] - c.indptr[1]) + at
    first, last = at * page, min((at + 1) * page, c.kv[1])
    call.table[0][int(c.indptr[1]) + at] = c.total + 3
    o, lse = call.run()
    assert call.flags() == pd.PD_FLAG_BAD_PAGE_ID
    ref = reference(c, call.q, call.masks, call.scale, {1: (first, last)})
    check_tree(o, lse, ref, dtype, (dtype, fp8, d, page, at))
