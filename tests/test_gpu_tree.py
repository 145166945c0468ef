"""Tree decode against a plain 64-bit form: types, head layouts, page sizes, masks, splits, refusals on the device."""
import math

import numpy as np
import pytest
import torch

from tests.spec_helpers import TYPES, Paged, check_tree, pack, tree_bits, tree_reference

pytestmark = pytest.mark.gpu


def _run(c, q, masks, words, sm_scale, dtype, stream=None, ws=None):
    import paged_kv_gqa_13_gb300 as pd

    hq, d = q.shape[1:]
    if ws is None:
        code = {"f32": pd.PD_F32, "f16": pd.PD_F16, "bf16": pd.PD_BF16}[dtype]
        ws = pd.alloc_workspace(pd.pd_paged_tree_decode_workspace_bytes(hq, c.k.shape[1], d, code))
    o = torch.full(q.shape, math.nan, dtype=TYPES[dtype], device="cuda")
    lse = torch.full(q.shape[:2], math.nan, device="cuda")
    mask = None if masks is None else pack(masks, words).cuda()
    if c.fp8:
        pd.pd_paged_tree_decode_fp8(q.cuda(), c.k.cuda(), c.v.cuda(), c.k_scale.cuda(), c.v_scale.cuda(), *c.table(), mask, o,
                                    lse, sm_scale, ws, stream=stream)
    else:
        pd.pd_paged_tree_decode(q.cuda(), c.k.cuda(), c.v.cuda(), *c.table(), mask, o, lse, sm_scale, ws, stream=stream)
    torch.cuda.synchronize()
    return o, lse, pd.pd_read_device_flags(ws)


def _case(kv, new, hq, hk, d, page, dtype, kind, seed=0, fp8=False, words=None, sm_scale=None):
    c = Paged(kv, new, hk, d, page, dtype, seed, fp8)
    rng = np.random.default_rng(seed + 7)
    q = torch.randn(sum(new), hq, d, generator=torch.Generator().manual_seed(seed + 3)).to(TYPES[dtype])
    masks = [tree_bits(rng, n, kind) for n in new]
    words = words or max(1, -(-max(new) // 32))
    sm_scale = 1 / math.sqrt(d) if sm_scale is None else sm_scale
    o, lse, flags = _run(c, q, None if kind == "chain" else masks, words, sm_scale, dtype)
    assert flags == 0
    check_tree(o, lse, tree_reference(c, q, masks, sm_scale), dtype, (kv, new, hq, hk, d, page, dtype, kind))
    return c, q, masks


SHAPES = [(8, 2, 64), (8, 2, 128), (4, 4, 128), (8, 1, 256), (7, 1, 128), (3, 3, 256), (16, 1, 64), (24, 1, 128)]


@pytest.mark.parametrize("dtype,fp8", [("f32", False), ("f16", False), ("bf16", False), ("f16", True), ("bf16", True)])
@pytest.mark.parametrize("hq,hk,d", SHAPES)
def test_types_and_head_layouts(dtype, fp8, hq, hk, d):
    _case([100, 1, 0, 333, 64, 17], [6, 1, 0, 9, 64, 17], hq, hk, d, 16, dtype, "tree", fp8=fp8)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("page", [1, 3, 5, 8, 16, 24, 32, 40, 64, 128, 200, 256, 384])
@pytest.mark.parametrize("kind", ["tree", "chain"])
def test_page_sizes(dtype, page, kind):
    _case([129, 400, 7], [12, 5, 7], 4, 2, 128, page, dtype, kind, seed=page)


@pytest.mark.parametrize("dtype,fp8", [("f32", False), ("f16", False), ("bf16", True)])
@pytest.mark.parametrize("kind", ["random", "nothing", "tree"])
@pytest.mark.parametrize("kv,new", [([40, 40], [40, 13]), ([130, 33], [100, 33]), ([300], [257])])
def test_masks_that_leave_rows_empty_and_requests_without_a_context(dtype, fp8, kind, kv, new):
    _case(kv, new, 4, 2, 64, 16, dtype, kind, fp8=fp8)


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("n", [1, 2, 15, 16, 31, 32, 33, 63, 64, 65, 127, 128, 129, 200, 300])
def test_numbers_of_nodes(dtype, n):
    _case([n, n + 1, n + 130], [n, n, n], 4, 2, 128, 16, dtype, "tree" if n % 2 else "chain")


def test_words_beyond_and_short_of_the_nodes():
    rng = np.random.default_rng(0)
    _case([90], [40], 4, 2, 128, 16, "bf16", "tree", words=5)
    # bits past the last word count as clear
    c = Paged([90], [40], 2, 128, 16, "bf16")
    q = torch.randn(40, 4, 128).bfloat16()
    full = tree_bits(rng, 40, "random")
    cut = full.copy()
    cut[:, 32:] = False
    o, lse, _ = _run(c, q, [full], 1, 0.1, "bf16")
    check_tree(o, lse, tree_reference(c, q, [cut], 0.1), "bf16")


@pytest.mark.parametrize("dtype,fp8", [("f32", False), ("f16", False), ("bf16", False), ("bf16", True)])
@pytest.mark.parametrize("hq,hk,d", [(8, 2, 128), (4, 4, 64), (2, 2, 256)])
def test_long_caches_are_split_over_the_card_and_merged(dtype, fp8, hq, hk, d):
    _case([9000, 3, 2500], [5, 3, 40], hq, hk, d, 16, dtype, "tree", fp8=fp8)
    _case([5000, 4100], [40, 1], hq, hk, d, 32, dtype, "chain", fp8=fp8)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_many_short_requests(dtype):
    rng = np.random.default_rng(5)
    new = [int(x) for x in rng.integers(0, 6, 700)]
    kv = [n + int(x) for n, x in zip(new, rng.integers(0, 40, 700))]
    _case(kv, new, 2, 1, 64, 16, dtype, "tree")


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("sm_scale", [0.0, -0.07, 0.5])
def test_score_scales(dtype, sm_scale):
    _case([200, 70], [9, 70], 4, 2, 64, 16, dtype, "tree", sm_scale=sm_scale)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_growing_scores_rescale_the_running_sums(dtype):
    """Keys that grow along the cache raise every row's maximum again and again."""
    c = Paged([700], [6], 2, 64, 16, dtype)
    q = torch.randn(6, 4, 64).to(TYPES[dtype])
    for t in range(700):
        p, r = c.rows(0, [t])
        c.k[p, :, r] = (c.k[p, :, r].float() * (0.02 * t)).to(c.k.dtype)
    masks = [tree_bits(np.random.default_rng(0), 6)]
    o, lse, _ = _run(c, q, masks, 1, 0.125, dtype)
    ro, rl, mag = tree_reference(c, q, masks, 0.125)
    # scores reach about 100: an f32 sum of 64 products of that size is off by up to 64 * 2^-24 * 100 = 4e-4, and a weight by as much
    half = torch.finfo(TYPES[dtype]).eps / 2
    tol = (1e-3 + (half if dtype != "f32" else 0.0)) * mag + half * ro.abs()
    assert bool(((o.double().cpu() - ro).abs() <= tol).all())
    assert float((lse.double().cpu() - rl).abs().max()) <= 1e-3


@pytest.mark.parametrize("dtype,fp8", [("f32", False), ("f16", False), ("bf16", False), ("f16", True), ("bf16", True)])
@pytest.mark.parametrize("what", ["nan", "inf"])
@pytest.mark.parametrize("d,n", [(64, 5), (128, 70), (256, 5)])
def test_what_a_node_does_not_attend_has_no_part_in_its_result(dtype, fp8, what, d, n):
    if fp8 and what == "inf":
        pytest.skip("E4M3 has no infinity")
    new, kv = [n, 3], [n + 200, 90]
    c = Paged(kv, new, 2, d, 16, dtype, fp8=fp8)
    q = torch.randn(sum(new), 4, d).to(TYPES[dtype])
    masks = [np.eye(m, dtype=bool) for m in new]  # each node sees itself alone, beside the context
    clean, clean_lse, _ = _run(c, q, masks, 3, 0.1, dtype)
    bad = (0, 2)  # request 0, node 2
    p, r = c.rows(0, [kv[0] - n + bad[1]])
    if fp8:
        c.k[p, :, r] = 0x7F
        c.v[p, :, r] = 0xFF
    else:
        c.k[p, :, r] = math.nan if what == "nan" else math.inf
        c.v[p, :, r] = math.nan if what == "nan" else -math.inf
    o, lse, flags = _run(c, q, masks, 3, 0.1, dtype)
    rows = [i for i in range(sum(new)) if i != bad[1]]
    assert flags == 0
    assert torch.equal(o[rows], clean[rows]) and torch.equal(lse[rows], clean_lse[rows])
    assert bool(torch.isnan(o[bad[1]]).any())


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_non_finite_values_reach_the_nodes_that_attend_them(dtype):
    c = Paged([150], [4], 2, 128, 16, dtype)
    q = torch.randn(4, 4, 128).to(TYPES[dtype])
    masks = [tree_bits(np.random.default_rng(0), 4, "chain")]
    clean, _, _ = _run(c, q, None, 0, 0.1, dtype)
    p, r = c.rows(0, [147])  # node 1
    c.v[p, :, r, 5] = math.inf
    c.v[p, :, r, 9] = math.nan
    o, lse, _ = _run(c, q, None, 0, 0.1, dtype)
    assert torch.equal(o[0], clean[0])
    assert bool(torch.isinf(o[1:, :, 5]).all()) and bool(torch.isnan(o[1:, :, 9]).all())
    rest = [i for i in range(128) if i not in (5, 9)]
    assert torch.equal(o[:, :, rest], clean[:, :, rest]) and bool(torch.isfinite(lse).all())
    assert masks[0][3, 1]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_bad_tables_are_flagged_and_spare_the_other_requests(dtype):
    import paged_kv_gqa_13_gb300 as pd

    kv, new = [40, 90, 20], [4, 5, 6]
    c = Paged(kv, new, 2, 64, 16, dtype)
    q = torch.randn(15, 4, 64).to(TYPES[dtype])
    masks = [tree_bits(np.random.default_rng(1), n) for n in new]
    ref = tree_reference(c, q, masks, 0.1)
    rows = {0: slice(0, 4), 1: slice(4, 9), 2: slice(9, 15)}
    saved = (c.indices.copy(), c.last.copy(), c.new_indptr.copy(), c.indptr.copy())

    def check(flag, good):
        o, lse, flags = _run(c, q, masks, 1, 0.1, dtype)
        assert flags == flag
        for b in good:
            check_tree(o[rows[b]], lse[rows[b]], tuple(x[rows[b]] for x in ref), dtype, b)
        c.indices, c.last, c.new_indptr, c.indptr = (x.copy() for x in saved)
        return o, lse

    c.indices[int(c.indptr[1]) + 1] = c.total + 5  # a page of request 1: its 16 tokens count as absent
    o, lse = check(pd.PD_FLAG_BAD_PAGE_ID, [0, 2])
    assert bool(torch.isfinite(o).all()) and bool(torch.isfinite(lse).all())
    # 20 tokens with a last page of 1: 17 tokens for 6 nodes is fine; a first page alone with 2 tokens is not
    c.last[2] = -1
    check(pd.PD_FLAG_BAD_LAST_PAGE_LEN, [0, 1])
    c.new_indptr[:] = [0, 4, 4 + 5, 15]
    c.indptr[3] = c.indptr[2]  # request 2 has no page and 6 nodes
    o, lse = check(pd.PD_FLAG_BAD_NEW_ROWS, [0, 1])
    assert float(o[rows[2]].abs().max()) == 0 and bool(torch.isneginf(lse[rows[2]]).all())


@pytest.mark.parametrize("dtype", ["f16", "f32"])
def test_results_repeat_bit_for_bit_and_on_another_stream_and_in_a_graph(dtype):
    import paged_kv_gqa_13_gb300 as pd

    c, q, masks = _case([6000, 700], [17, 33], 8, 2, 128, 16, dtype, "tree")
    a = _run(c, q, masks, 2, 0.1, dtype)
    b = _run(c, q, masks, 2, 0.1, dtype)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    s = _run(c, q, masks, 2, 0.1, dtype, stream=side)
    code = {"f32": pd.PD_F32, "f16": pd.PD_F16}[dtype]
    ws = pd.alloc_workspace(pd.pd_paged_tree_decode_workspace_bytes(8, 2, 128, code))
    dev = [x.cuda() for x in (q, c.k, c.v)]
    t, m = c.table(), pack(masks, 2).cuda()
    o, lse = torch.empty_like(dev[0]), torch.empty(50, 8, device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pd.pd_paged_tree_decode(*dev, *t, m, o, lse, 0.1, ws)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    for x in (b, s, (o, lse)):
        assert torch.equal(a[0], x[0]) and torch.equal(a[1], x[1])


def test_one_node_without_a_tree_is_the_decode():
    """A chain of one node is pd_paged_decode's call."""
    import paged_kv_gqa_13_gb300 as pd

    kv = [1, 500, 77, 3000]
    c, q, masks = _case(kv, [1] * 4, 8, 2, 128, 16, "bf16", "chain")
    o, lse, _ = _run(c, q, None, 0, 0.1, "bf16")
    ws = pd.alloc_workspace(pd.pd_paged_decode_workspace_bytes(4, 8, 2, 128, pd.PD_BF16))
    o2, lse2 = torch.empty_like(o), torch.empty_like(lse)
    i, p, l, _ = c.table()
    pd.pd_paged_decode(q.cuda(), c.k.cuda(), c.v.cuda(), i, p, l, o2, lse2, 0.1, ws)
    assert float((o.float() - o2.float()).abs().max()) < 2e-2 and float((lse - lse2).abs().max()) < 1e-4


@pytest.mark.parametrize("dtype", ["bf16"])
def test_pools_past_two_to_the_31_elements(dtype):
    import paged_kv_gqa_13_gb300 as pd

    if torch.cuda.get_device_properties(0).total_memory < (60 << 30):
        pytest.skip("needs a large card")
    small = Paged([300], [7], 2, 128, 16, dtype)
    total = (1 << 31) // (2 * 16 * 128) * 2 + 100  # 2^32 elements and a few
    pages = len(small.indices)
    far = torch.arange(total - pages, total, dtype=torch.int32)
    k = torch.empty(total, 2, 16, 128, dtype=TYPES[dtype], device="cuda")
    v = torch.empty_like(k)
    at = torch.from_numpy(small.indices.astype(np.int64))
    k[total - pages:], v[total - pages:] = small.k[at].cuda(), small.v[at].cuda()
    q = torch.randn(7, 8, 128).to(TYPES[dtype])
    masks = [tree_bits(np.random.default_rng(0), 7)]
    ws = pd.alloc_workspace(pd.pd_paged_tree_decode_workspace_bytes(8, 2, 128, pd.PD_BF16))
    o, lse = torch.empty(7, 8, 128, dtype=TYPES[dtype], device="cuda"), torch.empty(7, 8, device="cuda")
    _, p, l, n = small.table()
    pd.pd_paged_tree_decode(q.cuda(), k, v, far.cuda(), p, l, n, pack(masks, 1).cuda(), o, lse, 0.1, ws)
    assert pd.pd_read_device_flags(ws) == 0
    check_tree(o, lse, tree_reference(small, q, masks, 0.1), dtype)
    # and an append and a commit there
    rows = torch.randn(7, 2, 128).to(TYPES[dtype]).cuda()
    pd.pd_paged_rope_append(None, rows, rows, None, None, None, k, v, far.cuda(), p, l, n, ws)
    rq, rr = small.rows(0, np.arange(293, 300))
    order = {int(x): i for i, x in enumerate(small.indices)}
    page = torch.tensor([total - pages + order[int(x)] for x in rq])
    assert torch.equal(v[page.cuda(), :, rr.cuda()], rows)
    path = torch.tensor([[1, 3, 6]], dtype=torch.int32, device="cuda")
    pd.pd_paged_tree_commit(k, v, far.cuda(), p, l, n, path, torch.tensor([3], dtype=torch.int32, device="cuda"), ws)
    assert torch.equal(v[page[:3].cuda(), :, rr[:3].cuda()], rows[[1, 3, 6]])
    assert pd.pd_read_device_flags(ws) == 0


@pytest.mark.parametrize("dtype,fp8", [("f32", False), ("f16", False), ("bf16", True)])
def test_tensors_that_start_16_bytes_off(dtype, fp8):
    """q and o need 16-byte alignment and no more."""
    import paged_kv_gqa_13_gb300 as pd

    c = Paged([300, 9], [3, 9], 2, 128, 16, dtype, fp8=fp8)
    q = torch.randn(12, 4, 128).to(TYPES[dtype])
    masks = [tree_bits(np.random.default_rng(0), n) for n in c.new]
    off = 16 // q.element_size()
    qd, o = (torch.empty(q.numel() + off, dtype=q.dtype, device="cuda")[off:].view(q.shape) for _ in range(2))
    qd.copy_(q)
    lse = torch.empty(12, 4, device="cuda")
    code = {"f32": pd.PD_F32, "f16": pd.PD_F16, "bf16": pd.PD_BF16}[dtype]
    ws = pd.alloc_workspace(pd.pd_paged_tree_decode_workspace_bytes(4, 2, 128, code))
    scales = (c.k_scale.cuda(), c.v_scale.cuda()) if fp8 else ()
    fn = pd.pd_paged_tree_decode_fp8 if fp8 else pd.pd_paged_tree_decode
    fn(qd, c.k.cuda(), c.v.cuda(), *scales, *c.table(), pack(masks, 1).cuda(), o, lse, 0.1, ws)
    check_tree(o, lse, tree_reference(c, q, masks, 0.1), dtype)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("size", [1e-30, 3e4])
def test_q_of_extreme_size_over_e4m3_pools(dtype, size):
    """bf16 rows far outside the range of f16, and rows of zeros, keep their scores."""
    if dtype == "f16" and size < 1e-7:
        pytest.skip("not an f16 value")
    c = Paged([300], [5], 2, 128, 16, dtype, fp8=True)
    q = torch.randn(5, 4, 128).to(TYPES[dtype]) * size
    q = q.clamp(-6e4, 6e4).to(TYPES[dtype])
    q[2] = 0
    masks = [tree_bits(np.random.default_rng(0), 5)]
    scale = 0.1 / size
    o, lse, _ = _run(c, q, masks, 1, scale, dtype)
    check_tree(o, lse, tree_reference(c, q, masks, float(np.float32(scale))), dtype)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n", [3, 90])
def test_a_copy_that_never_lands_is_reported_and_later_calls_are_right(fp8, n):
    import paged_kv_gqa_13_gb300 as pd

    c = Paged([40000, 100], [n, 3], 2, 128, 16, "bf16", fp8=fp8)  # long enough for the first CTA to have a copy
    q = torch.randn(n + 3, 4, 128).bfloat16()
    masks = [tree_bits(np.random.default_rng(0), m) for m in c.new]
    ws = pd.alloc_workspace(pd.pd_paged_tree_decode_workspace_bytes(4, 2, 128, pd.PD_BF16))
    pd.pd_test_inject_wait_timeout(16)
    try:
        _, _, flags = _run(c, q, masks, 3, 0.1, "bf16", ws=ws)
    finally:
        pd.pd_test_inject_wait_timeout(0)
    assert flags & pd.PD_FLAG_WAIT_TIMEOUT
    pd.pd_workspace_init(ws)
    o, lse, flags = _run(c, q, masks, 3, 0.1, "bf16", ws=ws)
    assert flags == 0
    check_tree(o, lse, tree_reference(c, q, masks, 0.1), "bf16")


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("kind", ["chain", "tree", "nothing"])
@pytest.mark.parametrize("hq,hk", [(2, 2), (8, 2), (16, 1)])
@pytest.mark.parametrize("kv,new", [([6000, 0, 33, 1], [2, 0, 1, 1]), ([500, 40, 77, 2100, 9], [1, 2, 0, 13, 1])])
def test_few_rows_in_f32(d, kind, hq, hk, kv, new):
    """Row tiles of 8, 16 and 32 rows; requests that have more rows than a tile, and none."""
    _case(kv, new, hq, hk, d, 16, "f32", kind)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n", [2, 4, 9])
def test_few_rows_in_f32_next_to_what_they_do_not_attend(d, n):
    c = Paged([n + 70], [n], 2, d, 16, "f32")
    q = torch.randn(n, 4, d)
    masks = [np.eye(n, dtype=bool)]
    clean, clean_lse, _ = _run(c, q, masks, 1, 0.1, "f32")
    p, r = c.rows(0, [70 + 1])
    c.k[p, :, r] = math.nan
    c.v[p, :, r] = math.inf
    o, lse, flags = _run(c, q, masks, 1, 0.1, "f32")
    rows = [i for i in range(n) if i != 1]
    assert flags == 0
    assert torch.equal(o[rows], clean[rows]) and torch.equal(lse[rows], clean_lse[rows])
    assert bool(torch.isnan(o[1]).any())
