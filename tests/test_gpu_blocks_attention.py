"""Attention over block-scaled E4M3 pools: one row per request, chains, pieces of prompts and trees."""
import math

import numpy as np
import pytest
import torch

from block_helpers import BlockPaged, attend_reference, check_attention, codes_of
from spec_helpers import TYPES, pack, tree_bits

pytestmark = pytest.mark.gpu


def _workspace(hq, hk, d, dtype):
    import paged_kv_gqa_13_gb300 as pd

    code = pd.PD_F16 if dtype == "f16" else pd.PD_BF16
    return pd.alloc_workspace(max(pd.pd_paged_tree_decode_fp8_blocks_workspace_bytes(hq, hk, d, code),
                                  pd.pd_paged_decode_fp8_blocks_workspace_bytes(16, hq, hk, d, code)))


def _run(c, q, masks=None, sm_scale=None, words=None, single=False, ws=None, table=None, mutate=None):
    import paged_kv_gqa_13_gb300 as pd

    hk, d = c.k.shape[1], c.k.shape[3]
    dtype = "f16" if q.dtype == torch.float16 else "bf16"
    ws = _workspace(q.shape[1], hk, d, dtype) if ws is None else ws
    k, v, ks, vs = c.pools()
    qd = q.cuda()
    o, lse = torch.full_like(qd, 7.0), torch.full(q.shape[:2], 7.0, device="cuda")
    scale = 1 / math.sqrt(d) if sm_scale is None else sm_scale
    ind, ptr, last = table or c.table()
    if single:
        pd.pd_paged_decode_fp8_blocks(qd, k, v, ks, vs, ind, ptr, last, o, lse, scale, ws)
    else:
        mask = None
        if masks is not None:
            mask = pack(masks, words or max(1, -(-max(c.new) // 32))).cuda()
        pd.pd_paged_tree_decode_fp8_blocks(qd, k, v, ks, vs, ind, ptr, last, torch.from_numpy(c.new_indptr).cuda(), mask, o, lse,
                                           scale, ws)
    return pd.pd_read_device_flags(ws), o, lse


def _q(rows, hq, d, dtype, seed=0, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(rows, hq, d, generator=g) * spread).to(TYPES[dtype])


SHAPES = [  # hq, hk, d, page, block
    (8, 2, 128, 16, 16), (32, 8, 128, 16, 1), (8, 1, 64, 16, 4), (7, 7, 256, 16, 16), (28, 4, 128, 20, 5),
    (12, 3, 64, 7, 7), (16, 1, 256, 64, 32), (64, 2, 128, 32, 32), (40, 1, 128, 16, 8), (100, 1, 64, 8, 8), (6, 2, 256, 50, 25),
    (130, 2, 128, 16, 16),
]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("hq,hk,d,page,block", SHAPES)
def test_decode(dtype, hq, hk, d, page, block):
    kv = [1, 0, 127, 128, 129, 300, 16, 1025]
    c = BlockPaged(kv, hk, d, page, block, seed=hq + d)
    q = _q(len(kv), hq, d, dtype)
    flags, o, lse = _run(c, q, single=True)
    assert flags == 0
    check_attention(o, lse, attend_reference(c, q, None, 1 / math.sqrt(d), dtype))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("hq,hk,d,page,block", SHAPES)
@pytest.mark.parametrize("kind,new", [("chain", [1, 5, 0, 17, 40, 3]), ("tree", [7, 1, 12, 0, 33, 64]), ("random", [4, 9, 2, 70, 1, 5]),
                                      ("nothing", [3, 1, 0, 0, 2, 2])])
def test_tree(dtype, hq, hk, d, page, block, kind, new):
    kv = [max(n, x) for n, x in zip(new, [7, 140, 64, 300, 600, 64])]
    c = BlockPaged(kv, hk, d, page, block, new, seed=hq + d + sum(new))
    rng = np.random.default_rng(d)
    masks = None if kind == "chain" else [tree_bits(rng, n, kind) for n in new]
    q = _q(sum(new), hq, d, dtype)
    flags, o, lse = _run(c, q, masks)
    assert flags == 0
    check_attention(o, lse, attend_reference(c, q, masks, 1 / math.sqrt(d), dtype))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("hq,hk,d,page,block,kv,new", [
    (8, 2, 128, 16, 16, [9000], [1]), (8, 2, 64, 16, 1, [20000, 5000], [1, 3]), (4, 4, 256, 16, 4, [3000, 7001], [2, 1]),
    (8, 1, 128, 64, 64, [6000, 300, 2000], [30, 2, 7]), (16, 2, 128, 16, 16, [2500, 900], [300, 900]),
    (4, 1, 64, 7, 7, [4000], [260]), (2, 1, 256, 16, 16, [1500], [400]),
])
def test_long_contexts_cut_and_merged(dtype, hq, hk, d, page, block, kv, new):
    """Requests that are cut over many workers; scores that climb, so that maxima move and O is rescaled."""
    c = BlockPaged(kv, hk, d, page, block, new, seed=sum(kv))
    for b, n in enumerate(kv):  # K grows along the context, and so do V's scales
        p, r = c.rows(b, np.arange(n))
        ramp = torch.linspace(0.2, 2.0, n)
        c.k_scale[p, :, r // block] = 2.0 ** -6 * ramp[:, None]
        c.v_scale[p, :, r // block] = 2.0 ** -7 * (1 + 30 * ramp[:, None])
    q = _q(sum(new), hq, d, dtype, spread=1.5)
    flags, o, lse = _run(c, q)
    assert flags == 0
    ref = attend_reference(c, q, None, 1 / math.sqrt(d), dtype)
    check_attention(o, lse, ref)
    # the same bits again, and with the workspace of the call before
    ws = _workspace(hq, hk, d, dtype)
    for _ in range(3):
        _, o2, lse2 = _run(c, q, ws=ws)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert int(ws[128:132].view(torch.int32)) == 0


@pytest.mark.parametrize("hq,d", [(8, 128), (2, 128), (8, 64)])
def test_one_node_is_the_decode(hq, d):
    """Either kernel of the decode, against the tree decode with one node per request."""
    c = BlockPaged([40, 333, 1, 2000], 2, d, 16, 16)
    q = _q(4, hq, d, "bf16")
    _, o, lse = _run(c, q, single=True)
    _, o2, lse2 = _run(c, q)
    ref = attend_reference(c, q, None, 1 / math.sqrt(d), "bf16")
    check_attention(o, lse, ref)
    check_attention(o2, lse2, ref)
    if hq == 2 or d == 64:  # one kernel for both
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_scales_and_queries_of_very_different_magnitude(dtype):
    """K and V scales over 40 octaves, blocks of zeros, q rows of 2^-20 to 2^10 and with one large element."""
    c = BlockPaged([700, 900], 2, 128, 16, 4, [2, 6], seed=3)
    g = torch.Generator().manual_seed(1)
    for s in (c.k_scale, c.v_scale):
        fine = ~torch.isnan(s)
        s[fine] = torch.exp2(torch.randint(-40, 1, (int(fine.sum()),), generator=g).float() - 8)
    for b in range(2):
        p, r = c.rows(b, np.arange(0, 40))
        c.v[p, :, r] = 0
        c.v_scale[p, :, r // 4] = 2.0 ** -126
    q = _q(8, 4, 128, "f16").float()
    q *= torch.exp2(torch.randint(-20, 8, (8, 4, 1), generator=g).float())
    q[:, :, 5] *= 64
    q = (q * (1.0 if dtype == "bf16" else 0.01)).to(TYPES[dtype])
    flags, o, lse = _run(c, q)
    assert flags == 0
    check_attention(o, lse, attend_reference(c, q, None, 1 / math.sqrt(128), dtype))


def test_v_of_zeros_keeps_lse():
    c = BlockPaged([300, 5], 1, 64, 16, 16, [1, 1])
    c.v[:], c.v_scale[:] = 0, 2.0 ** -126
    q = _q(2, 4, 64, "bf16")
    flags, o, lse = _run(c, q)
    ref = attend_reference(c, q, None, 1 / 8, "bf16")
    assert flags == 0 and not o.any()
    assert float((lse.cpu().double() - ref[1]).abs().max()) <= 1e-4
    c.v_scale[:] = 0.0
    flags, o, lse2 = _run(c, q)
    assert not o.any() and torch.equal(lse, lse2)


def test_negative_and_zero_score_scale():
    c = BlockPaged([300, 50], 2, 128, 16, 16, [3, 2])
    q = _q(5, 8, 128, "bf16")
    for scale in (-0.07, 0.0):
        flags, o, lse = _run(c, q, sm_scale=scale)
        check_attention(o, lse, attend_reference(c, q, None, scale, "bf16"))


def test_what_a_row_does_not_attend_has_no_part():
    """NaN codes and scales past the end (BlockPaged puts them there), NaN in masked node rows' K and V, and in a row's own."""
    rng = np.random.default_rng(5)
    new, kv = [9, 20], [50, 20]
    c = BlockPaged(kv, 2, 64, 16, 1, new, seed=8)
    masks = [tree_bits(rng, n) for n in new]
    masks[0][:, 4] = False
    masks[0][4, :] = False  # node 4 sees the context only, and nobody sees node 4
    masks[1][:, 7] = False
    masks[1][11, 7] = True  # node 11 of request 1 sees node 7
    for b, j in ((0, 4), (1, 7)):
        p, r = c.rows(b, [kv[b] - new[b] + j])
        c.v[p, :, r, 3] = 0x7F
        if b == 0:
            c.k[p, :, r, 9] = 0xFF
            c.k_scale[p, :, r] = math.nan
            c.v_scale[p, :, r] = math.nan
    q = _q(29, 4, 64, "bf16")
    flags, o, lse = _run(c, q, masks)
    assert flags == 0
    spoiled = torch.zeros(29, dtype=torch.bool)
    spoiled[9 + 11] = True
    assert torch.equal(torch.isnan(o[:, :, 3]).all(1).cpu(), spoiled) and not torch.isnan(o[:, :, :3]).any() and not torch.isnan(o[:, :, 4:]).any()
    # the rest as if those elements were zeros
    p, r = c.rows(0, [kv[0] - new[0] + 4])
    c.k_scale[p, :, r], c.v_scale[p, :, r] = 0.01, 0.01
    c.k[p, :, r, 9] = 0
    for b, j in ((0, 4), (1, 7)):
        p, r = c.rows(b, [kv[b] - new[b] + j])
        c.v[p, :, r, 3] = 0
    ref = attend_reference(c, q, masks, 1 / 8, "bf16")
    o = o.clone()
    o[9 + 11, :, 3] = ref[0][9 + 11, :, 3].to(o)
    check_attention(o, lse, ref)


def test_nan_among_attended_scores():
    c = BlockPaged([200, 60, 3000], 1, 64, 16, 16, [2, 1, 1])
    p, r = c.rows(0, [17])
    c.k[p, 0, r, 5] = 0x7F
    p, r = c.rows(2, [2900])
    c.k[p, 0, r, 5] = 0x7F
    q = _q(4, 4, 64, "bf16")
    q[2, 1, 3] = math.nan
    flags, o, lse = _run(c, q)
    bad = torch.zeros(4, 4, dtype=torch.bool)
    bad[:2] = bad[3] = True
    bad[2, 1] = True
    assert torch.equal(torch.isnan(o).all(-1).cpu(), bad) and torch.equal(torch.isnan(o).any(-1).cpu(), bad)
    assert torch.equal(torch.isnan(lse).cpu(), bad)


def test_bad_pages_and_tables():
    import paged_kv_gqa_13_gb300 as pd

    kv, new = [100, 50, 200], [2, 1, 3]
    c = BlockPaged(kv, 2, 128, 16, 16, new, seed=2)
    q = _q(6, 8, 128, "bf16")
    _, o, lse = _run(c, q)
    ind, ptr, last = c.table()
    bad = ind.clone()
    bad[1], bad[int(c.indptr[2]) + 3] = -1, 2 ** 31 - 1
    flags, o2, lse2 = _run(c, q, table=(bad, ptr, last))
    assert flags == pd.PD_FLAG_BAD_PAGE_ID
    assert torch.equal(o[2], o2[2]) and not torch.isnan(o2).any()
    # the page counts as empty: the same as masking its tokens
    for b, page in ((0, 1), (2, 3)):
        k, v = c.held(b)
        keep = torch.ones(kv[b], dtype=torch.bool)
        keep[16 * page:16 * page + 16] = False
        for j in range(new[b]):
            t, seen = int(c.new_indptr[b]) + j, keep.clone()
            seen[kv[b] - new[b] + j + 1:] = False
            for h in range(2):
                x = q[t, 4 * h:4 * h + 4].double() @ k[seen, h].T / math.sqrt(128)
                assert float((torch.logsumexp(x, -1) - lse2[t, 4 * h:4 * h + 4].cpu()).abs().max()) <= 1e-4
    flags, o2, _ = _run(c, q, table=(ind, ptr, torch.tensor([17, c.last[1], c.last[2]], dtype=torch.int32, device="cuda")))
    assert flags == pd.PD_FLAG_BAD_LAST_PAGE_LEN and torch.equal(o[2:], o2[2:])
    flags, o2, lse2 = _run(c, q, table=(ind, torch.tensor([0, 7, 11, 1000], dtype=torch.int32, device="cuda"), last))
    assert flags == pd.PD_FLAG_BAD_INDPTR and torch.equal(o[:3], o2[:3])
    assert not o2[3:].any() and torch.isinf(lse2[3:]).all()
    # more new rows than tokens; without new_indptr an empty request is none
    short = torch.tensor([7, 7, 11, 24], dtype=torch.int32, device="cuda")  # request 0 has no page
    flags, o2, lse2 = _run(c, q, table=(ind, short, last))
    assert flags == pd.PD_FLAG_BAD_NEW_ROWS and not o2[:2].any() and torch.isinf(lse2[:2]).all()
    flags, o2, lse2 = _run(c, q[:3], single=True, table=(ind, short, last))
    assert flags == 0 and not o2[0].any() and torch.isinf(lse2[0]).all() and torch.isfinite(lse2[1:]).all()


def test_no_rows_at_all():
    c = BlockPaged([30, 40], 2, 64, 16, 16, [0, 0])
    flags, o, lse = _run(c, _q(0, 4, 64, "bf16"))
    assert flags == 0 and o.numel() == 0


def test_mask_words_beyond_and_short():
    """Bits past the words count as clear; extra words are ignored."""
    new, kv = [40, 3], [90, 30]
    c = BlockPaged(kv, 1, 128, 16, 16, new, seed=4)
    rng = np.random.default_rng(2)
    masks = [tree_bits(rng, n, "random") for n in new]
    q = _q(43, 4, 128, "f16")
    _, o, lse = _run(c, q, masks, words=5)
    check_attention(o, lse, attend_reference(c, q, masks, 1 / math.sqrt(128), "f16"))
    short = [m.copy() for m in masks]
    short[0][:, 32:] = False
    _, o, lse = _run(c, q, masks, words=1)
    check_attention(o, lse, attend_reference(c, q, short, 1 / math.sqrt(128), "f16"))


def test_captured_and_replayed_over_other_lengths():
    import paged_kv_gqa_13_gb300 as pd

    c = BlockPaged([900, 2500], 2, 128, 16, 16)
    q = _q(2, 8, 128, "bf16")
    k, v, ks, vs = c.pools()
    ind, ptr, last = c.table()
    qd, ws = q.cuda(), _workspace(8, 2, 128, "bf16")
    o, lse = torch.empty_like(qd), torch.empty(2, 8, device="cuda")
    call = lambda: pd.pd_paged_decode_fp8_blocks(qd, k, v, ks, vs, ind, ptr, last, o, lse, 0.1, ws)  # noqa: E731
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    short = BlockPaged([900, 2500], 2, 128, 16, 16)
    short.kv = [900 - 16 * 9, 2500]  # the request's last nine pages go
    n0 = int(c.indptr[1])
    table = torch.cat([ind[:n0 - 9], ind[n0:], ind[n0 - 9:n0]])
    short.indices, short.indptr = table.cpu().numpy(), (c.indptr - np.array([0, 9, 9])).astype(np.int32)
    ind.copy_(table)
    ptr.copy_(torch.from_numpy(short.indptr))
    g.replay()
    torch.cuda.synchronize()
    assert pd.pd_read_device_flags(ws) == 0
    check_attention(o, lse, attend_reference(short, q, None, 0.1, "bf16"))


def test_a_wait_that_runs_out_is_reported():
    import paged_kv_gqa_13_gb300 as pd

    c = BlockPaged([60000, 3000, 100], 2, 128, 16, 16)  # long enough for the first CTA to have a copy
    q = _q(3, 8, 128, "bf16")
    ws = _workspace(8, 2, 128, "bf16")
    _, o, lse = _run(c, q, ws=ws)
    pd.pd_test_inject_wait_timeout(16)
    try:
        flags, _, _ = _run(c, q, ws=ws)
    finally:
        pd.pd_test_inject_wait_timeout(0)
    assert flags & pd.PD_FLAG_WAIT_TIMEOUT
    pd.pd_workspace_init(ws)
    flags, o2, lse2 = _run(c, q, ws=ws)
    assert flags == 0 and torch.equal(o, o2) and torch.equal(lse, lse2)


def test_the_cache_that_the_append_writes():
    """Append a prompt and then tokens one at a time, attend, and read back what was attended."""
    import paged_kv_gqa_13_gb300 as pd

    hq, hk, d, page = 8, 2, 64, 16
    freqs, _ = pd.pd_rope_frequencies(d, 10000.0)
    n = 70
    k = torch.zeros(8, hk, page, d, dtype=torch.uint8, device="cuda")
    v, ks, vs = torch.zeros_like(k), torch.zeros(8, hk, 1, device="cuda"), torch.zeros(8, hk, 1, device="cuda")
    ws = _workspace(hq, hk, d, "bf16")
    x = torch.randn(n, hq + 2 * hk, d, device="cuda").to(torch.bfloat16)
    w = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    ind = torch.tensor([5, 1, 7, 0, 3], dtype=torch.int32, device="cuda")
    at = 0
    for count in (40, 1, 1, 1, 20, 1, 1, 5):
        at += count
        pages = -(-at // page)
        table = (ind[:pages], torch.tensor([0, pages], dtype=torch.int32, device="cuda"),
                 torch.tensor([at - (pages - 1) * page], dtype=torch.int32, device="cuda"))
        nptr = torch.tensor([0, count], dtype=torch.int32, device="cuda")
        new = x[at - count:at]
        q = torch.empty(count, hq, d, dtype=torch.bfloat16, device="cuda")
        o, lse = torch.empty_like(q), torch.empty(count, hq, device="cuda")
        pd.pd_paged_rope_append_fp8_blocks(new[:, :hq], new[:, hq:hq + hk], new[:, hq + hk:], None, freqs, q, ks, vs, k, v, *table,
                                           nptr, ws, w, w, 1e-6)
        pd.pd_paged_tree_decode_fp8_blocks(q, k, v, ks, vs, *table, nptr, None, o, lse, 0.125, ws)
        kr, vr = torch.empty(at, hk, d, device="cuda"), torch.empty(at, hk, d, device="cuda")
        pd.pd_paged_read_fp8_blocks(k, v, ks, vs, *table, torch.tensor([0, at], dtype=torch.int32, device="cuda"), None, kr, vr, ws)
        assert pd.pd_read_device_flags(ws) == 0
        # what is cached, against the rows that went in (a code's half step; subnormals of a scale below 1 / 64)
        want = x[:at, hq + hk:].float()
        assert bool(((vr - want).abs() <= 2.0 ** -4 * want.abs() + 2.0 ** -15).all())
        xs = torch.einsum("ngd,tgd->ngt", q.double(), kr.double().repeat_interleave(hq // hk, 1)) * 0.125
        ban = torch.arange(at, device="cuda") > torch.arange(at - count, at, device="cuda")[:, None]
        xs = xs.masked_fill(ban[:, None], -math.inf)
        ref = torch.einsum("ngt,tgd->ngd", xs.softmax(-1), vr.double().repeat_interleave(hq // hk, 1))
        # parts of a weight 2^-8, the result's half step 2^-8, at values below 5
        assert float((o.double() - ref).abs().max()) <= 2 * 2.0 ** -8 * 5
        assert float((lse.double() - torch.logsumexp(xs, -1)).abs().max()) <= 1e-4


@pytest.mark.parametrize("hq,hk,d,page,block", [(96, 4, 128, 16, 16), (48, 2, 64, 16, 4), (64, 2, 256, 8, 8), (100, 4, 64, 32, 32)])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_many_requests_of_17_to_32_rows(dtype, hq, hk, d, page, block):
    rng = np.random.default_rng(hq)
    kv = [5000, 0, 1, 31] + rng.integers(1, 300, 68).tolist()
    c = BlockPaged(kv, hk, d, page, block, seed=hq + d)
    q = _q(len(kv), hq, d, dtype)
    flags, o, lse = _run(c, q, single=True)
    assert flags == 0
    check_attention(o, lse, attend_reference(c, q, None, 1 / math.sqrt(d), dtype))


@pytest.mark.parametrize("block", [16, 2])
@pytest.mark.parametrize("kind", ["chain", "tree", "random"])
def test_many_trees_of_17_to_32_rows(block, kind):
    rng = np.random.default_rng(block)
    new = rng.integers(6, 18, 72).tolist()
    kv = [n + int(x) for n, x in zip(new, rng.integers(0, 400, 72))]
    c = BlockPaged(kv, 4, 128, 16, block, new, seed=block)
    masks = None if kind == "chain" else [tree_bits(rng, n, kind) for n in new]
    q = _q(sum(new), 8, 128, "bf16")
    flags, o, lse = _run(c, q, masks)
    assert flags == 0
    check_attention(o, lse, attend_reference(c, q, masks, 1 / math.sqrt(128), "bf16"))
