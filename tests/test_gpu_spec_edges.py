"""Edges of the speculative-decoding calls: rows in place, empty tables, NaN, bits of copied rows."""

import math

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


def _tree(c, q, masks, words, sm_scale, dtype):
    """(o, lse, flags)"""
    import paged_kv_gqa_13_gb300 as pd
    from tests.spec_helpers import pack

    hq, d = q.shape[1:]
    ws = pd.alloc_workspace(pd.pd_paged_tree_decode_workspace_bytes(hq, c.k.shape[1], d, {"f32": 0, "f16": 1, "bf16": 2}[dtype]))
    o = torch.full(q.shape, 7.0, dtype=TYPES[dtype], device="cuda")
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    scales = (c.k_scale.cuda(), c.v_scale.cuda()) if c.fp8 else ()
    fn = pd.pd_paged_tree_decode_fp8 if c.fp8 else pd.pd_paged_tree_decode
    fn(q.cuda(), c.k.cuda(), c.v.cuda(), *scales, *c.table(), None if masks is None else pack(masks, words).cuda(), o, lse,
       sm_scale, ws)
    torch.cuda.synchronize()
    return o.cpu(), lse.cpu(), pd.pd_read_device_flags(ws)


@pytest.mark.parametrize("dtype,fp8,d", [("bf16", False, 64), ("f16", False, 128), ("bf16", True, 64), ("f16", False, 256)])
@pytest.mark.parametrize("hq,nodes", [(4, 3), (16, 20)])
def test_non_finite_values_of_many_short_requests(dtype, fp8, d, hq, nodes):
    """A non-finite V row in every request of one block: segment after segment of every worker has one to add."""
    hk, batch = 2, 1500
    new = [nodes] * batch
    c = Paged([n + 11 for n in new], new, hk, d, 8, dtype, fp8=fp8)
    q = torch.randn(sum(new), hq, d).to(TYPES[dtype])
    clean, clean_lse, _ = _tree(c, q, None, 0, 0.1, dtype)
    bad = 1  # the node with the row
    for b in range(batch):
        p, r = c.rows(b, [11 + bad])
        if fp8:
            c.v[p, :, r, 5] = 0x7F
        else:
            c.v[p, :, r, 5] = math.inf
    o, lse, flags = _tree(c, q, None, 0, 0.1, dtype)
    assert flags == 0 and torch.equal(lse, clean_lse)
    o, clean = o.view(batch, nodes, hq, d), clean.view(batch, nodes, hq, d)
    rest = [i for i in range(d) if i != 5]
    assert torch.equal(o[:, :, :, rest], clean[:, :, :, rest]) and torch.equal(o[:, :bad], clean[:, :bad])
    assert int(torch.isfinite(o[:, bad:, :, 5]).sum()) == 0


NAN_FORMS = [("f32", False, 64), ("f32", False, 128), ("f32", False, 256), ("f16", False, 128), ("bf16", False, 64),
             ("bf16", False, 256), ("f16", True, 128), ("bf16", True, 64), ("bf16", True, 256)]


@pytest.mark.parametrize("dtype,fp8,d", NAN_FORMS)
@pytest.mark.parametrize("kv,n", [(3, 3), (40, 3), (9000, 3), (30, 20), (9000, 40)])
def test_nan_in_q_makes_its_rows_nan(dtype, fp8, d, kv, n):
    """Whether the segment is cut or not: o and lse of the row are NaN, never those of a row that attends nothing."""
    hq, hk = 8, 2
    c = Paged([kv, 70], [n, 2], hk, d, 16, dtype, fp8=fp8)
    q = torch.randn(n + 2, hq, d).to(TYPES[dtype])
    masks = [np.tril(np.ones((m, m), bool)) for m in (n, 2)]
    masks[0][0] = False
    masks[0][0, 0] = True
    clean, clean_lse, _ = _tree(c, q, masks, 2, 0.1, dtype)
    broken = q.clone()
    broken[1, 3, 7] = math.nan
    broken[n - 1, 6] = math.nan
    o, lse, flags = _tree(c, broken, masks, 2, 0.1, dtype)
    hit = torch.zeros(n + 2, hq, dtype=torch.bool)
    hit[1, 3] = hit[n - 1, 6] = True
    assert flags == 0
    assert bool(torch.isnan(lse[hit]).all()) and bool(torch.isnan(o[hit]).all())
    assert torch.equal(o[~hit], clean[~hit]) and torch.equal(lse[~hit], clean_lse[~hit])


@pytest.mark.parametrize("dtype,fp8,d", NAN_FORMS)
@pytest.mark.parametrize("kv", [12, 9000])
def test_nan_in_a_cached_key_makes_every_row_nan(dtype, fp8, d, kv):
    hq, hk, n = 4, 2, 3
    c = Paged([kv, 70], [n, 2], hk, d, 16, dtype, fp8=fp8)
    q = torch.randn(n + 2, hq, d).to(TYPES[dtype])
    clean, clean_lse, _ = _tree(c, q, None, 0, 0.1, dtype)
    p, r = c.rows(0, [kv - n - 1])
    c.k[p, 0, r, 3] = 0x7F if fp8 else math.nan
    o, lse, flags = _tree(c, q, None, 0, 0.1, dtype)
    assert flags == 0
    assert bool(torch.isnan(lse[:n, :2]).all()) and bool(torch.isnan(o[:n, :2]).all())
    assert torch.equal(o[:n, 2:], clean[:n, 2:]) and torch.equal(lse[:n, 2:], clean_lse[:n, 2:])
    assert torch.equal(o[n:], clean[n:]) and torch.equal(lse[n:], clean_lse[n:])


@pytest.mark.parametrize("elem", [1, 2, 4])
@pytest.mark.parametrize("n,length", [(6, 3), (64, 50), (100, 80)])
@pytest.mark.parametrize("where", ["from", "to", "late"])
def test_commit_leaves_a_request_with_a_bad_page_as_it_is(elem, n, length, where):
    import paged_kv_gqa_13_gb300 as pd

    kv, new = [n + 20, n + 9], [n, n]
    c = Paged(kv, new, 3, 64, 2, {1: "f16", 2: "f16", 4: "f32"}[elem], fp8=elem == 1)
    rng = np.random.default_rng(n)
    path = np.stack([np.sort(rng.choice(np.arange(1, n), length, replace=False)) for _ in range(2)]).astype(np.int32)
    t = c.table()
    # the page of the last node's row, of its place, or of a place in the middle
    token = 20 + {"from": int(path[0, -1]), "to": length - 1, "late": length // 2}[where]
    t[0][int(c.indptr[0]) + token // 2] = -1
    k, v, ws = c.k.cuda(), c.v.cuda(), pd.alloc_workspace(256)
    pd.pd_paged_tree_commit(k, v, *t, torch.from_numpy(path).cuda(), torch.full((2,), length, dtype=torch.int32, device="cuda"), ws)
    assert pd.pd_read_device_flags(ws) == pd.PD_FLAG_BAD_PAGE_ID
    for got, old in ((k.cpu(), c.k), (v.cpu(), c.v)):
        want = old.clone()
        src, dst = c.rows(1, 9 + path[1].astype(np.int64)), c.rows(1, 9 + np.arange(length))
        want[dst[0], :, dst[1]] = old[src[0], :, src[1]]
        assert torch.equal(got.view(torch.uint8), want.view(torch.uint8))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("off", [0, 1])
@pytest.mark.parametrize("layout", [0, 1])
def test_copied_elements_keep_every_bit(dtype, off, layout):
    """v rows, and q and k elements past rot_dim: NaNs of every payload and sign among them."""
    import paged_kv_gqa_13_gb300 as pd

    n, hq, hk, d, rot = 512, 1, 1, 256, 128
    size = 4 if dtype == "f32" else 2
    word = torch.int32 if size == 4 else torch.int16
    bits = torch.arange(n * 128, dtype=torch.int64)  # every 16-bit pattern
    if size == 4:
        bits = bits * 65536 + (bits * 40503) % 65536
        bits = torch.where(bits >= 1 << 31, bits - (1 << 32), bits)
    else:
        bits = torch.where(bits >= 1 << 15, bits - (1 << 16), bits)
    x = torch.zeros(n, hq + 2 * hk, d, dtype=word)
    x[:, :, rot:] = bits.to(word).view(n, 1, 128)
    x[:, hq + hk:, :rot] = bits.to(word).view(n, 1, 128).flip(0)
    flat = torch.zeros(x.numel() + 8, dtype=word, device="cuda")
    flat[off:off + x.numel()] = x.flatten().cuda()  # (off 1: rows off their 16 bytes, one element per access)
    dev = flat[off:off + x.numel()].view(x.shape).view(TYPES[dtype])
    c = Paged([n], [n], hk, d, 16, dtype)
    q_out = torch.empty(n, hq, d, dtype=TYPES[dtype], device="cuda")
    freqs, _ = pd.pd_rope_frequencies(rot)
    k, v, ws = c.k.cuda(), c.v.cuda(), pd.alloc_workspace(256)
    pd.pd_paged_rope_append(dev[:, :hq], dev[:, hq:hq + hk], dev[:, hq + hk:], None, freqs, q_out, k, v, *c.table(), ws,
                            layout=layout)
    p, r = c.rows(0, np.arange(n))
    assert torch.equal(v.cpu().view(word)[p, :, r], x[:, hq + hk:])
    assert torch.equal(k.cpu().view(word)[p, :, r, rot:], x[:, hq:hq + hk, rot:])
    assert torch.equal(q_out.cpu().view(word)[..., rot:], x[:, :hq, rot:])
    out = torch.empty(n, hq + 2 * hk, d, dtype=TYPES[dtype], device="cuda")
    pd.pd_rope(dev, torch.zeros(n, dtype=torch.int32, device="cuda"), freqs, out, layout=layout)
    assert torch.equal(out.cpu().view(word)[..., rot:], x[..., rot:])


@pytest.mark.parametrize("dtype,fp8", [("f32", False), ("bf16", False), ("f16", True)])
def test_a_step_without_a_new_token(dtype, fp8):
    """Tables with requests and no new row: every call returns and writes nothing."""
    import paged_kv_gqa_13_gb300 as pd

    c = Paged([20, 0, 3], [0, 0, 0], 2, 128, 16, dtype, fp8=fp8)
    rows = torch.zeros(0, 6, 128, dtype=TYPES[dtype], device="cuda")
    q_out, lse = torch.empty(0, 2, 128, dtype=TYPES[dtype], device="cuda"), torch.empty(0, 2, device="cuda")
    ws = pd.alloc_workspace(pd.pd_paged_tree_decode_workspace_bytes(2, 2, 128, {"f32": 0, "f16": 1, "bf16": 2}[dtype]))
    k, v, t = c.k.cuda(), c.v.cuda(), c.table()
    scales = (c.k_scale.cuda(), c.v_scale.cuda()) if fp8 else ()
    freqs, _ = pd.pd_rope_frequencies(128)
    pos = torch.empty(0, dtype=torch.int32, device="cuda")
    pd.pd_rope(rows[:, :2], pos, freqs, q_out)
    for p in (pos, None):
        (pd.pd_paged_rope_append_fp8 if fp8 else pd.pd_paged_rope_append)(
            rows[:, :2], rows[:, 2:4], rows[:, 4:], p, freqs, q_out, *scales, k, v, *t, ws)
    for mask in (torch.empty(0, 2, dtype=torch.int32, device="cuda"), None):
        (pd.pd_paged_tree_decode_fp8 if fp8 else pd.pd_paged_tree_decode)(q_out, k, v, *scales, *t, mask, q_out.clone(), lse, 0.1, ws)
    path = torch.zeros(3, 4, dtype=torch.int32, device="cuda")
    pd.pd_paged_tree_commit(k, v, *t, path, torch.zeros(3, dtype=torch.int32, device="cuda"), ws)
    assert pd.pd_read_device_flags(ws) == 0
    assert torch.equal(k.cpu().view(torch.uint8), c.k.view(torch.uint8)) and torch.equal(v.cpu().view(torch.uint8), c.v.view(torch.uint8))


@pytest.mark.parametrize("dtype,fp8", [("f32", False), ("bf16", False), ("f16", True)])
def test_an_allocated_page_that_is_still_empty(dtype, fp8):
    """last_page_len = 0: the new tokens end in the page before, for the append, the tree decode and the commit alike."""
    import paged_kv_gqa_13_gb300 as pd
    from tests.spec_helpers import check_tree, pack, tree_bits, tree_reference

    kv, new, hq, hk, d, page = [48, 16, 32, 21], [5, 16, 1, 4], 4, 2, 64, 16
    c = Paged(kv, new, hk, d, page, dtype, fp8=fp8)
    # a page more for the first three requests, with nothing in it
    spare = [x for x in range(c.total) if x not in set(c.indices.tolist())]
    parts = np.split(c.indices, c.indptr[1:-1])
    parts = [np.append(p, spare[b]).astype(np.int32) if b < 3 else p for b, p in enumerate(parts)]
    indices, indptr = np.concatenate(parts), np.concatenate([[0], np.cumsum([len(p) for p in parts])]).astype(np.int32)
    last = np.array([0, 0, 0, c.last[3]], np.int32)
    t = tuple(torch.from_numpy(x).cuda() for x in (indices, indptr, last, c.new_indptr))
    # the nodes' rows go in by the append
    want_k, want_v = c.k.clone(), c.v.clone()
    n = sum(new)
    x = torch.randn(n, 2 * hk, d).to(TYPES[dtype])
    for b in range(4):
        p, r = c.rows(b, np.arange(kv[b] - new[b], kv[b]))
        rows = slice(int(c.new_indptr[b]), int(c.new_indptr[b + 1]))
        for pool, scale, part in ((want_k, "k_scale", x[rows, :hk]), (want_v, "v_scale", x[rows, hk:])):
            if fp8:
                part = (part.float() / getattr(c, scale)[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            pool[p, :, r] = part
    k, v = c.k.cuda(), c.v.cuda()
    ws = pd.alloc_workspace(pd.pd_paged_tree_decode_workspace_bytes(hq, hk, d, {"f32": 0, "f16": 1, "bf16": 2}[dtype]))
    scales = (c.k_scale.cuda(), c.v_scale.cuda()) if fp8 else ()
    dev = x.cuda()
    (pd.pd_paged_rope_append_fp8 if fp8 else pd.pd_paged_rope_append)(
        None, dev[:, :hk], dev[:, hk:], None, None, None, *scales, k, v, *t, ws)
    assert pd.pd_read_device_flags(ws) == 0
    assert torch.equal(k.cpu().view(torch.uint8), want_k.view(torch.uint8))
    assert torch.equal(v.cpu().view(torch.uint8), want_v.view(torch.uint8))
    c.k, c.v = want_k, want_v
    q = torch.randn(n, hq, d).to(TYPES[dtype])
    masks = [tree_bits(np.random.default_rng(b), m) for b, m in enumerate(new)]
    o, lse = torch.empty(n, hq, d, dtype=TYPES[dtype], device="cuda"), torch.empty(n, hq, device="cuda")
    (pd.pd_paged_tree_decode_fp8 if fp8 else pd.pd_paged_tree_decode)(
        q.cuda(), k, v, *scales, *t, pack(masks, 1).cuda(), o, lse, 0.1, ws)
    assert pd.pd_read_device_flags(ws) == 0
    check_tree(o, lse, tree_reference(c, q, masks, 0.1), dtype)
    path = torch.tensor([[1, 4], [3, 15], [0, 0], [2, 3]], dtype=torch.int32)
    length = torch.tensor([2, 2, 1, 2], dtype=torch.int32)
    pd.pd_paged_tree_commit(k, v, *t, path.cuda(), length.cuda(), ws)
    assert pd.pd_read_device_flags(ws) == 0
    for b in range(4):
        first = kv[b] - new[b]
        src, dst = c.rows(b, first + path[b, :length[b]].numpy()), c.rows(b, first + np.arange(int(length[b])))
        kept = [pool[src[0], :, src[1]].clone() for pool in (c.k, c.v)]
        for pool, rows in zip((want_k, want_v), kept):
            pool[dst[0], :, dst[1]] = rows
    assert torch.equal(k.cpu().view(torch.uint8), want_k.view(torch.uint8))
    assert torch.equal(v.cpu().view(torch.uint8), want_v.view(torch.uint8))
