"""Block-scaled E4M3 pools: what the append writes, older rows under a scale that grows, and reading back."""
import math

import numpy as np
import pytest
import torch

from block_helpers import (BlockPaged, append_reference, codes_of, norm_reference, norm_rope_reference,
                           norm_rope_tolerance, values)
from spec_helpers import TYPES

pytestmark = pytest.mark.gpu

EPS = 1e-6


def _append(c, x, hq, freqs=None, positions=None, weights=(None, None), eps=0.0, layout=0, pools=None, table=None):
    """Runs the append of x [tokens, hq + 2 hk, d] (host); returns flags, pools (host), q_out."""
    import paged_kv_gqa_13_gb300 as pd

    k, v, ks, vs = pools or c.pools()
    hk = k.shape[1]
    dev = x.cuda()
    qo = torch.full((x.shape[0], hq, x.shape[2]), 7.0, dtype=x.dtype, device="cuda") if hq else None
    ws = pd.alloc_workspace(256)
    table = table or (*c.table(), torch.from_numpy(c.new_indptr).cuda())
    pd.pd_paged_rope_append_fp8_blocks(dev[:, :hq] if hq else None, dev[:, hq:hq + hk], dev[:, hq + hk:], positions, freqs, qo,
                                       ks, vs, k, v, *table, ws, *weights, eps, layout)
    return pd.pd_read_device_flags(ws), tuple(y.cpu() for y in (k, v, ks, vs)), qo


def _check_request(c, which, b, got, got_scale, new, exact, slack=None):
    """Request b's blocks after `new` [n, heads, dim] (64 bits, or f32 values exactly) became its last rows."""
    n = new.shape[0]
    if n == 0:
        return
    scales, first, lead, older = append_reference(c, which, b, new, exact)
    starts = np.arange(first, c.kv[b], c.block)
    p, r = c.rows(b, starts)
    s = got_scale[p, :, r // c.block]
    if exact:
        assert torch.equal(s, scales), (which, b)
    else:  # the largest magnitude to a rotation's and a norm's error
        assert float((s / scales - 1).abs().max()) <= 2.0 ** -17, (which, b)
    if lead:
        p, r = c.rows(b, np.arange(first, c.kv[b] - n))
        assert torch.equal(got[p, :, r], older), (which, b)
    p, r = c.rows(b, np.arange(c.kv[b] - n, c.kv[b]))
    each = s.repeat_interleave(c.block, 0)[lead:lead + n]
    if exact:
        want = codes_of(new.float() * (1.0 / each)[..., None])
        assert torch.equal(got[p, :, r], want), (which, b)
    else:
        e = each.double()[..., None]
        lim = new.clamp(-448 * e, 448 * e)
        # half a step of a code, of a subnormal one; a value up to 464 scales becomes 448, within half a step of it
        tol = slack + 2.0 ** -4 * new.abs() + 2.0 ** -10 * e
        assert bool(((values(got[p, :, r]) * e - lim).abs() <= tol).all()), (which, b)


def _others_kept(c, got, got_scale, which):
    """Rows that are no request's last ones, and the scales of untouched blocks, as they were."""
    touched = torch.zeros(c.total, c.page, dtype=torch.bool)
    blocks = torch.zeros(c.total, c.page // c.block, dtype=torch.bool)
    for b, (l, n) in enumerate(zip(c.kv, c.new)):
        if n:
            p, r = c.rows(b, np.arange((l - n) // c.block * c.block, l))
            touched[p, r] = True
            blocks[p, r // c.block] = True
    assert torch.equal(got.permute(0, 2, 1, 3)[~touched], getattr(c, which).permute(0, 2, 1, 3)[~touched])
    was = getattr(c, which + "_scale")
    assert torch.equal(got_scale.permute(0, 2, 1)[~blocks].view(torch.int32), was.permute(0, 2, 1)[~blocks].view(torch.int32))


CASES = [  # page, block, kv, new
    (16, 16, [1, 16, 17, 40, 90, 33], [1, 1, 1, 8, 33, 0]),
    (16, 1, [1, 20, 33], [1, 20, 2]),
    (16, 4, [3, 22, 61, 7], [1, 5, 40, 3]),
    (20, 5, [19, 44, 100], [1, 13, 71]),
    (64, 64, [64, 100, 200, 65], [1, 30, 200, 2]),
    (64, 32, [31, 130], [3, 100]),
    (50, 25, [60, 26, 149], [11, 1, 75]),
    (7, 7, [20, 8, 6], [20, 2, 1]),
]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("hk,d", [(2, 64), (3, 128), (1, 256)])
@pytest.mark.parametrize("page,block,kv,new", CASES)
def test_append_is_the_definition_bit_for_bit(dtype, hk, d, page, block, kv, new):
    """Without norm and rotation nothing is rounded before the codes."""
    c = BlockPaged(kv, hk, d, page, block, new, seed=page + d)
    g = torch.Generator().manual_seed(d)
    # rows of many magnitudes: scales that stay and scales that grow
    x = (torch.randn(sum(new), 2 * hk, d, generator=g) * torch.exp2(torch.randint(-6, 5, (sum(new), 1, 1), generator=g))).to(TYPES[dtype])
    flags, (k, v, ks, vs), _ = _append(c, x, 0)
    assert flags == 0
    for b, n in enumerate(new):
        s = int(c.new_indptr[b])
        _check_request(c, "k", b, k, ks, x[s:s + n, :hk].double(), True)
        _check_request(c, "v", b, v, vs, x[s:s + n, hk:].double(), True)
    _others_kept(c, k, ks, "k")
    _others_kept(c, v, vs, "v")


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("layout,d,rot,hq,norm,given", [(0, 128, 128, 4, True, False), (1, 128, 64, 6, True, True), (0, 64, 64, 0, False, False),
                                                        (1, 256, 256, 2, True, False), (0, 128, 6, 3, True, True), (1, 64, 10, 1, False, True)])
@pytest.mark.parametrize("page,block,kv,new", CASES[:1] + CASES[3:5])
def test_append_with_norm_and_rotation(dtype, layout, d, rot, hq, norm, given, page, block, kv, new):
    import paged_kv_gqa_13_gb300 as pd

    hk, t = 2, sum(new)
    c = BlockPaged(kv, hk, d, page, block, new, seed=page + d)
    g = torch.Generator().manual_seed(d)
    x = (torch.randn(t, hq + 2 * hk, d, generator=g) * 2).to(TYPES[dtype])
    qw, kw = ((1 + 0.3 * torch.randn(d, generator=g)).to(TYPES[dtype]) if norm else None for _ in range(2))
    at = torch.from_numpy(np.concatenate([np.arange(l - n, l) for l, n in zip(kv, new)])).int()
    positions = at + 60000 if given else at
    freqs, _ = pd.pd_rope_frequencies(rot, 500000.0)
    inv = 500000.0 ** (-2.0 * np.arange(rot // 2) / rot)
    eps = EPS if norm else 0.0
    flags, (k, v, ks, vs), qo = _append(c, x, hq, freqs, positions.cuda() if given else None,
                                        tuple(w.cuda() if norm else None for w in (qw, kw)), eps, layout)
    assert flags == 0

    def ref(y, w, pos):
        normed = norm_reference(y, w, EPS) if norm else y.double()
        r = norm_rope_reference(y, w, eps, pos, inv, layout)
        return r, normed

    if hq:
        r, normed = ref(x[:, :hq], qw, positions)
        assert float(((qo.double().cpu() - r).abs() - norm_rope_tolerance(r, normed, dtype)).max()) <= 0
    for b, n in enumerate(new):
        s = int(c.new_indptr[b])
        if n:
            r, normed = ref(x[s:s + n, hq:hq + hk], kw, positions[s:s + n])
            _check_request(c, "k", b, k, ks, r, False, norm_rope_tolerance(r, normed, None))
        _check_request(c, "v", b, v, vs, x[s:s + n, hq + hk:].double(), True)
    _others_kept(c, k, ks, "k")
    _others_kept(c, v, vs, "v")


def test_rows_one_at_a_time_are_as_good_as_rows_together():
    """Every row of a block within the rounding of a code at the block's last scale, however the rows came."""
    block = 16
    g = torch.Generator().manual_seed(1)
    x = (torch.randn(48, 2, 64, generator=g) * torch.exp2(4 * torch.rand(48, 1, 1, generator=g))).to(torch.bfloat16)
    full = BlockPaged([48], 1, 64, 16, block, [48])
    pools = full.pools()
    for t in range(48):
        c = BlockPaged([t + 1], 1, 64, 16, block, [1])
        table = (torch.from_numpy(full.indices[:t // 16 + 1]).cuda(), torch.tensor([0, t // 16 + 1], dtype=torch.int32, device="cuda"),
                 torch.tensor([t % 16 + 1], dtype=torch.int32, device="cuda"), torch.tensor([0, 1], dtype=torch.int32, device="cuda"))
        flags, host, _ = _append(c, x[t:t + 1], 0, pools=pools, table=table)
        assert flags == 0
    k, v, ks, vs = host
    for pool, scale, new in ((k, ks, x[:, :1]), (v, vs, x[:, 1:])):
        p, r = full.rows(0, np.arange(48))
        s = scale[p, :, r // block].double()[..., None]
        got, want = values(pool[p, :, r]) * s, new.double()
        # half a step for the row itself, and half a step of a subnormal code each time that the scale doubles at once (at
        # most 15 rows come after), each at the scale of that time: below 2^-10 s + 2^-10 s / 2 + ...
        tol = 2.0 ** -4 * want.abs() + 2 * 2.0 ** -10 * s
        assert bool(((got - want).abs() <= tol).all())
        top = want.abs().amax(-1).view(3, block).amax(1)
        at = scale[p, :, r // block].double()[::block, 0]
        assert bool((top <= 464 * at).all()) and bool((top * 2 > 447 * at).all())


def test_zeros_infinities_nan_and_the_largest_values():
    block = 4
    x = torch.zeros(20, 2, 64, dtype=torch.bfloat16)
    x[4:8, 0, 3] = 1.0
    x[5, 0, 7], x[6, 0, 8] = float("inf"), float("nan")
    x[7, 0, 9] = -float("inf")
    x[8:12, 0, 0] = torch.finfo(torch.bfloat16).max
    x[12:16, 0, 0] = 1e-38
    x[16, 0] = 5.0
    c = BlockPaged([20], 1, 64, 20, block, [20])
    flags, (k, v, ks, vs), _ = _append(c, x, 0)
    assert flags == 0
    p = int(c.indices[0])
    _check_request(c, "k", 0, k, ks, x[:, :1].double(), True)
    assert float(ks[p, 0, 0]) == 2.0 ** -126 and not k[p, 0, :4].any()  # zeros
    assert k[p, 0, 5, 7] == 0x7E and k[p, 0, 7, 9] == 0xFE and (k[p, 0, 6, 8] & 0x7F) == 0x7F
    assert float(ks[p, 0, 1]) == float(np.float32(1) / np.float32(448))  # infinities and NaN have no say
    assert math.isfinite(float(ks[p, 0, 2])) and k[p, 0, 8, 0] == 0x7E
    assert not v[p, 0].any()


@pytest.mark.parametrize("dtype,magnitude", [(torch.float16, 1.0), (torch.bfloat16, 2.0 ** 126), (torch.bfloat16, 2.0 ** -125)])
def test_zero_blocks_take_larger_rows_later(dtype, magnitude):
    """A block of zeros (scale 2^-126) whose next row is ordinary, and one whose scale was never written."""
    import paged_kv_gqa_13_gb300 as pd

    c = BlockPaged([3, 3], 1, 64, 16, 16, [1, 1])
    for b in range(2):
        p, r = c.rows(b, np.arange(2))
        for pool, scale in ((c.k, c.k_scale), (c.v, c.v_scale)):
            pool[p, :, r] = 0
            scale[p] = 2.0 ** -126 if b == 0 else math.nan
    x = torch.randn(2, 2, 64, generator=torch.Generator().manual_seed(2)).to(dtype) * magnitude
    flags, (k, v, ks, vs), _ = _append(c, x, 0)
    assert flags == 0
    for b in range(2):
        p, r = c.rows(b, np.arange(3))
        s = float(ks[p[0], 0, 0])
        assert math.log2(s) == round(math.log2(s)) and (232 * s < float(x[b, 0].abs().max()) or s == 2.0 ** -126)
        assert float(x[b, 0].abs().max()) <= 464 * s
        assert not k[p[:2], 0, r[:2]].any()
        assert bool(((values(k[p[2], 0, r[2]]) * s - x[b, 0].double()).abs() <= 2.0 ** -4 * x[b, 0].double().abs() + 2.0 ** -10 * s).all())


@pytest.mark.parametrize("what", ["page", "last", "indptr", "rows", "ctx"])
def test_bad_requests_are_flagged_and_keep_their_pools(what):
    import paged_kv_gqa_13_gb300 as pd

    kv, new = [40, 21, 37], [9, 3, 20]
    c = BlockPaged(kv, 2, 64, 16, 8, new, seed=5)
    x = torch.randn(32, 6, 64, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16)
    ind, ptr, last, nptr = c.indices.copy(), c.indptr.copy(), c.last.copy(), c.new_indptr.copy()
    hurt = [1]
    if what == "page":
        ind[ptr[2] - 1] = -1
        want = pd.PD_FLAG_BAD_PAGE_ID
    elif what == "last":
        last[1] = 17
        want = pd.PD_FLAG_BAD_LAST_PAGE_LEN
    elif what == "indptr":
        ptr[2:] = 10000
        want, hurt = pd.PD_FLAG_BAD_INDPTR, [1, 2]
    elif what == "rows":
        nptr[2:] = [5, 32]  # request 1 has none left, request 2 would have 27
        nptr[1] = 9
        want, hurt = pd.PD_FLAG_BAD_NEW_ROWS, [1]
    else:
        last[1], ptr = 1, ptr.copy()
        ptr[2] = ptr[1] + 1  # one row for three new ones; request 2 begins a page early
        want, hurt = pd.PD_FLAG_BAD_NEW_ROWS, [1, 2]
    table = tuple(torch.from_numpy(a).cuda() for a in (ind, ptr, last, nptr))
    flags, (k, v, ks, vs), _ = _append(c, x, 2, table=table)
    assert flags & want
    for b in hurt:
        if what in ("rows", "ctx") and b == 2:
            continue
        p, r = c.rows(b, np.arange(kv[b] // 16 * 16 if what == "page" else kv[b] - new[b], kv[b]))
        assert torch.equal(k[p, :, r], c.k[p, :, r]) and torch.equal(v[p, :, r], c.v[p, :, r])
        assert torch.equal(ks[p, :, r // 8].view(torch.int32), c.k_scale[p, :, r // 8].view(torch.int32))
    if what in ("page", "last"):
        for b in (0, 2):
            s = int(c.new_indptr[b])
            _check_request(c, "v", b, v, vs, x[s:s + new[b], 4:].double(), True)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("hk,d,page,block", [(2, 64, 16, 16), (3, 128, 16, 1), (1, 256, 20, 5), (8, 128, 64, 32)])
@pytest.mark.parametrize("part", [False, True])
def test_read_back(dtype, hk, d, page, block, part):
    import paged_kv_gqa_13_gb300 as pd

    kv = [1, 0, 100, 16, 33, 64]
    c = BlockPaged(kv, hk, d, page, block, seed=d)
    first = [0, 0, 37, 15, 0, 5] if part else [0] * 6
    count = [1, 0, 41, 1, 0, 50] if part else kv
    ptr = np.concatenate([[0], np.cumsum(count)]).astype(np.int32)
    t = int(ptr[-1])
    out = [torch.full((t + 2, hk, d), 7.0, dtype=TYPES[dtype], device="cuda") for _ in range(2)]
    ws = pd.alloc_workspace(256)
    k, v, ks, vs = c.pools()
    pd.pd_paged_read_fp8_blocks(k, v, ks, vs, *c.table(), torch.from_numpy(ptr).cuda(),
                                torch.tensor(first, dtype=torch.int32, device="cuda") if part else None, *out, ws)
    assert pd.pd_read_device_flags(ws) == 0
    for b, n in enumerate(count):
        p, r = c.rows(b, np.arange(first[b], first[b] + n))
        for pool, scale, y in ((c.k, c.k_scale, out[0]), (c.v, c.v_scale, out[1])):
            want = (pool[p, :, r].view(torch.float8_e4m3fn).float() * scale[p, :, r // block][..., None]).to(TYPES[dtype])
            assert torch.equal(y[ptr[b]:ptr[b + 1]].cpu(), want), b
    assert all(bool((y[t:] == 7).all()) for y in out)  # rows past the last request's


def test_read_refuses_tokens_that_are_not_there():
    import paged_kv_gqa_13_gb300 as pd

    c = BlockPaged([20, 30], 2, 64, 16, 16)
    k, v, ks, vs = c.pools()
    ind, ptr, last = c.table()

    def run(out_indptr, first, indices=ind):
        out = [torch.full((40, 2, 64), 7.0, device="cuda") for _ in range(2)]
        ws = pd.alloc_workspace(256)
        pd.pd_paged_read_fp8_blocks(k, v, ks, vs, indices, ptr, last, torch.tensor(out_indptr, dtype=torch.int32, device="cuda"),
                                    torch.tensor(first, dtype=torch.int32, device="cuda"), *out, ws)
        return pd.pd_read_device_flags(ws), out[0].cpu()

    flags, out = run([0, 20, 40], [1, 10])
    assert flags == pd.PD_FLAG_BAD_NEW_ROWS and bool((out[:20] == 7).all()) and not bool((out[20:] == 7).all(-1).any())
    assert run([0, 20, 40], [-1, 10])[0] == pd.PD_FLAG_BAD_NEW_ROWS
    assert run([0, 20, 40], [0, 2147483647])[0] == pd.PD_FLAG_BAD_NEW_ROWS
    assert run([0, 20, 41], [0, 0])[0] == pd.PD_FLAG_BAD_NEW_ROWS
    assert run([20, 0, 10], [0, 0])[0] == pd.PD_FLAG_BAD_NEW_ROWS
    bad = ind.clone()
    bad[1] = c.total
    flags, out = run([0, 20, 40], [0, 0], bad)
    assert flags == pd.PD_FLAG_BAD_PAGE_ID and bool((out[16:20] == 0).all()) and not bool((out[:16] == 0).all(-1).any())


def test_append_then_read_in_one_graph():
    """A step's calls captured on a side stream and replayed over other lengths."""
    import paged_kv_gqa_13_gb300 as pd

    c = BlockPaged([40, 17], 2, 64, 16, 16, [3, 1], seed=1)
    k, v, ks, vs = c.pools()
    ind, ptr, last = c.table()
    nptr = torch.tensor([0, 3, 4], dtype=torch.int32, device="cuda")
    first = torch.tensor([37, 16], dtype=torch.int32, device="cuda")
    x = torch.randn(4, 4, 64, device="cuda").to(torch.bfloat16)
    out = [torch.empty(4, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    ws = pd.alloc_workspace(256)

    def step():
        pd.pd_paged_rope_append_fp8_blocks(None, x[:, :2], x[:, 2:], None, None, None, ks, vs, k, v, ind, ptr, last, nptr, ws)
        pd.pd_paged_read_fp8_blocks(k, v, ks, vs, ind, ptr, last, nptr, first, *out, ws)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for y in (k, v, ks, vs):
        y.copy_({k: c.k, v: c.v, ks: c.k_scale, vs: c.v_scale}[y])
    x.copy_(torch.randn(4, 4, 64) * 3)
    last.copy_(torch.tensor([c.last[0] - 2, c.last[1]], dtype=torch.int32))
    first.copy_(torch.tensor([35, 16], dtype=torch.int32))
    g.replay()
    torch.cuda.synchronize()
    assert pd.pd_read_device_flags(ws) == 0
    for y, new in ((out[0], x[:, :2]), (out[1], x[:, 2:])):
        # half a step of the code and of bf16; half a step of a subnormal code at scales below 1 / 8
        tol = (2.0 ** -4 + 2.0 ** -8) * new.float().abs() + 2.0 ** -13
        assert bool(((y.float() - new.float()).abs() <= tol).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_read_into_rows_that_lie_16_bytes_off_a_sector(dtype):
    import paged_kv_gqa_13_gb300 as pd

    c = BlockPaged([37, 64], 2, 64, 16, 16, seed=5)
    ptr = torch.tensor([0, 37, 101], dtype=torch.int32, device="cuda")
    out, off = [], []
    for shift in (0, 16):
        for _ in range(2):
            n = shift // TYPES[dtype].itemsize
            (off if shift else out).append(torch.zeros(101 * 2 * 64 + n, dtype=TYPES[dtype], device="cuda")[n:].view(101, 2, 64))
    assert all(x.data_ptr() % 32 == 16 for x in off)
    ws = pd.alloc_workspace(256)
    k, v, ks, vs = c.pools()
    for to in (out, off):
        pd.pd_paged_read_fp8_blocks(k, v, ks, vs, *c.table(), ptr, None, *to, ws)
    assert pd.pd_read_device_flags(ws) == 0
    assert torch.equal(out[0], off[0]) and torch.equal(out[1], off[1])
