"""Norms of q and k heads with the rotation in the same pass, alone and on the way into pools that exist."""
import numpy as np
import pytest
import torch

from block_helpers import codes_of, norm_reference, norm_rope_reference, norm_rope_tolerance
from spec_helpers import TYPES, Paged

pytestmark = pytest.mark.gpu

EPS = 1e-6


def _freqs(rot, theta=500000.0):
    """The library's table and the frequencies in radians."""
    import paged_kv_gqa_13_gb300 as pd

    if rot == 0:
        return None, np.zeros(0)
    freqs, _ = pd.pd_rope_frequencies(rot, theta)
    return freqs, theta ** (-2.0 * np.arange(rot // 2) / rot)


def _check(got, x, weight, positions, inv, layout, dtype, scale=1.0, eps=EPS):
    normed = norm_reference(x, weight, eps)
    ref = norm_rope_reference(x, weight, eps, positions, inv, layout, scale)
    off = (got.double().cpu() - ref).abs() - norm_rope_tolerance(ref, normed, dtype, scale)
    assert not torch.isnan(got).any() and float(off.max()) <= 0, float(off.max())


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("tokens,hq,hk,d,rot", [(1, 32, 8, 128, 128), (3, 5, 1, 64, 64), (17, 4, 2, 256, 128), (40, 3, 0, 128, 64),
                                                (33, 2, 2, 80, 80), (16, 1, 3, 96, 32), (15, 2, 1, 192, 64), (5, 3, 1, 2, 2),
                                                (31, 2, 2, 20, 6), (7, 2, 1, 128, 0), (200, 7, 2, 128, 96), (18, 1, 1, 254, 254)])
def test_norm_rope(dtype, layout, tokens, hq, hk, d, rot):
    import paged_kv_gqa_13_gb300 as pd

    g = torch.Generator().manual_seed(tokens + d)
    qkv = (torch.randn(tokens, hq + 2 * hk, d, generator=g) * torch.exp2(torch.randint(-4, 5, (tokens, 1, 1), generator=g))).to(TYPES[dtype])
    qw, kw = ((1 + 0.3 * torch.randn(d, generator=g)).to(TYPES[dtype]) for _ in range(2))
    positions = torch.randint(-5, 200000, (tokens,), generator=g, dtype=torch.int32)
    freqs, inv = _freqs(rot)
    dev = qkv.cuda()
    q, k = dev[:, :hq], dev[:, hq:hq + hk] if hk else None
    qo = torch.full((tokens, hq, d), 7.0, dtype=TYPES[dtype], device="cuda")
    ko = torch.full((tokens, hk, d), 7.0, dtype=TYPES[dtype], device="cuda") if hk else None
    scale = 1.25 if rot else 1.0
    pd.pd_norm_rope(q, k, qw.cuda(), kw.cuda() if hk else None, positions.cuda(), freqs, qo, ko, EPS, layout, scale)
    _check(qo, qkv[:, :hq], qw, positions, inv, layout, dtype, scale)
    if hk:
        _check(ko, qkv[:, hq:hq + hk], kw, positions, inv, layout, dtype, scale)
    # in place, without weights, in views of one projection: what lies between stays
    pd.pd_norm_rope(q, k, None, None, positions.cuda(), freqs, q, k, EPS, layout, scale)
    _check(q, qkv[:, :hq], None, positions, inv, layout, dtype, scale)
    if hk:
        _check(k, qkv[:, hq:hq + hk], None, positions, inv, layout, dtype, scale)
        assert torch.equal(dev[:, hq + hk:].cpu(), qkv[:, hq + hk:])


def test_no_tokens_and_rows_of_nothing():
    import paged_kv_gqa_13_gb300 as pd

    freqs, inv = _freqs(64)
    e = torch.empty(0, 4, 64, device="cuda")
    pd.pd_norm_rope(e, None, None, None, torch.empty(0, dtype=torch.int32, device="cuda"), freqs, e, None)
    # rows of zeros stay zeros, rows far below eps are scaled by 1 / sqrt(eps)
    x = torch.zeros(3, 4, 64)
    x[1] = 1e-8 * torch.randn(4, 64)
    x[2] = 1e15
    out = torch.empty(3, 4, 64, device="cuda")
    positions = torch.arange(3, dtype=torch.int32)
    pd.pd_norm_rope(x.cuda(), None, None, None, positions.cuda(), freqs, out, None, 1e-6)
    assert torch.equal(out[0].cpu(), torch.zeros(4, 64))
    _check(out, x, None, positions, inv, 0, "f32")


def test_far_positions_and_every_slice():
    import paged_kv_gqa_13_gb300 as pd

    freqs, inv = _freqs(128)
    x = torch.randn(2, 100, 128, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16)
    positions = torch.tensor([2 ** 31 - 1, -(2 ** 31)], dtype=torch.int32)
    turns = freqs.cpu().numpy().view(np.uint64)
    out = torch.empty_like(x, device="cuda")
    pd.pd_norm_rope(x.cuda(), x.cuda()[:, :3].clone(), None, None, positions.cuda(), freqs, out, torch.empty(2, 3, 128, dtype=x.dtype, device="cuda"))
    # the table's own fraction of a turn, exactly
    angle = np.array([[float((int(p) * int(t)) % (1 << 64)) / 2.0 ** 64 * 2 * np.pi for t in turns] for p in positions])
    y = norm_reference(x, None, 1e-6)
    c, s = torch.from_numpy(np.cos(angle))[:, None], torch.from_numpy(np.sin(angle))[:, None]
    ref = torch.cat([y[..., :64] * c - y[..., 64:] * s, y[..., 64:] * c + y[..., :64] * s], -1)
    off = (out.double().cpu() - ref).abs() - norm_rope_tolerance(ref, y, "bf16")
    assert float(off.max()) <= 0


def test_a_row_with_an_infinity_or_nan_spoils_itself_only():
    import paged_kv_gqa_13_gb300 as pd

    freqs, inv = _freqs(64)
    x = torch.randn(20, 3, 128, generator=torch.Generator().manual_seed(4))
    x[4, 1, 5], x[9, 0, 120] = float("inf"), float("nan")
    out = torch.empty_like(x, device="cuda")
    positions = torch.arange(20, dtype=torch.int32)
    pd.pd_norm_rope(x.cuda(), None, None, None, positions.cuda(), freqs, out, None)
    spoiled = torch.isnan(out).any(-1).cpu()
    want = torch.zeros(20, 3, dtype=torch.bool)
    want[4, 1] = want[9, 0] = True
    assert torch.equal(spoiled, want)
    # the infinite head's other elements are 0, those that meet the infinity in a rotation are not numbers
    assert bool((out[4, 1, 64:] == 0).all())


@pytest.mark.parametrize("dtype,pool", [("f32", "f32"), ("f16", "f16"), ("bf16", "bf16"), ("f16", "e4m3"), ("bf16", "e4m3")])
@pytest.mark.parametrize("layout,hq,hk,d,rot,page,given", [(0, 8, 2, 128, 128, 16, False), (1, 0, 3, 64, 32, 20, True),
                                                           (0, 5, 1, 256, 256, 7, False), (1, 4, 4, 128, 6, 16, True)])
def test_norm_append_into_plain_and_head_scaled_pools(dtype, pool, layout, hq, hk, d, rot, page, given):
    import paged_kv_gqa_13_gb300 as pd

    fp8 = pool == "e4m3"
    new = [1, 0, 33, 5, 1, 16]
    kv = [1, 9, 50, 5, 90, 16 + 3 * page]
    c = Paged(kv, new, hk, d, page, dtype, seed=d + page, fp8=fp8)
    g = torch.Generator().manual_seed(9)
    t = sum(new)
    qkv = torch.randn(t, hq + 2 * hk, d, generator=g).to(TYPES[dtype])
    qw, kw = ((1 + 0.3 * torch.randn(d, generator=g)).to(TYPES[dtype]) for _ in range(2))
    at = torch.from_numpy(np.concatenate([np.arange(l - n, l) for l, n in zip(kv, new)])).int()
    positions = at * 3 + 11 if given else at
    freqs, inv = _freqs(rot)
    dev, k, v = qkv.cuda(), c.k.cuda(), c.v.cuda()
    ws = pd.alloc_workspace(256)
    qo = torch.full((t, hq, d), 7.0, dtype=TYPES[dtype], device="cuda") if hq else None
    scales = (c.k_scale.cuda(), c.v_scale.cuda()) if fp8 else ()
    call = pd.pd_paged_norm_rope_append_fp8 if fp8 else pd.pd_paged_norm_rope_append
    call(dev[:, :hq] if hq else None, dev[:, hq:hq + hk], dev[:, hq + hk:], qw.cuda(), kw.cuda(),
         positions.cuda() if given else None, freqs, qo, *scales, k, v, *c.table(), ws, EPS, layout)
    assert pd.pd_read_device_flags(ws) == 0
    if hq:
        _check(qo, qkv[:, :hq], qw, positions, inv, layout, dtype)
    k, v = k.cpu(), v.cpu()
    touched = torch.zeros(c.total, page, dtype=torch.bool)
    for b, (l, n) in enumerate(zip(kv, new)):
        p, r = c.rows(b, np.arange(l - n, l))
        touched[p, r] = True
        s = int(c.new_indptr[b])
        kn, vn = qkv[s:s + n, hq:hq + hk], qkv[s:s + n, hq + hk:]
        normed = norm_reference(kn, kw, EPS)
        ref = norm_rope_reference(kn, kw, EPS, positions[s:s + n], inv, layout)
        if not fp8:
            assert torch.equal(v[p, :, r], vn)
            if n:
                off = (k[p, :, r].double() - ref).abs() - norm_rope_tolerance(ref, normed, dtype)
                assert float(off.max()) <= 0
            continue
        assert torch.equal(v[p, :, r], codes_of(vn.float() / c.v_scale[:, None]))
        if n:
            ks = c.k_scale.double()[:, None]
            lim = ref.clamp(-448 * ks, 448 * ks)
            tol = norm_rope_tolerance(ref, normed, None) + 2.0 ** -4 * lim.abs() + 2.0 ** -10 * ks
            assert bool(((c.value(k[p, :, r], c.k_scale) - lim).abs() <= tol).all())
    for x, was in ((k, c.k), (v, c.v)):  # every other row keeps its bits
        bits = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[x.element_size()]
        assert torch.equal(x.view(bits).permute(0, 2, 1, 3)[~touched], was.view(bits).permute(0, 2, 1, 3)[~touched])


def test_bad_tables_are_flagged_and_nothing_is_written():
    import paged_kv_gqa_13_gb300 as pd

    kv, new = [20, 40, 33], [4, 20, 3]
    c = Paged(kv, new, 2, 64, 16, "bf16")
    freqs, inv = _freqs(64)
    x = torch.randn(27, 8, 64, dtype=torch.bfloat16, generator=torch.Generator().manual_seed(1))
    positions = torch.arange(27, dtype=torch.int32)

    def run(indices=None, indptr=None, last=None, new_indptr=None):
        k, v = c.k.cuda(), c.v.cuda()
        ind, ptr, lst, nptr = (torch.from_numpy(np.asarray(a if b is None else b, np.int32)).cuda() for a, b in
                               ((c.indices, indices), (c.indptr, indptr), (c.last, last), (c.new_indptr, new_indptr)))
        ws = pd.alloc_workspace(256)
        qo = torch.zeros(27, 4, 64, dtype=torch.bfloat16, device="cuda")
        dev = x.cuda()
        pd.pd_paged_norm_rope_append(dev[:, :4], dev[:, 4:6], dev[:, 6:], None, None, positions.cuda(), freqs, qo, k, v, ind, ptr,
                                     lst, nptr, ws)
        return pd.pd_read_device_flags(ws), k.cpu(), v.cpu(), qo

    def unchanged(k, v, requests):
        for b in range(3):
            p, r = c.rows(b, np.arange(kv[b] - new[b], kv[b]))
            same = torch.equal(k[p, :, r].view(torch.int16), c.k[p, :, r].view(torch.int16))
            assert same == (b in requests), b

    flags, k, v, qo = run()
    assert flags == 0
    unchanged(k, v, [])
    bad = c.indices.copy()
    bad[c.indptr[2] - 1] = c.total  # the page of request 1's last rows
    flags, k, v, qo = run(indices=bad)
    assert flags == pd.PD_FLAG_BAD_PAGE_ID
    _check(qo, x[:, :4], None, positions, inv, 0, "bf16")  # positions are given: every q row is turned
    p, r = c.rows(1, np.arange(32, 40))
    assert torch.equal(k[p, :, r].view(torch.int16), c.k[p, :, r].view(torch.int16))
    flags, k, v, qo = run(last=[17, c.last[1], c.last[2]])
    assert flags == pd.PD_FLAG_BAD_LAST_PAGE_LEN
    unchanged(k, v, [0])
    flags, k, v, qo = run(new_indptr=[0, 4, 24, 26])  # the last row is no request's: flagged, as by pd_paged_rope_append
    assert flags == pd.PD_FLAG_BAD_NEW_ROWS
    flags, k, v, qo = run(new_indptr=[0, 24, 4, 27])
    assert flags & pd.PD_FLAG_BAD_NEW_ROWS
    flags, k, v, qo = run(new_indptr=[0, 4, 24, 1000])
    assert flags == pd.PD_FLAG_BAD_NEW_ROWS
    unchanged(k, v, [2])
    flags, k, v, qo = run(indptr=[0, c.indptr[1], 1000, 1000])
    assert flags & pd.PD_FLAG_BAD_INDPTR
    unchanged(k, v, [1, 2])


def test_captured_on_a_stream_of_its_own():
    import paged_kv_gqa_13_gb300 as pd

    freqs, inv = _freqs(128)
    x = torch.randn(5, 6, 128, device="cuda")
    out = torch.empty_like(x)
    positions = torch.arange(5, dtype=torch.int32, device="cuda")
    pd.pd_norm_rope(x, None, None, None, positions, freqs, out, None)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pd.pd_norm_rope(x, None, None, None, positions, freqs, out, None)
    x.copy_(torch.randn(5, 6, 128))
    positions.add_(100)
    g.replay()
    torch.cuda.synchronize()
    _check(out, x.cpu(), None, positions.cpu(), inv, 0, "f32")
