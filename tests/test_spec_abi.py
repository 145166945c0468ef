"""The speculative-decoding calls without a GPU: refusals, and the rotary frequency table."""
import ctypes
import math

import numpy as np
import pytest

FAKE = 1 << 20  # an aligned address that is never dereferenced: every call below fails its checks first


def _freqs(**kw):
    import paged_kv_gqa_13_gb300 as pd

    args = dict(rot_dim=64, theta=10000.0, scaling=pd.PD_ROPE_PLAIN, device="cpu")
    args.update(kw)
    f, scale = pd.pd_rope_frequencies(**args)
    return f.numpy().view(np.uint64).astype(np.longdouble) / np.longdouble(2) ** 64 * 2 * math.pi, scale


def test_plain_and_linear_and_base_frequencies():
    import paged_kv_gqa_13_gb300 as pd

    i = np.arange(32)
    want = 10000.0 ** (-2.0 * i / 64)
    got, scale = _freqs()
    assert scale == 1.0 and np.max(np.abs(got / want - 1)) < 1e-14
    got, _ = _freqs(scaling=pd.PD_ROPE_LINEAR, factor=4.0)
    assert np.max(np.abs(got * 4 / want - 1)) < 1e-14
    got, _ = _freqs(scaling=pd.PD_ROPE_BASE, factor=4.0)
    # the longest wavelength is stretched by the factor, the shortest not at all
    assert abs(got[0] - 1) < 1e-14 and abs(got[-1] * 4 / want[-1] - 1) < 1e-12


def test_banded_and_yarn_keep_short_and_stretch_long_wavelengths():
    import paged_kv_gqa_13_gb300 as pd

    want = 500000.0 ** (-2.0 * np.arange(64) / 128)
    turns = 8192 * want / (2 * math.pi)
    got, scale = _freqs(rot_dim=128, theta=500000.0, scaling=pd.PD_ROPE_BANDED, factor=8.0, low=1.0, high=4.0)
    ratio = np.asarray(got / want, float)
    assert scale == 1.0
    assert np.allclose(ratio[turns > 4], 1, atol=1e-14) and np.allclose(ratio[turns < 1], 1 / 8, atol=1e-14)
    mid = (turns > 1) & (turns < 4)
    assert mid.any() and np.allclose(ratio[mid], (turns[mid] - 1) / 3 * 7 / 8 + 1 / 8, atol=1e-12)
    got, scale = _freqs(rot_dim=128, theta=500000.0, scaling=pd.PD_ROPE_YARN, factor=8.0, low=1.0, high=32.0)
    ratio = np.asarray(got / want, float)
    assert abs(scale - (0.1 * math.log(8.0) + 1)) < 1e-6
    assert np.allclose(ratio[turns > 64], 1) and np.allclose(ratio[turns < 0.5], 1 / 8) and np.all(np.diff(ratio) <= 1e-12)


@pytest.mark.parametrize("kw", [dict(rot_dim=0), dict(rot_dim=3), dict(theta=1.0), dict(theta=float("nan")),
                                dict(scaling=9), dict(scaling=1, factor=0.5), dict(scaling=3, factor=2.0, low=4.0, high=1.0),
                                dict(scaling=4, factor=2.0, original_positions=0), dict(scaling=2, factor=2.0, rot_dim=2)])
def test_frequencies_refuse(kw):
    import paged_kv_gqa_13_gb300 as pd

    with pytest.raises(pd.PagedecodeError):
        _freqs(**kw)


def _call(name, defaults, **kw):
    import paged_kv_gqa_13_gb300 as pd

    assert set(kw) <= set(defaults)
    return getattr(pd._lib, name)(*{**defaults, **kw}.values())


ROPE = dict(x=FAKE, positions=FAKE, freqs=FAKE, out=FAKE, tokens=4, heads=2, d=128, rot=128, xs=256, os=256, layout=0,
            scale=1.0, dtype=2, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), 1), (dict(out=None), 1), (dict(positions=None), 1), (dict(freqs=None), 1), (dict(tokens=-1), 1),
    (dict(heads=0), 1), (dict(d=0), 1), (dict(rot=130), 1), (dict(rot=3), 1), (dict(rot=-2), 1), (dict(xs=255), 1),
    (dict(os=100), 1), (dict(xs=512), 1), (dict(layout=2), 1), (dict(scale=float("inf")), 1), (dict(dtype=5), 2),
    (dict(x=FAKE + 1), 2), (dict(positions=FAKE + 2), 2), (dict(freqs=FAKE + 4), 2)])
def test_rope_refuses(kw, status):
    import paged_kv_gqa_13_gb300 as pd

    assert _call("pd_rope", ROPE, **kw) == status
    assert pd.pd_last_error_string() != ""
    assert _call("pd_rope", ROPE, tokens=0) == 0


APPEND = dict(q=FAKE, k=FAKE, v=FAKE, positions=FAKE, freqs=FAKE, q_out=FAKE, kd=FAKE, vd=FAKE, indices=FAKE, indptr=FAKE,
              last=FAKE, new=FAKE, batch=2, total=4, hq=8, hk=2, d=128, rot=128, page=16, pages=10, nidx=4, qs=1024, ks=256,
              vs=256, layout=0, scale=1.0, dtype=2, ws=FAKE, wsb=256, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(k=None), 1), (dict(v=None), 1), (dict(q=None), 1), (dict(q_out=None), 1), (dict(freqs=None), 1), (dict(kd=None), 1),
    (dict(new=None), 1), (dict(indptr=None), 1), (dict(indices=None), 1), (dict(batch=0), 1), (dict(total=-1), 1),
    (dict(hk=0), 1), (dict(hq=-1), 1), (dict(d=96), 2), (dict(page=0), 1), (dict(pages=0), 1), (dict(nidx=-1), 1),
    (dict(qs=8), 1), (dict(ks=255), 1), (dict(vs=1), 1), (dict(layout=-1), 1), (dict(dtype=3), 2), (dict(kd=FAKE + 8), 2),
    (dict(ws=None), 3), (dict(wsb=255), 3), (dict(ws=FAKE + 16), 2), (dict(rot=256), 1)])
def test_append_refuses(kw, status):
    import paged_kv_gqa_13_gb300 as pd

    assert _call("pd_paged_rope_append", APPEND, **kw) == status
    assert pd.pd_last_error_string() != ""
    assert _call("pd_paged_rope_append", APPEND, total=0, hq=0, q=None, q_out=None) == 0


def test_append_fp8_refuses_f32_and_missing_scales():
    d = {}
    for k, v in APPEND.items():
        d[k] = v
        if k == "q_out":
            d["k_scale"] = d["v_scale"] = FAKE
    assert _call("pd_paged_rope_append_fp8", d, dtype=0) == 2
    assert _call("pd_paged_rope_append_fp8", d, k_scale=None) == 1
    assert _call("pd_paged_rope_append_fp8", d, v_scale=FAKE + 2) == 2


TREE = dict(q=FAKE, kd=FAKE, vd=FAKE, indices=FAKE, indptr=FAKE, last=FAKE, new=FAKE, mask=FAKE, o=FAKE, lse=FAKE, batch=2,
            total=4, words=1, hq=8, hk=2, d=128, page=16, pages=10, nidx=4, scale=0.1, dtype=2, ws=FAKE, wsb=1 << 40,
            stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), 1), (dict(o=None), 1), (dict(lse=None), 1), (dict(kd=None), 1), (dict(new=None), 1), (dict(batch=0), 1),
    (dict(total=-1), 1), (dict(words=0), 1), (dict(mask=None), 1), (dict(hq=9), 1), (dict(hk=0), 1), (dict(d=80), 2),
    (dict(page=0), 1), (dict(pages=-1), 1), (dict(nidx=-2), 1), (dict(indices=None), 1), (dict(scale=float("nan")), 1),
    (dict(dtype=4), 2), (dict(q=FAKE + 8), 2), (dict(mask=FAKE + 1), 2), (dict(lse=FAKE + 2), 2)])
def test_tree_decode_refuses(kw, status):
    import paged_kv_gqa_13_gb300 as pd

    assert _call("pd_paged_tree_decode", TREE, **kw) == status
    assert pd.pd_last_error_string() != ""


def test_tree_decode_fp8_refuses_f32_and_missing_scales():
    d = {}
    for k, v in TREE.items():
        d[k] = v
        if k == "vd":
            d["k_scale"] = d["v_scale"] = FAKE
    assert _call("pd_paged_tree_decode_fp8", d, dtype=0) == 2
    assert _call("pd_paged_tree_decode_fp8", d, v_scale=None) == 1


COMMIT = dict(kd=FAKE, vd=FAKE, indices=FAKE, indptr=FAKE, last=FAKE, new=FAKE, path=FAKE, plen=FAKE, batch=2, total=4, most=3,
              hk=2, d=128, page=16, pages=10, nidx=4, elem=2, ws=FAKE, wsb=256, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(kd=None), 1), (dict(path=None), 1), (dict(plen=None), 1), (dict(batch=0), 1), (dict(most=-1), 1), (dict(total=-1), 1),
    (dict(d=100), 2), (dict(elem=3), 2), (dict(page=0), 1), (dict(vd=FAKE + 4), 2), (dict(path=FAKE + 2), 2), (dict(ws=None), 3)])
def test_commit_refuses(kw, status):
    import paged_kv_gqa_13_gb300 as pd

    assert _call("pd_paged_tree_commit", COMMIT, **kw) == status
    assert pd.pd_last_error_string() != ""
    assert _call("pd_paged_tree_commit", COMMIT, most=0) == 0


def test_python_wrappers_refuse_shapes_and_types_before_the_library():
    import torch

    import paged_kv_gqa_13_gb300 as pd

    x = torch.zeros(4, 2, 128)
    pos = torch.zeros(4, dtype=torch.int32)
    f = torch.zeros(64, dtype=torch.int64)
    for bad in (dict(out=torch.zeros(4, 2, 64)), dict(positions=torch.zeros(3, dtype=torch.int32)),
                dict(positions=torch.zeros(4, dtype=torch.int64)), dict(freqs=torch.zeros(64)), dict(out=x.half()),
                dict(x=torch.zeros(4, 128, 2).transpose(1, 2))):
        args = {**dict(x=x, positions=pos, freqs=f, out=torch.zeros(4, 2, 128)), **bad}
        with pytest.raises(pd.PagedecodeError):
            pd.pd_rope(args["x"], args["positions"], args["freqs"], args["out"], stream=0)
    pool = torch.zeros(3, 2, 16, 128)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    ws = torch.zeros(4096, dtype=torch.uint8)
    table = (i32(0), i32(0, 1), i32(4), i32(0, 4))
    q = torch.zeros(4, 2, 128)
    lse = torch.zeros(4, 2)
    for bad in (dict(q=q.half()), dict(mask=torch.zeros(3, 1, dtype=torch.int32)), dict(lse=lse.half()),
                dict(table=(i32(0), i32(0, 1), i32(4), i32(0)))):
        a = {**dict(q=q, mask=None, lse=lse, table=table), **bad}
        with pytest.raises(pd.PagedecodeError):
            pd.pd_paged_tree_decode(a["q"], pool, pool, *a["table"], a["mask"], torch.zeros_like(a["q"]), a["lse"], 0.1, ws,
                                    stream=0)
    with pytest.raises(pd.PagedecodeError):
        pd.pd_paged_tree_commit(pool, pool, *table, i32(0, 1), i32(2), ws, stream=0)
    assert ctypes.sizeof(ctypes.c_void_p) == 8
