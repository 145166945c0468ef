"""Norms with the rotation and block-scaled pools without a GPU: refusals and empty calls."""
import pytest

from tests.test_spec_abi import APPEND, FAKE, TREE, _call

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3

NORM = dict(q=FAKE, k=FAKE, qw=FAKE, kw=FAKE, positions=FAKE, freqs=FAKE, q_out=FAKE, k_out=FAKE, tokens=4, hq=8, hk=2, d=128,
            rot=128, qs=1024, ks=256, qos=1024, kos=256, eps=1e-6, layout=0, scale=1.0, dtype=2, stream=None)


def _with(defaults, **after):
    """`defaults` with further arguments after the one that each names: {name: [(new name, value), ...]}."""
    d = {}
    for k, v in defaults.items():
        d[k] = v
        d.update(after.get(k, []))
    return d


NORM_APPEND = _with(APPEND, v=[("qw", FAKE), ("kw", FAKE)], vs=[("eps", 1e-6)])
SCALES = [("k_scale", FAKE), ("v_scale", FAKE)]
NORM_APPEND_FP8 = _with(NORM_APPEND, q_out=SCALES)
BLOCK_APPEND = _with(NORM_APPEND_FP8, nidx=[("block", 16)])
READ = dict(kd=FAKE, vd=FAKE, k_scale=FAKE, v_scale=FAKE, indices=FAKE, indptr=FAKE, last=FAKE, out=FAKE, first=FAKE, ko=FAKE,
            vo=FAKE, batch=2, total=4, hk=2, d=128, page=16, pages=10, nidx=4, block=16, dtype=2, ws=FAKE, wsb=256, stream=None)
BLOCK_TREE = _with(TREE, vd=SCALES, nidx=[("block", 16)])
BLOCK_DECODE = {k: v for k, v in BLOCK_TREE.items() if k not in ("new", "mask", "total", "words")}


def _refused(name, defaults, kw, status):
    import paged_kv_gqa_13_gb300 as pd

    assert _call(name, defaults, **kw) == status
    assert pd.pd_last_error_string() != ""


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), 1), (dict(q_out=None), 1), (dict(k=None), 1), (dict(k_out=None), 1), (dict(positions=None), 1),
    (dict(freqs=None), 1), (dict(tokens=-1), 1), (dict(hq=0), 1), (dict(hk=-1), 1), (dict(hq=(1 << 20) + 1), 1),
    (dict(hk=(1 << 20) + 1), 1), (dict(d=0), 2), (dict(d=127), 2), (dict(d=258), 2), (dict(rot=130), 1), (dict(rot=3), 1),
    (dict(rot=-2), 1), (dict(qs=1023), 1), (dict(ks=255), 1), (dict(qos=1023), 1), (dict(kos=128), 1), (dict(qs=2048), 1),
    (dict(kos=512), 1), (dict(layout=2), 1), (dict(scale=float("nan")), 1), (dict(eps=0.0), 1), (dict(eps=-1.0), 1),
    (dict(eps=float("inf")), 1), (dict(eps=float("nan")), 1), (dict(dtype=3), 2), (dict(q=FAKE + 1), 2), (dict(k_out=FAKE + 1), 2),
    (dict(qw=FAKE + 1), 2), (dict(kw=FAKE + 1), 2), (dict(positions=FAKE + 2), 2), (dict(freqs=FAKE + 4), 2),
    (dict(dtype=0, qw=FAKE + 2), 2)])
def test_norm_rope_refuses(kw, status):
    _refused("pd_norm_rope", NORM, kw, status)


def test_norm_rope_of_no_token():
    assert _call("pd_norm_rope", NORM, tokens=0, q=None, k=None, q_out=None, k_out=None, positions=None) == 0
    assert _call("pd_norm_rope", NORM, tokens=0, hk=0, k=None, k_out=None, ks=0, kos=0) == 0
    assert _call("pd_norm_rope", NORM, tokens=0, d=96) == INVALID  # rot 128 of 96
    assert _call("pd_norm_rope", NORM, tokens=0, d=6, rot=0, positions=None, freqs=None) == 0


COMMON = [
    (dict(k=None), 1), (dict(v=None), 1), (dict(q=None), 1), (dict(q_out=None), 1), (dict(freqs=None), 1), (dict(kd=None), 1),
    (dict(vd=None), 1), (dict(new=None), 1), (dict(indptr=None), 1), (dict(last=None), 1), (dict(indices=None), 1),
    (dict(batch=0), 1), (dict(batch=(1 << 28) + 1), 1), (dict(total=-1), 1), (dict(hk=0), 1), (dict(hq=-1), 1),
    (dict(hk=(1 << 20) + 1), 1), (dict(d=96), 2), (dict(page=0), 1), (dict(pages=0), 1), (dict(nidx=-1), 1), (dict(qs=8), 1),
    (dict(qs=1280), 1), (dict(ks=255), 1), (dict(vs=1), 1), (dict(layout=-1), 1), (dict(dtype=3), 2), (dict(kd=FAKE + 8), 2),
    (dict(vd=FAKE + 4), 2), (dict(qw=FAKE + 1), 2), (dict(eps=-1e-6), 1), (dict(eps=float("nan")), 1),
    (dict(eps=float("inf")), 1), (dict(positions=FAKE + 1), 2), (dict(last=FAKE + 2), 2), (dict(scale=float("inf")), 1),
    (dict(ws=None), 3), (dict(wsb=255), 3), (dict(ws=FAKE + 16), 2), (dict(rot=256), 1)]


@pytest.mark.parametrize("name,defaults", [("pd_paged_norm_rope_append", NORM_APPEND),
                                           ("pd_paged_norm_rope_append_fp8", NORM_APPEND_FP8),
                                           ("pd_paged_rope_append_fp8_blocks", BLOCK_APPEND)])
@pytest.mark.parametrize("kw,status", COMMON)
def test_appends_refuse(name, defaults, kw, status):
    _refused(name, defaults, kw, status)
    assert _call(name, defaults, total=0, hq=0, q=None, q_out=None, k=None, v=None, positions=None) == 0


CODES = [(dict(k_scale=None), 1), (dict(v_scale=None), 1), (dict(k_scale=FAKE + 2), 2), (dict(v_scale=FAKE + 1), 2)]
BLOCKS = [(dict(block=0), 1), (dict(block=-1), 1), (dict(block=5), 1), (dict(block=32), 1), (dict(page=128, block=128), 1),
          (dict(page=65, block=65), 1), (dict(page=48, block=32), 1)]


@pytest.mark.parametrize("kw,status", CODES + [(dict(dtype=0), 2)])
def test_norm_append_fp8_refuses(kw, status):
    _refused("pd_paged_norm_rope_append_fp8", NORM_APPEND_FP8, kw, status)


def test_the_norms_are_left_out_in_blocks_only():
    assert _call("pd_paged_norm_rope_append", NORM_APPEND, eps=0.0, total=0) == INVALID
    assert _call("pd_paged_norm_rope_append_fp8", NORM_APPEND_FP8, eps=0.0, total=0) == INVALID
    assert _call("pd_paged_rope_append_fp8_blocks", BLOCK_APPEND, eps=0.0, total=0, qw=None, kw=None) == 0
    for w in (dict(qw=None), dict(kw=None), {}):
        assert _call("pd_paged_rope_append_fp8_blocks", BLOCK_APPEND, eps=0.0, total=0, **w) == INVALID


@pytest.mark.parametrize("kw,status", CODES + BLOCKS + [(dict(dtype=0), 2)])
def test_block_append_refuses(kw, status):
    _refused("pd_paged_rope_append_fp8_blocks", BLOCK_APPEND, kw, status)


@pytest.mark.parametrize("kw,status", CODES + BLOCKS + [
    (dict(kd=None), 1), (dict(vd=None), 1), (dict(indices=None), 1), (dict(indptr=None), 1), (dict(last=None), 1),
    (dict(out=None), 1), (dict(ko=None), 1), (dict(vo=None), 1), (dict(batch=0), 1), (dict(batch=(1 << 28) + 1), 1),
    (dict(total=-1), 1), (dict(hk=0), 1), (dict(hk=(1 << 20) + 1), 1), (dict(d=80), 2), (dict(page=0), 1), (dict(pages=0), 1),
    (dict(nidx=-1), 1), (dict(dtype=7), 2), (dict(kd=FAKE + 8), 2), (dict(ko=FAKE + 8), 2), (dict(vo=FAKE + 2), 2),
    (dict(out=FAKE + 2), 2), (dict(first=FAKE + 2), 2), (dict(ws=None), 3), (dict(wsb=128), 3), (dict(ws=FAKE + 8), 2)])
def test_read_refuses(kw, status):
    _refused("pd_paged_read_fp8_blocks", READ, kw, status)


def test_read_of_no_token():
    assert _call("pd_paged_read_fp8_blocks", READ, total=0, ko=None, vo=None, first=None, dtype=0) == 0
    assert _call("pd_paged_read_fp8_blocks", READ, total=0, nidx=0, indices=None) == 0


ATTENTION = [
    (dict(q=None), 1), (dict(o=None), 1), (dict(lse=None), 1), (dict(kd=None), 1), (dict(vd=None), 1), (dict(last=None), 1),
    (dict(indptr=None), 1), (dict(indices=None), 1), (dict(batch=0), 1), (dict(hq=9), 1), (dict(hk=0), 1), (dict(hq=0), 1),
    (dict(d=80), 2), (dict(page=0), 1), (dict(pages=-1), 1), (dict(nidx=-2), 1), (dict(scale=float("nan")), 1),
    (dict(scale=float("inf")), 1), (dict(dtype=4), 2), (dict(dtype=0), 2), (dict(q=FAKE + 8), 2), (dict(o=FAKE + 4), 2),
    (dict(lse=FAKE + 2), 2), (dict(kd=FAKE + 8), 2), (dict(indptr=FAKE + 1), 2)]


@pytest.mark.parametrize("kw,status", CODES + BLOCKS + ATTENTION + [
    (dict(new=None), 1), (dict(total=-1), 1), (dict(words=0), 1), (dict(mask=None), 1), (dict(mask=FAKE + 1), 2)])
def test_block_tree_refuses(kw, status):
    _refused("pd_paged_tree_decode_fp8_blocks", BLOCK_TREE, kw, status)


# groups of 4 at head_dim 128 and of 2 take different kernels
@pytest.mark.parametrize("hk", [2, 4])
@pytest.mark.parametrize("kw,status", CODES + BLOCKS + ATTENTION)
def test_block_decode_refuses(hk, kw, status):
    _refused("pd_paged_decode_fp8_blocks", BLOCK_DECODE, {"hk": hk, **kw}, status)


def test_workspace_bytes():
    import paged_kv_gqa_13_gb300 as pd

    lib = pd._lib
    for kw in ((0, 8, 2, 128, 2), (4, 8, 3, 128, 2), (4, 8, 2, 96, 2), (4, 8, 2, 128, 0), (4, 8, 2, 128, 9), (4, 0, 2, 128, 2),
               (4, 8, 0, 128, 2), (-1, 8, 2, 64, 1)):
        assert lib.pd_paged_decode_fp8_blocks_workspace_bytes(*kw) == 0, kw
        with pytest.raises(pd.PagedecodeError):
            pd.pd_paged_decode_fp8_blocks_workspace_bytes(*kw)
    for kw in ((8, 3, 128, 2), (8, 2, 96, 2), (8, 2, 128, 0), (0, 2, 128, 2), (8, -2, 128, 2)):
        assert lib.pd_paged_tree_decode_fp8_blocks_workspace_bytes(*kw) == 0, kw
        with pytest.raises(pd.PagedecodeError):
            pd.pd_paged_tree_decode_fp8_blocks_workspace_bytes(*kw)


def test_wrappers_refuse_shapes_and_types():
    import torch

    import paged_kv_gqa_13_gb300 as pd

    i32 = lambda *v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    codes, s = torch.zeros(3, 2, 16, 128, dtype=torch.uint8), torch.ones(3, 2, 4)
    ws, f = torch.zeros(4096, dtype=torch.uint8), torch.zeros(64, dtype=torch.int64)
    table = (i32(0), i32(0, 1), i32(4))
    q, lse = torch.zeros(1, 8, 128).half(), torch.zeros(1, 8)

    def decode(ks=s, vs=s, k=codes, v=codes, o=q, l=lse):  # noqa: E741
        pd.pd_paged_decode_fp8_blocks(q, k, v, ks, vs, *table, o, l, 0.1, ws, stream=0)

    for kw in (dict(ks=torch.ones(3, 2, 8)), dict(ks=torch.ones(3, 2, 3), vs=torch.ones(3, 2, 3)), dict(ks=s.half(), vs=s.half()),
               dict(ks=torch.ones(2), vs=torch.ones(2)), dict(ks=torch.ones(4, 2, 4), vs=torch.ones(4, 2, 4)),
               dict(k=codes.half(), v=codes.half()), dict(v=codes[:, :, :8]), dict(o=q.float()), dict(l=lse[:, :4]),
               dict(l=lse.int()), dict(o=torch.zeros(2, 8, 128).half())):
        with pytest.raises(pd.PagedecodeError) as e:
            decode(**kw)
        assert e.value.status == INVALID, kw
    x = torch.zeros(4, 2, 128).half()

    def append(k=x, v=x, qq=None, out=None, w=None, pools=codes, new=i32(0, 4), pos=None):
        pd.pd_paged_rope_append_fp8_blocks(qq, k, v, pos, f, out, s, s, pools, pools, *table, new, ws, w, w, eps=1e-6, stream=0)

    for kw in (dict(v=x.float()), dict(v=x[:2]), dict(k=torch.zeros(4, 3, 128).half(), v=torch.zeros(4, 3, 128).half()),
               dict(w=torch.ones(64).half()), dict(w=torch.ones(128)), dict(qq=x[:3], out=x[:3]), dict(qq=x, out=x.float()),
               dict(pools=codes.half()), dict(new=i32(0, 2, 4)), dict(pos=i32(0, 1))):
        with pytest.raises(pd.PagedecodeError) as e:
            append(**kw)
        assert e.value.status == INVALID, kw
    for kw in (dict(k=x.float()), dict(q_out=x[:2]), dict(q_weight=torch.ones(128)), dict(positions=i32(0))):
        args = dict(q=x, k=x, q_weight=None, k_weight=None, positions=i32(0, 1, 2, 3), freqs=f, q_out=x, k_out=x)
        with pytest.raises(pd.PagedecodeError) as e:
            pd.pd_norm_rope(**{**args, **kw}, stream=0)
        assert e.value.status == INVALID, kw
    out = torch.zeros(4, 2, 128)
    for kw in (dict(k_out=out[:, :1]), dict(v_out=out.half()), dict(first=i32(0, 0)), dict(out_indptr=i32(0, 1, 4))):
        args = dict(out_indptr=i32(0, 4), first=None, k_out=out, v_out=out)
        with pytest.raises(pd.PagedecodeError) as e:
            pd.pd_paged_read_fp8_blocks(codes, codes, s, s, *table, **{**args, **kw}, workspace=ws, stream=0)
        assert e.value.status == INVALID, kw
