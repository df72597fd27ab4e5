"""Refusals of the norm-and-rotation, cache-append and chunk-attention entry
points: decided on the host, before any CUDA call."""
import ctypes

import pytest

FAKE = 0x100000  # 16-byte aligned, never dereferenced


@pytest.fixture(scope="module")
def fs():
    import __graft_entry__

    __graft_entry__.build()
    import mxfp8_swiglu_mlp_gb300 as fs

    return fs


def _call(fs, name, **change):
    rope = fs._Rope(FAKE, 128, 0)
    if "rope" in change and isinstance(change["rope"], tuple):
        rope = fs._Rope(*change.pop("rope"))
    args = {
        "fsops_qk_norm_rope": dict(q=FAKE, ldq=512, k=FAKE, ldk=512, gq=FAKE, gk=FAKE, eps=1e-6, pos=FAKE,
                                   rope=ctypes.byref(rope), qo=FAKE, ldqo=512, ko=FAKE, ldko=512, T=3, Hq=4, Hkv=2,
                                   D=128, stream=None),
        "fsops_mxfp8_kv_append": dict(k=FAKE, ldk=256, v=FAKE, ldv=256, gk=FAKE, eps=1e-6, pos=None,
                                      rope=ctypes.byref(rope), kc=FAKE, ks=FAKE, vc=FAKE, vs=FAKE, pages=9, table=FAKE,
                                      max_pages=4, cu=FAKE, lens=FAKE, T=3, B=2, Hkv=2, D=128, P=16, status=FAKE,
                                      stream=None),
        "fsops_mxfp8_paged_chunk_attention": dict(q=FAKE, ldq=512, kc=FAKE, ks=FAKE, vc=FAKE, vs=FAKE, pages=9,
                                                  table=FAKE, max_pages=4, cu=FAKE, lens=FAKE, out=2 * FAKE, ldo=512,
                                                  T=3, B=2, Hq=4, Hkv=2, D=128, P=16, window=0, sm=0.1, ws=FAKE,
                                                  ws_bytes=1 << 40, stream=None),
    }[name]
    assert set(change) <= set(args), change
    args.update(change)
    return getattr(fs.lib, name)(*args.values())


NR, AP, CH = "fsops_qk_norm_rope", "fsops_mxfp8_kv_append", "fsops_mxfp8_paged_chunk_attention"
INVALID, SHAPE, ALIGN = 1, 2, 3


@pytest.mark.parametrize("name,change,status", [
    (NR, dict(q=None), INVALID), (NR, dict(ko=None), INVALID), (NR, dict(pos=None), INVALID),
    (NR, dict(Hq=0), INVALID), (NR, dict(eps=-1.0), INVALID), (NR, dict(eps=float("nan")), INVALID),
    (NR, dict(rope=(None, 64, 0)), INVALID), (NR, dict(rope=(FAKE, 64, 2)), INVALID),
    (NR, dict(ldqo=520), INVALID),  # in place with another row distance
    (NR, dict(D=0), SHAPE), (NR, dict(D=120), SHAPE), (NR, dict(D=272), SHAPE), (NR, dict(T=-1), SHAPE),
    (NR, dict(rope=(FAKE, 48, 0)), SHAPE), (NR, dict(rope=(FAKE, 160, 0)), SHAPE), (NR, dict(rope=(FAKE, -32, 0)), SHAPE),
    (NR, dict(ldq=508), SHAPE), (NR, dict(ldk=248), SHAPE), (NR, dict(T=1 << 30), SHAPE), (NR, dict(Hq=65536), SHAPE),
    (NR, dict(q=FAKE + 8), ALIGN), (NR, dict(gk=FAKE + 2), ALIGN), (NR, dict(pos=FAKE + 2), ALIGN),
    (NR, dict(rope=(FAKE + 2, 64, 0)), ALIGN),
    (AP, dict(k=None), INVALID), (AP, dict(vs=None), INVALID), (AP, dict(status=None), INVALID),
    (AP, dict(cu=None), INVALID), (AP, dict(eps=float("inf")), INVALID),
    (AP, dict(D=64), SHAPE), (AP, dict(P=8), SHAPE), (AP, dict(P=48), SHAPE), (AP, dict(B=0), SHAPE),
    (AP, dict(T=-1), SHAPE), (AP, dict(ldk=248), SHAPE), (AP, dict(ldv=260), SHAPE), (AP, dict(pages=0), SHAPE),
    (AP, dict(max_pages=1 << 21), SHAPE), (AP, dict(pages=1 << 27), SHAPE), (AP, dict(rope=(FAKE, 100, 0)), SHAPE),
    (AP, dict(kc=FAKE + 4), ALIGN), (AP, dict(table=FAKE + 1), ALIGN), (AP, dict(status=FAKE + 2), ALIGN),
    (CH, dict(q=None), INVALID), (CH, dict(ws=None), INVALID), (CH, dict(window=-1), INVALID),
    (CH, dict(sm=float("nan")), INVALID), (CH, dict(sm=1e31), INVALID), (CH, dict(out=FAKE), INVALID),
    (CH, dict(D=64), SHAPE), (CH, dict(Hq=3), SHAPE), (CH, dict(Hq=130), SHAPE), (CH, dict(Hkv=0), SHAPE),
    (CH, dict(P=17), SHAPE), (CH, dict(B=65536), SHAPE), (CH, dict(T=1 << 29), SHAPE), (CH, dict(ldq=504), SHAPE),
    (CH, dict(ldo=516), SHAPE), (CH, dict(max_pages=0), SHAPE),
    (CH, dict(ws=FAKE + 128), ALIGN), (CH, dict(lens=FAKE + 2), ALIGN), (CH, dict(out=FAKE + 2), ALIGN),
])
def test_refusals(fs, name, change, status):
    assert _call(fs, name, **change) == status


def test_nothing_to_do_is_ok(fs):
    for name in (NR, AP, CH):
        assert _call(fs, name, T=0) == fs.OK


def test_a_host_tensor_is_refused(fs):
    import torch

    x = torch.zeros(3, 256, dtype=torch.bfloat16)
    with pytest.raises(fs.FsopsError) as e:
        fs.fsops_qk_norm_rope(x, 256, None, 0, None, None, 0.0, None, None, x, 256, None, 0, 3, 2, 0, 128, stream=0)
    assert e.value.status == fs.ERR_INVALID_ARG


def test_workspace_of_an_unsupported_shape_is_zero(fs):
    assert fs.fsops_paged_chunk_attention_workspace_bytes(4, 1, 8, 2, 64, 16, 4) == 0
    assert fs.fsops_paged_chunk_attention_workspace_bytes(4, 1, 8, 3, 128, 16, 4) == 0
