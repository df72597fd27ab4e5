"""A tensor of another GPU than the current one is refused by the binding of the
attention-side operators (stand-ins for tensors: one GPU is enough, or none)."""
import pytest

FAKE = 0x100000


@pytest.fixture(scope="module")
def fs():
    import __graft_entry__

    __graft_entry__.build()
    import mxfp8_swiglu_mlp_gb300 as fs

    return fs


class OnDevice:
    """What the binding asks of a tensor."""

    def __init__(self, index):
        self.index, self.is_cuda = index, index >= 0

    def get_device(self):
        return self.index

    def data_ptr(self):
        return FAKE


def _calls(fs, x, **other):
    """The three operators with T = 0 (nothing is launched), one argument replaced."""
    def arg(name):
        return other.get(name, x)

    return {
        "fsops_qk_norm_rope": (["q", "k", "gq", "gk", "pos", "rope", "qo", "ko"], lambda: fs.fsops_qk_norm_rope(
            arg("q"), 512, arg("k"), 256, arg("gq"), arg("gk"), 1e-6, arg("pos"), (arg("rope"), 128, False), arg("qo"), 512,
            arg("ko"), 256, 0, 4, 2, 128, stream=0)),
        "fsops_mxfp8_kv_append": (["k", "v", "gk", "pos", "rope", "kc", "ks", "vc", "vs", "table", "cu", "lens", "status"],
                                  lambda: fs.fsops_mxfp8_kv_append(
            arg("k"), 256, arg("v"), 256, arg("gk"), 1e-6, arg("pos"), (arg("rope"), 128, False), arg("kc"), arg("ks"),
            arg("vc"), arg("vs"), 9, arg("table"), 4, arg("cu"), arg("lens"), 0, 2, 2, 128, 16, arg("status"), stream=0)),
        "fsops_mxfp8_paged_chunk_attention": (["q", "kc", "ks", "vc", "vs", "table", "cu", "lens", "out", "ws"],
                                              lambda: fs.fsops_mxfp8_paged_chunk_attention(
            arg("q"), 512, arg("kc"), arg("ks"), arg("vc"), arg("vs"), 9, arg("table"), 4, arg("cu"), arg("lens"), arg("out"),
            512, 0, 2, 4, 2, 128, 16, 0, 0.1, arg("ws"), 1 << 40, stream=0)),
    }


NAMES = ["fsops_qk_norm_rope", "fsops_mxfp8_kv_append", "fsops_mxfp8_paged_chunk_attention"]


@pytest.mark.parametrize("name", NAMES)
def test_a_tensor_of_another_device_is_refused(fs, name, monkeypatch):
    monkeypatch.setattr(fs, "_current_device", lambda: 0, raising=False)
    here, there = OnDevice(0), OnDevice(1)
    out = OnDevice(0)
    out.data_ptr = lambda: 2 * FAKE  # (the attention's output is not its input)
    names, call = _calls(fs, here, out=out)[name]
    call()  # all on the current device: nothing to do, and no error
    for a in names:
        with pytest.raises(fs.FsopsError) as e:
            _calls(fs, here, **{"out": out, a: there})[name][1]()
        assert e.value.status == fs.ERR_INVALID_ARG, a
        with pytest.raises(fs.FsopsError) as e:
            _calls(fs, here, **{"out": out, a: OnDevice(-1)})[name][1]()
        assert e.value.status == fs.ERR_INVALID_ARG, a


@pytest.mark.parametrize("name", NAMES)
def test_addresses_pass_as_they_are(fs, name):
    _calls(fs, FAKE, out=2 * FAKE)[name][1]()
