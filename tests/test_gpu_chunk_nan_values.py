"""Values that are not finite, in places that some row sees: a NaN code or a NaN
scale byte of V makes the rows that see its token NaN (in its dimensions, and in
no other where all rows of the call see it), and leaves the rows that do not see
it as they are.  Both kernels, single tiles and parts.  Tolerances of finite
outputs are those of tests/test_gpu_chunk_attention.py (derived there)."""
import numpy as np
import pytest

from tests._util import bf16_bits_to_f64
from tests.test_gpu_chunk_attention import Run, _finite_cache
from tests.test_gpu_norm_rope import Batch, _dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fs():
    import mxfp8_swiglu_mlp_gb300 as fs

    return fs


def _check(fs, new, ctx, Hkv, G, marks, window=0, sm=None, grow=0, seed=0):
    """One sequence; marks: (token, what), what a byte for the code of dimension
    37 or ("scale", byte) for the block of dimensions 64 .. 95, in the last KV
    head."""
    import torch

    bt = Batch([new], [ctx], Hkv, 16, 200 + seed)
    _finite_cache(bt)
    L = new + ctx
    if grow:  # key scales that double every `grow` tokens: the weight of the first tokens underflows
        t = np.arange(L)
        page, slot = bt.table[0, t // 16], t % 16
        bt.scales[0][page, :, slot] = np.clip(bt.scales[0][page, :, slot].astype(int) + (t // grow)[:, None, None], 1, 200)
    r = Run(fs, bt, G, window, sm)
    ref = r.want()  # of the finite values: where NaN reaches, it is not looked at
    codes, scales = bt.codes[1].copy(), bt.scales[1].copy()
    pos = np.arange(ctx, L)
    sure = np.zeros((new, r.Hq, 128), bool)   # has to be NaN
    may = np.zeros((new, r.Hq, 128), bool)    # may be
    heads = np.arange((Hkv - 1) * G, Hkv * G)
    for tok, what in marks:
        page, slot = bt.table[0, tok // 16], tok % 16
        seen = (tok <= pos) & ((tok > pos - window) if window else True)
        assert seen.any()
        if isinstance(what, tuple):
            scales[page, Hkv - 1, slot, 2] = what[1]
            dims = np.arange(64, 96)
        else:
            codes[page, Hkv - 1, slot, 37] = what
            dims = np.array([37])
        sure[np.ix_(seen, heads, dims)] = True
        may[np.ix_(seen, heads, dims if seen.all() else np.arange(128))] = True
    r.cache[2].copy_(_dev(codes))
    r.cache[3].copy_(_dev(scales))
    r.call()
    torch.cuda.synchronize()
    assert r.status() == 0
    got = bf16_bits_to_f64(r.got()[:new, :r.Hq * 128]).reshape(new, r.Hq, 128)
    out, A, mag = ref["out"][:new], ref["absv"][:new], ref["mag"][:new, :, None]
    tol = 2.0 ** -8 * np.abs(out) + (2.0 ** -8 + 2 * (2.0 ** -17 * mag + 2.0 ** -18)) * (A + np.abs(out))
    assert np.isnan(got[sure]).all()
    assert np.all(np.abs(got - out)[~may] <= tol[~may])


# rows in one tile of the kernel for few rows; of the other with one stream a half and two streams sharing the
# rows; each whole and in parts
SHAPES = [(6, 130, 2, 4), (1, 0, 1, 8), (2, 9000, 1, 4), (120, 130, 2, 4), (300, 40, 1, 1), (70, 9000, 1, 4), (33, 300, 2, 2)]


@pytest.mark.parametrize("what", [0x7F, 0xFF, ("scale", 0xFF)], ids=str)
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_nan_that_all_rows_see(fs, i, what):
    new, ctx, Hkv, G = SHAPES[i]
    _check(fs, new, ctx, Hkv, G, [(0, what)], seed=i)
    _check(fs, new, ctx, Hkv, G, [(ctx // 2, what), (ctx, what)], seed=i)


@pytest.mark.parametrize("what", [0x7F, 0xFF, ("scale", 0xFF)], ids=str)
@pytest.mark.parametrize("i", [i for i in range(len(SHAPES)) if SHAPES[i][0] > 1])
def test_nan_that_later_rows_see(fs, i, what):
    """At a new token: the rows before it do not see it."""
    new, ctx, Hkv, G = SHAPES[i]
    for back in sorted({1, new // 2, new - 1}):
        _check(fs, new, ctx, Hkv, G, [(ctx + new - back, what)], seed=i)


@pytest.mark.parametrize("window", [1, 3, 40, 200])
@pytest.mark.parametrize("i", [0, 2, 3, 4, 5])
def test_nan_that_a_window_leaves(fs, i, window):
    """Seen by the first rows only, by rows in the middle, by the last."""
    new, ctx, Hkv, G = SHAPES[i]
    for tok in {max(0, ctx - window + 1), ctx + new // 2, ctx + new - 1, max(0, ctx + new // 3 - window)}:
        if tok > ctx - window:
            _check(fs, new, ctx, Hkv, G, [(tok, 0x7F)], window=window, seed=i)


@pytest.mark.parametrize("new,ctx,G,grow", [(3, 2600, 4, 300), (90, 2500, 1, 300), (300, 2500, 1, 300), (2, 9000, 4, 900)])
def test_nan_of_no_weight_shows(fs, new, ctx, G, grow):
    """A row that sees NaN is NaN however small the token's probability."""
    _check(fs, new, ctx, 1, G, [(5, 0x7F)], grow=grow, sm=1.0)


@pytest.mark.parametrize("new,ctx,G", [(6, 100, 4), (120, 100, 4)])
def test_nan_among_appended_values(fs, new, ctx, G):
    """A NaN in the layer's v is a NaN code in the cache and NaN in the rows that
    see it."""
    import torch

    bt = Batch([new], [ctx], 1, 16, 240)
    _finite_cache(bt)
    r = Run(fs, bt, G)
    v = bt.v.copy()
    v[new // 2, 0, 11] = 0x7FC0
    k, d = _dev(bt.k.view(np.int16)), _dev(v.view(np.int16))
    fs.fsops_mxfp8_kv_append(k, 128, d, 128, None, 0.0, None, None, *r.cache, bt.pages, r.meta[0], bt.max_pages, r.meta[1],
                             r.meta[2], bt.T, 1, 1, 128, 16, r.ws)
    r.call()
    torch.cuda.synchronize()
    assert r.status() == 0
    got = bf16_bits_to_f64(r.got()[:new, :G * 128]).reshape(new, G, 128)
    assert np.isnan(got[new // 2:, :, 11]).all() and np.isfinite(got[:new // 2]).all()


@pytest.mark.parametrize("new,ctx,Hkv,G", [(6, 130, 2, 4), (120, 130, 2, 4), (2, 9000, 1, 4), (70, 9000, 1, 4)])
def test_nan_scale_of_a_key(fs, new, ctx, Hkv, G):
    """Of the keys, too, a NaN scale byte is seen by the rows that see its token."""
    import torch

    bt = Batch([new], [ctx], Hkv, 16, 250)
    _finite_cache(bt)
    r = Run(fs, bt, G)
    ref = r.want()
    tok = ctx + new // 2
    scales = bt.scales[0].copy()
    scales[bt.table[0, tok // 16], Hkv - 1, tok % 16, 1] = 0xFF
    r.cache[1].copy_(_dev(scales))
    r.call()
    torch.cuda.synchronize()
    assert r.status() == 0
    bad = np.zeros((new, r.Hq), bool)
    bad[new // 2:, (Hkv - 1) * G:] = True
    got = bf16_bits_to_f64(r.got()[:new, :r.Hq * 128]).reshape(new, r.Hq, 128)
    out, A, mag = ref["out"][:new], ref["absv"][:new], ref["mag"][:new, :, None]
    tol = 2.0 ** -8 * np.abs(out) + (2.0 ** -8 + 2 * (2.0 ** -17 * mag + 2.0 ** -18)) * (A + np.abs(out))
    assert np.isnan(got[bad]).all()
    assert np.all(np.abs(got - out)[~bad] <= tol[~bad])


@pytest.mark.parametrize("new,ctx,G", [(1, 130, 4), (6, 130, 4), (40, 130, 1), (300, 40, 1)])
def test_neighbours_of_a_nan_code_stay(fs, new, ctx, G):
    """The largest codes beside NaN codes, in every place of a word of four."""
    import torch

    bt = Batch([new], [ctx], 1, 16, 260)
    _finite_cache(bt)
    codes, page, slot = bt.codes[1], bt.table[0, 0], 3
    for d in range(0, 128, 2):
        codes[page, 0, slot, d + (d >> 2 & 1)] = 0x7E if d & 8 else 0xFE
    r = Run(fs, bt, G)
    ref = r.want()
    bad = np.zeros(128, bool)
    codes = codes.copy()
    for d in range(0, 128, 2):
        at = d + 1 - (d >> 2 & 1)
        codes[page, 0, slot, at] = 0xFF if d & 16 else 0x7F
        bad[at] = True
    r.cache[2].copy_(_dev(codes))
    r.call()
    torch.cuda.synchronize()
    assert r.status() == 0
    got = bf16_bits_to_f64(r.got()[:new, :G * 128]).reshape(new, G, 128)
    out, A, mag = ref["out"][:new], ref["absv"][:new], ref["mag"][:new, :, None]
    tol = 2.0 ** -8 * np.abs(out) + (2.0 ** -8 + 2 * (2.0 ** -17 * mag + 2.0 ** -18)) * (A + np.abs(out))
    assert np.isnan(got[:, :, bad]).all()  # (all rows see the token)
    assert np.all((np.abs(got - out) <= tol)[:, :, ~bad])
