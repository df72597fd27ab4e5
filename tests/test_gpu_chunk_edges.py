"""Corners of the chunk attention and the append: query tiles at the sizes where
the kernel for few rows and the one for many meet, scores that keep growing
along the keys, results of many parts, scales at the top of their range, NaN in
hidden places, batches larger than the grid.  Tolerances are those of
tests/test_gpu_chunk_attention.py and tests/test_gpu_norm_rope.py (derived
there)."""
import numpy as np
import pytest

import oracle
from tests._util import bf16_bits_to_f64
from tests.test_gpu_chunk_attention import Run, _check, _compare, _finite_cache
from tests.test_gpu_norm_rope import FP32, Batch, _append, _freq, _pair_length

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fs():
    import mxfp8_swiglu_mlp_gb300 as fs

    return fs


# rows of a sequence around 16, 32 and 64, and ragged ones: (new, ctx, Hkv, G)
ROWS = [([15, 16], [120, 97], 1, 1), ([17, 31], [222, 113], 2, 1), ([32, 32], [80, 300], 1, 1), ([33, 33], [79, 111], 1, 1),
        ([4, 4], [220, 5], 2, 8), ([1, 2], [700, 112], 1, 31), ([1, 1], [111, 224], 1, 33), ([64, 1], [50, 400], 1, 1),
        ([40, 1, 1, 1], [200, 112, 113, 447], 2, 2), ([1, 100, 0, 1, 1, 1, 1, 1], [9, 30, 3, 500, 1, 2, 223, 224], 1, 2),
        ([65, 63], [60, 200], 1, 1), ([3, 3], [108, 109], 1, 5)]


@pytest.mark.parametrize("i", range(len(ROWS)))
def test_rows_around_the_tiles(fs, i):
    new, ctx, Hkv, G = ROWS[i]
    _check(fs, new, ctx, Hkv, 16, G, pad=i % 3, seed=60 + i, qgap=8 * (i % 4))


@pytest.mark.parametrize("window", [1, 30, 112, 113, 224, 500])
def test_windows_of_few_rows(fs, window):
    _check(fs, [1, 5, 8, 2], [500, 222, 0, 1000], 2, 16, 4, window=window, seed=window)


@pytest.mark.parametrize("new,ctx,Hkv,G", [([2, 3], [2600, 1500], 1, 4), ([150], [2500], 1, 4), ([40], [3000], 1, 2)])
def test_scores_that_grow_along_the_keys(fs, new, ctx, Hkv, G):
    """Key scales that double every 400 tokens: the running maximum passes its
    limit again and again, and what was added up is rescaled."""
    import torch

    bt = Batch(new, ctx, Hkv, 16, 70)
    _finite_cache(bt)
    for b in range(bt.B):
        t = np.arange(bt.lens[b])
        page, slot = bt.table[b, t // 16], t % 16
        s = bt.scales[0][page, :, slot].astype(int)
        bt.scales[0][page, :, slot] = np.clip(s - 1 + (t // 400)[:, None, None], 1, 200)
    r = Run(fs, bt, G)
    r.call()
    torch.cuda.synchronize()
    assert r.status() == 0
    _compare(r)


@pytest.mark.parametrize("new,ctx,Hkv,P,G", [([1], [12000], 1, 16, 4), ([64], [8000], 1, 64, 4), ([1] * 3, [300, 10, 0], 4, 16, 8),
                                             ([1] * 40, [1000 + 7 * i for i in range(40)], 1, 16, 2),
                                             ([300], [1200], 8, 32, 4)])
def test_parts_and_whole_tiles(fs, new, ctx, Hkv, P, G):
    """One query tile over more than 32 blocks; a tile a block; several a block."""
    _check(fs, new, ctx, Hkv, P, G, seed=80)


@pytest.mark.parametrize("new,ctx,G", [([2], [300], 4), ([90], [200], 4)])
def test_value_scales_at_the_top(fs, new, ctx, G):
    """Values of 2^20 to 2^80 beside ordinary ones, in blocks of their own."""
    import torch

    bt = Batch(new, ctx, 1, 16, 90)
    _finite_cache(bt)
    s = bt.scales[1]
    s[..., 1] = np.where(s[..., 1] == 0xFF, 0xFF, 134 + bt.rng.integers(0, 3, s[..., 1].shape))
    s[..., 2] = np.where(s[..., 2] == 0xFF, 0xFF, 200)
    r = Run(fs, bt, G)
    r.call()
    torch.cuda.synchronize()
    assert r.status() == 0
    n, ref = int(bt.cu[-1]), r.want()
    got = bf16_bits_to_f64(r.got()[:n, :r.Hq * 128]).reshape(n, r.Hq, 128)
    out, A, mag = ref["out"][:n], ref["absv"][:n], ref["mag"][:n, :, None]
    tol = 2.0 ** -8 * np.abs(out) + (2.0 ** -8 + 2 * (2.0 ** -17 * mag + 2.0 ** -18)) * (A + np.abs(out))
    assert np.all(np.abs(got - out) <= tol)


@pytest.mark.parametrize("new,G", [([6], 4), ([120], 4)])
def test_nan_key_in_a_hidden_place(fs, new, G):
    """The last token's key is NaN: only its own rows may see it."""
    import torch

    bt = Batch(new, [130], 2, 16, 91)
    _finite_cache(bt)
    last = int(bt.lens[0]) - 1
    r = Run(fs, bt, G)
    ref = r.want()
    keys = bt.codes[0].copy()
    keys[bt.table[0, last // 16], :, last % 16] = 0x7F
    r.cache[0].copy_(torch.from_numpy(keys).cuda())
    r.call()
    torch.cuda.synchronize()
    assert r.status() == 0
    n = new[0] - 1
    got = bf16_bits_to_f64(r.got()[:n, :r.Hq * 128]).reshape(n, r.Hq, 128)
    out, A, mag = ref["out"][:n], ref["absv"][:n], ref["mag"][:n, :, None]
    tol = 2.0 ** -8 * np.abs(out) + (2.0 ** -8 + 2 * (2.0 ** -17 * mag + 2.0 ** -18)) * (A + np.abs(out))
    assert np.all(np.abs(got - out) <= tol)


def test_many_single_tokens(fs):
    """More sequences than blocks and than a warp's lanes, some without a token."""
    rng = np.random.default_rng(5)
    new = [int(x) for x in rng.choice([0, 1, 1, 1, 1, 2], 700)]
    _check(fs, new, [int(x) for x in rng.integers(0, 300, 700)], 1, 16, 4, pad=3, seed=92)


@pytest.mark.parametrize("norm,R,inter", [(True, 128, False), (False, 32, False), (True, 96, True)])
def test_append_of_many_tokens(fs, norm, R, inter):
    """More tokens than warps of the grid."""
    bt = Batch([2500, 0, 3100, 17], [3, 9, 0, 100], 1, 64, 93, pad=70)
    (kc, ks, vc, vs), status = _append(fs, bt, norm, R, inter)
    assert status == 0
    b, place, page, slot = bt.where()
    n = len(b)
    c, s = oracle.quantize_bf16(bt.v[:n].reshape(-1, 128))
    assert np.array_equal(vc[page, :, slot].reshape(n, 128), c) and np.array_equal(vs[page, :, slot].reshape(n, 4), s)
    g = bf16_bits_to_f64(bt.gamma) if norm else None
    x = bf16_bits_to_f64(bt.k[:n])
    want = oracle.norm_rope(x, g, 1e-6, place, _freq(R), R, inter)
    err = 2 * FP32 * _pair_length(oracle.norm_rope(x, g, 1e-6, place, _freq(R), 0, inter), R, inter)
    gk, gs = kc[page, :, slot], ks[page, :, slot]
    unit = np.repeat(np.ldexp(1.0, gs.astype(np.int64) - 127), 32, axis=-1)
    got = oracle.dequantize(gk.reshape(-1, 128), gs.reshape(-1, 4)).reshape(want.shape)
    clipped = np.clip(want, -448 * unit, 448 * unit)
    assert np.all(np.abs(got - clipped) <= np.maximum(2.0 ** -4 * np.abs(clipped), 2.0 ** -10 * unit) + err)
    for got, was in ((kc, bt.codes[0]), (ks, bt.scales[0]), (vc, bt.codes[1]), (vs, bt.scales[1])):
        was = was.copy()
        was[page, :, slot] = got[page, :, slot]
        assert np.array_equal(got, was)


@pytest.mark.parametrize("new,ctx,Hkv,G", [([6], [130], 2, 4), ([120], [130], 2, 4), ([2], [9000], 1, 4), ([70], [9000], 1, 4)])
def test_what_is_not_finite_shows(fs, new, ctx, Hkv, G):
    """A NaN or infinite query and a NaN key that a row sees make that row NaN,
    never zeros; the rows that see none of it are right."""
    import torch

    bt = Batch(new, ctx, Hkv, 16, 94)
    _finite_cache(bt)
    n, last = new[0], int(bt.lens[0]) - 1
    r = Run(fs, bt, G)
    ref = r.want()
    keys = bt.codes[0].copy()
    keys[bt.table[0, last // 16], Hkv - 1, last % 16] = 0x7F
    r.cache[0].copy_(torch.from_numpy(keys).cuda())
    q = r.q.view(torch.int16)
    q[0, 5] = 0x7FC0                # NaN in row 0, head 0
    q[n - 2, 128 + 7] = 0x7F80      # infinity in row n - 2, head 1
    r.call()
    torch.cuda.synchronize()
    assert r.status() == 0
    bad = np.zeros((n, r.Hq), bool)
    bad[0, 0] = bad[n - 2, 1] = True
    bad[n - 1, (Hkv - 1) * G:] = True
    got = bf16_bits_to_f64(r.got()[:n, :r.Hq * 128]).reshape(n, r.Hq, 128)
    out, A, mag = ref["out"][:n], ref["absv"][:n], ref["mag"][:n, :, None]
    tol = 2.0 ** -8 * np.abs(out) + (2.0 ** -8 + 2 * (2.0 ** -17 * mag + 2.0 ** -18)) * (A + np.abs(out))
    assert np.isnan(got[bad]).all()
    assert np.all(np.abs(got - out)[~bad] <= tol[~bad])


def test_few_rows_in_a_graph(fs):
    """A captured decode step replayed with other lengths and fewer rows."""
    import torch

    bt = Batch([1, 2, 1], [700, 260, 3], 2, 16, 95, pad=2)
    _finite_cache(bt)
    r = Run(fs, bt, 4)
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        r.call(stream=s)
    for new, lens in (([1, 2, 1], [701, 262, 4]), ([1, 0, 1], [650, 0, 2]), ([2, 1, 1], [449, 113, 1])):
        bt.new, bt.lens = np.array(new), np.array(lens)
        bt.cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        for x, y in zip(r.meta[1:], (bt.cu, bt.lens.astype(np.int32))):
            x.copy_(torch.from_numpy(y).cuda())
        r.out.fill_(-7.0)
        g.replay()
        torch.cuda.synchronize()
        assert r.status() == 0
        _compare(r)


def test_two_calls_at_once(fs):
    """Calls on two streams, each with a workspace of its own."""
    import torch

    runs = []
    for seed, (new, ctx) in enumerate((([1, 1, 3], [3000, 40, 900]), ([90, 300], [1500, 0]))):
        bt = Batch(new, ctx, 2, 16, 96 + seed)
        _finite_cache(bt)
        runs.append(Run(fs, bt, 4))
    streams = [torch.cuda.Stream() for _ in runs]
    for _ in range(5):
        for r, s in zip(runs, streams):
            r.call(stream=s)
    torch.cuda.synchronize()
    for r in runs:
        assert r.status() == 0
        _compare(r)
