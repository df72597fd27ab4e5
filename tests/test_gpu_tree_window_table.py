"""Trees with a window: a table with more room than the window changes nothing, to
the last bit; and windows where there are many query tiles."""
import numpy as np
import pytest

from tests._util import bf16_bits_to_f64
from tests.test_gpu_chunk_attention import _compare, _finite_cache
from tests.test_gpu_norm_rope import Batch, _dev
from tests.test_gpu_tree_attention import Run, _wide, fs  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("new,ctx,Hkv,G,window", [([16], [3000], 8, 4, 512), ([64], [1500], 8, 4, 100), ([16, 9, 12], [900, 40, 700], 2, 4, 300)])
def test_the_tables_room_behind_a_window_does_not_matter(fs, new, ctx, Hkv, G, window):  # noqa: F811
    """The same kernel and plan: what a sequence's rows see is no longer for it."""
    import torch

    outs = []
    for wide in (False, True):
        bt = Batch(new, ctx, Hkv, 16, 90)
        _finite_cache(bt)
        r = Run(fs, _wide(bt) if wide else bt, G, window=window)
        r.call()
        torch.cuda.synchronize()
        assert r.status() == 0
        _compare(r)
        outs.append(r.got())
    assert np.array_equal(*outs)


# More query tiles than there are blocks (32 rows each): the kernel for many rows, whatever the window.
def _many_tiles(bt, G):
    rows = -(-bt.T * G // bt.B)
    assert -(-rows // 32) * bt.B * bt.Hkv > 152
    return bt


@pytest.mark.parametrize("kind", ["tree", "bits", "gaps"])
@pytest.mark.parametrize("window", [1, 5, 40, 100, 300])
def test_windows_and_many_query_tiles(fs, window, kind):  # noqa: F811
    import torch

    bt = _many_tiles(Batch([90, 200], [260, 400], 8, 16, window % 89), 3)
    _finite_cache(bt)
    r = Run(fs, bt, 3, kind, window)
    r.call()
    torch.cuda.synchronize()
    assert r.status() == 0
    _compare(r)


def test_rows_that_see_nothing_and_many_query_tiles(fs):  # noqa: F811
    """A window of one leaves no held token to a row of an empty mask."""
    import torch

    bt = _many_tiles(Batch([150, 20], [90, 2000], 8, 16, 5), 4)
    _finite_cache(bt)
    r = Run(fs, bt, 4, "empty", 1)
    r.call()
    torch.cuda.synchronize()
    assert r.status() == 0
    _compare(r)


@pytest.mark.parametrize("window", [40, 300])
def test_nan_at_the_ends_of_windows_and_many_query_tiles(fs, window):  # noqa: F811
    """NaN in the first and last token that not every row sees."""
    import torch

    n, ctx = 256, 333
    for which in (0, 1):
        bt = _many_tiles(Batch([n, 3], [ctx, 50], 5, 16, 50 + n), 4)
        _finite_cache(bt)
        r = Run(fs, bt, 4, "bits", window)
        ref = r.want()["out"]
        nan = np.zeros(bt.T, bool)
        for t in (ctx - window + 1, ctx + n - window if window < n else ctx, ctx + n - 1, ctx):
            r.cache[2 * which][bt.table[0, t // 16], :, t % 16, 9] = 0x7F
            for i in range(n):
                nan[i] |= (r.masks[0][i, t - ctx] and t - ctx <= i) if t >= ctx else t > r.pos[i] - window
        r.call()
        torch.cuda.synchronize()
        assert r.status() == 0
        got = bf16_bits_to_f64(r.got()).reshape(bt.T, r.Hq, 128)
        assert np.array_equal(np.isnan(got).any(axis=2), np.repeat(nan[:, None], r.Hq, 1))
        assert np.abs(got - ref)[~nan].max() <= 0.02 * np.abs(ref).max()


# both kernels
@pytest.mark.parametrize("Hkv", [2, 8])
@pytest.mark.parametrize("window", [1, 7, 33])
def test_a_chain_longer_than_a_sliding_window(fs, window, Hkv):  # noqa: F811
    """With the bits of the nodes a window away left out it is a causal chunk with that window."""
    import oracle
    import torch

    bt = Batch([150, 70], [90, 10], Hkv, 16, 40 + window)
    _finite_cache(bt)
    r = Run(fs, bt, 4, "tree", window)
    r.masks = [np.tril(np.ones((n, n), bool)) & ~np.tril(np.ones((n, n), bool), -window) for n in (150, 70)]
    r.pos = np.concatenate([c + np.arange(n) for n, c in ((150, 90), (70, 10))]).astype(np.int32)
    r.mask.copy_(_dev(oracle.pack_mask(r.masks, r.words, bt.T).view(np.int32)))
    r.dpos.copy_(_dev(r.pos))
    chunk = oracle.paged_chunk_attention(bf16_bits_to_f64(r.qbits), bt.codes[0], bt.scales[0], bt.codes[1], bt.scales[1],
                                         bt.table, bt.cu, bt.lens, window, r.sm)
    assert np.abs(r.want()["out"] - chunk["out"]).max() <= 1e-12 * np.abs(chunk["out"]).max()
    r.call()
    torch.cuda.synchronize()
    assert r.status() == 0
    _compare(r)
