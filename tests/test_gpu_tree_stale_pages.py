"""Which page ids the attention of trees looks up: those of the tokens from the
first that the window leaves to a node at the root's place on, whatever masks and
positions say; none before them, none behind the sequence."""
import numpy as np
import pytest

from tests._util import bf16_bits_to_f64
from tests.test_gpu_chunk_attention import _compare, _finite_cache
from tests.test_gpu_norm_rope import Batch, _dev
from tests.test_gpu_tree_attention import Run, fs  # noqa: F401

pytestmark = pytest.mark.gpu


# both kernels: few query tiles, more than there are blocks
@pytest.mark.parametrize("Hkv,G,n", [(2, 4, 12), (8, 4, 180)])
@pytest.mark.parametrize("window", [1, 17, 200])
def test_stale_ids_outside_what_is_looked_up(fs, Hkv, G, n, window):  # noqa: F811
    import torch

    P = 16
    bt = Batch([n, 3], [500, 60], Hkv, P, window)
    _finite_cache(bt)
    r = Run(fs, bt, G, "gaps", window)
    table = bt.table.copy()
    for b in range(bt.B):
        base = int(bt.lens[b] - bt.new[b])
        table[b, :max(0, base - window + 1) // P] = bt.pages + 7
        table[b, -(-int(bt.lens[b]) // P):] = -5
    r.meta[0].copy_(_dev(table))
    r.call()
    torch.cuda.synchronize()
    assert r.status() == 0
    _compare(r)


@pytest.mark.parametrize("Hkv,G,n", [(2, 4, 12), (8, 4, 180)])
def test_an_id_that_no_mask_names_is_looked_up(fs, Hkv, G, n):  # noqa: F811
    """Unused nodes at the end of a padded tree want valid ids as well: a bad one is
    reported and not followed, and the other sequence is right."""
    import torch

    bt = Batch([n, 3], [500, 60], Hkv, 16, 3)
    _finite_cache(bt)
    r = Run(fs, bt, G, "empty", 200)
    ref = r.want()["out"]
    table = bt.table.copy()
    table[0, (500 + n - 1) // 16] = bt.pages
    r.meta[0].copy_(_dev(table))
    r.call()
    torch.cuda.synchronize()
    assert r.status() == (fs.ERR_INVALID_ARG << 24) | 2 << 16
    got = bf16_bits_to_f64(r.got()).reshape(bt.T, r.Hq, 128)
    assert np.linalg.norm(got[n:] - ref[n:]) <= 3.5e-3 * np.linalg.norm(ref[n:])
