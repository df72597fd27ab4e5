"""Scores beyond what a running maximum in fp32 can stand for: the rows whose
largest score (in powers of two) is 2^31 or more away from zero are NaN, never
zeros or something finite; below, outputs are averages of the values."""
import numpy as np
import pytest

import oracle
from tests._util import bf16_bits_to_f64
from tests.test_gpu_chunk_attention import Run, _finite_cache
from tests.test_gpu_norm_rope import Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fs():
    import mxfp8_swiglu_mlp_gb300 as fs

    return fs


def _check(fs, new, ctx, G, sm, key_scale, every):
    """Key scales 2^key_scale times those of ordinary keys, doubled every `every`
    tokens (0: never)."""
    import torch

    bt = Batch([new], [ctx], 1, 16, 500)
    _finite_cache(bt)
    L = new + ctx
    t = np.arange(L)
    page, slot = bt.table[0, t // 16], t % 16
    up = key_scale + (t // every if every else 0 * t)
    bt.scales[0][page, :, slot] = np.clip(bt.scales[0][page, :, slot].astype(int) + up[:, None, None], 1, 250)
    r = Run(fs, bt, G, sm=sm)
    r.call()
    torch.cuda.synchronize()
    assert r.status() == 0
    got = bf16_bits_to_f64(r.got()[:new, :G * 128]).reshape(new, G, 128)
    k, v = (oracle.dequantize(bt.codes[i][page, 0, slot], bt.scales[i][page, 0, slot]) for i in (0, 1))
    q = bf16_bits_to_f64(r.qbits)
    top = np.empty((new, G))
    for h in range(G):
        s = sm * (q[:, h] @ k.T) * np.log2(np.e)
        top[:, h] = np.where(t <= np.arange(ctx, L)[:, None], s, -np.inf).max(1)
    # (the largest score is off by 2^-16 of the sum of its products' magnitudes, far below a factor of two)
    beyond, within = np.abs(top) >= 2.0 ** 32, np.abs(top) <= 2.0 ** 29
    assert np.isnan(got[beyond]).all()
    assert np.isfinite(got[within]).all() and np.abs(got[within]).max(initial=0) <= (1 + 2.0 ** -6) * np.abs(v).max()
    return beyond.mean(), within.mean()


SHAPES = [(2, 300, 4), (2, 9000, 4), (60, 200, 1), (300, 40, 2), (64, 9000, 1)]


@pytest.mark.parametrize("sm", [1e30, -1e30, 1e15])
@pytest.mark.parametrize("new,ctx,G", SHAPES)
def test_scales_that_no_softmax_has(fs, new, ctx, G, sm):
    beyond, _ = _check(fs, new, ctx, G, sm, 0, 0)
    assert beyond == 1


@pytest.mark.parametrize("new,ctx,G", SHAPES)
def test_keys_that_keep_growing(fs, new, ctx, G):
    _check(fs, new, ctx, G, 1.0, 8, 40 if ctx < 1000 else 300)


@pytest.mark.parametrize("sm", [1.0, -1.0])
@pytest.mark.parametrize("new,ctx,G", SHAPES)
def test_large_scores_within_the_limit(fs, new, ctx, G, sm):
    _, within = _check(fs, new, ctx, G, sm, 20, 0)
    assert within > 0.9
