"""Sequences of a padded batch that have nothing to move, whatever their other numbers are."""
import numpy as np
import pytest

import oracle
from tests.test_gpu_norm_rope import _dev
from tests.test_gpu_pages import _cache, _status, fs  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("start", [-1, -(2 ** 31), 64, 2 ** 31 - 1])
def test_a_sequence_without_tokens_is_not_an_error(fs, start):  # noqa: F811
    import torch

    rng = np.random.default_rng(8)
    cache = _cache(rng, 2, 12, 2, 16)
    table = np.arange(12, dtype=np.int32).reshape(3, 4)
    table[1] = -1
    starts, path = np.array([5, start, 9], np.int32), np.array([[1, 4], [-3, -3], [0, 20]], np.int32)
    counts = np.array([2, 0, 2], np.int32)
    dev, st = [_dev(x) for x in cache], _status()
    fs.fsops_mxfp8_kv_compact(*dev, 12, 2, _dev(table), 4, _dev(starts), _dev(path), 2, _dev(counts), 3, 2, 128, 16, st)
    torch.cuda.synchronize()
    for x, y in zip(oracle.compact(cache, table, starts, path, counts, 16), dev):
        assert np.array_equal(y.cpu().numpy(), x)
    assert fs.fsops_read_kernel_status(st) == 0


def test_a_start_below_zero_with_tokens_still_is(fs):  # noqa: F811
    import torch

    rng = np.random.default_rng(9)
    cache = _cache(rng, 2, 12, 2, 16)
    table = np.arange(12, dtype=np.int32).reshape(3, 4)
    starts, path = np.array([5, -1, 9], np.int32), np.array([[1, 4], [2, 3], [0, 20]], np.int32)
    counts = np.array([2, 2, 2], np.int32)
    dev, st = [_dev(x) for x in cache], _status()
    fs.fsops_mxfp8_kv_compact(*dev, 12, 2, _dev(table), 4, _dev(starts), _dev(path), 2, _dev(counts), 3, 2, 128, 16, st)
    torch.cuda.synchronize()
    assert fs.fsops_read_kernel_status(st) == 1 << 24 | 1 << 16 | 1
    counts[1] = 0
    for x, y in zip(oracle.compact(cache, table, starts, path, counts, 16), dev):
        assert np.array_equal(y.cpu().numpy(), x)
