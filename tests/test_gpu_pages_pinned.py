"""Pages held very often by something else: their counts stay counts, a shared
last page is split off before it is written to, and none is handed out."""
import numpy as np
import pytest

import oracle
from tests.test_gpu_pages import Tables, fs  # noqa: F401

pytestmark = pytest.mark.gpu
MOST = 1 << 30  # larger numbers count as this one


@pytest.mark.parametrize("pages", [64, 20000])  # one block, the cluster
@pytest.mark.parametrize("times", [MOST, MOST + 5, 2 ** 31 - 1])
def test_pinned_pages(fs, pages, times):  # noqa: F811
    lens = [20, 33, 16, 1, 0]
    t = Tables(fs, lens, 16, pages, 8, 11)
    held = np.zeros(pages, np.int64)
    held[t.table[0, 1]] = held[t.table[1, 0]] = held[t.table[3, 0]] = times  # a partly filled page, a full one, another partly filled
    held[np.setdiff1d(np.arange(pages), t.table)[:3]] = times                # free ones otherwise
    for parent in (None, [0, 0, 1, 3, 3]):
        keep = [18, 20, 16, 1, 1]
        want = [40, 60, 30, 1, 30]
        got, word = t.step(parent, keep, want, held)
        ref, short = oracle.pages_update(t.table, t.lens, parent, keep, want, np.minimum(held, MOST), t.P)
        assert word == 0 and short < 0
        assert ref["copy_src"][0] == t.table[0, 1]  # the oracle splits it too
        for n in ref:
            assert np.array_equal(got[n], ref[n]), n
