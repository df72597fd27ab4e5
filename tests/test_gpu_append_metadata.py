"""What the append reports: offsets and lengths outside the limits (site 1), as
the chunk attention does.  Rows of a sequence that is reported are not written."""
import numpy as np
import pytest

from tests.test_gpu_norm_rope import Batch, _append

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fs():
    import mxfp8_swiglu_mlp_gb300 as fs

    return fs


# offsets, lengths, the sequences that are reported (any of them), those appended all the same
BAD = {
    "behind the buffer": ([0, 4, 9, 23], [24, 25, 34], {2}, [0, 1]),
    "before the buffer": ([-3, 4, 9, 15], [27, 25, 26], {0}, [1, 2]),
    "decreasing": ([0, 8, 4, 15], [28, 25, 31], {1}, []),
    "shorter than its rows": ([0, 4, 9, 15], [24, 4, 26], {1}, [0, 2]),
    "beyond the table": ([0, 4, 9, 15], [24, 25, 10 ** 6], {2}, [0, 1]),
    "all behind the buffer": ([18, 19, 20, 21], [24, 25, 26], {0, 1, 2}, []),
    "all before the buffer": ([-9, -7, -5, -3], [24, 25, 26], {0, 1, 2}, []),
    "of a sequence without rows here": ([0, 4, 15, 30], [24, 31, 35], {2}, [0, 1]),
}


@pytest.mark.parametrize("what", sorted(BAD))
def test_bad_offsets_are_reported(fs, what):
    cu, lens, bad, good = BAD[what]
    bt = Batch([4, 5, 6], [20, 20, 20], 2, 16, 300)
    bt.table = np.arange(12, dtype=np.int32).reshape(3, 4)  # every place of 64 tokens has a page
    bt.max_pages, bt.pages = 4, 12
    rng = bt.rng
    bt.codes = [rng.integers(0, 255, (12, 2, 16, 128)).astype(np.uint8) for _ in range(2)]
    bt.scales = [rng.integers(100, 140, (12, 2, 16, 4)).astype(np.uint8) for _ in range(2)]
    bt.cu, bt.lens = np.array(cu, np.int32), np.array(lens)
    got, word = _append(fs, bt, False, 0, False)
    assert word >> 16 == (fs.ERR_INVALID_ARG << 8 | 1), hex(word)
    assert word & 0xFFFF in bad
    was = [bt.codes[0], bt.scales[0], bt.codes[1], bt.scales[1]]
    for b in range(3):
        t = np.arange(64)
        page, slot = bt.table[b, t // 16], t % 16
        n = cu[b + 1] - cu[b]
        new = (t >= lens[b] - n) & (t < lens[b])
        for x, y in zip(got, was):
            same = (x[page, :, slot] == y[page, :, slot]).reshape(64, -1).all(1)
            if b in bad:
                assert same.all()
            elif b in good:
                assert same[~new].all() and not same[new].any()


@pytest.mark.parametrize("B", [1, 40, 300, 1000])
def test_one_bad_length_among_many(fs, B):
    """Every sequence is looked at, whichever block and thread it falls to."""
    for b in sorted({0, B // 2, B - 1}):
        bt = Batch([1] * B, [3] * B, 1, 16, 301)
        bt.lens[b] = 0
        _, word = _append(fs, bt, False, 0, False)
        assert word == (fs.ERR_INVALID_ARG << 24 | 1 << 16 | b), hex(word)


def test_lengths_of_sequences_without_new_tokens_do_not_matter(fs):
    """Empty slots of a padded batch may hold anything."""
    bt = Batch([2, 0, 3], [5, 0, 7], 1, 16, 302)
    bt.lens[1] = -7
    got, word = _append(fs, bt, False, 0, False)
    assert word == 0
    bt.lens[1] = 0
    again, word = _append(fs, bt, False, 0, False)
    assert word == 0 and all(np.array_equal(x, y) for x, y in zip(got, again))
