"""A wait of the chunk attention that runs out: the block leaves its roles, what
it has in flight ends, FSOPS_ERR_TIMEOUT is in the status word, and with the
workspace zeroed the next call is right.  The hook asks for one arrival more
than any product makes on the barriers that say that outputs are done; the
limit is short."""
import pytest

from tests.test_gpu_chunk_attention import Run, _compare, _finite_cache
from tests.test_gpu_norm_rope import Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fs():
    import mxfp8_swiglu_mlp_gb300 as fs

    return fs


@pytest.fixture
def short(fs):
    fs.fsops_set_wait_timeout_ns(5_000_000)
    yield
    fs.fsops_debug_set_extra_arrivals(0)
    fs.fsops_set_wait_timeout_ns(1_000_000_000)


# the last item of a block (its product warps have left by then), an item among others, long ones split over
# blocks; few rows and many
CASES = [([1], [40], 1, 1), ([3], [1000], 2, 4), ([4] * 70, [500] * 70, 4, 8), ([1], [12000], 1, 4),
         ([40], [60], 1, 1), ([300], [200], 1, 2), ([512] * 3, [700] * 3, 8, 4), ([64], [9000], 1, 4)]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_a_wait_that_runs_out_is_reported(fs, short, i):
    import torch

    new, ctx, Hkv, G = CASES[i]
    bt = Batch(new, ctx, Hkv, 16, 400 + i)
    _finite_cache(bt)
    r = Run(fs, bt, G)
    fs.fsops_debug_set_extra_arrivals(1)
    r.call()
    torch.cuda.synchronize()
    word = r.status()
    # (the site is whichever of the block's warps gave up first: others wait for those that wait for the outputs)
    assert word >> 24 == fs.ERR_TIMEOUT and (word >> 16) & 0xFF != 0, hex(word)
    fs.fsops_debug_set_extra_arrivals(0)
    fs.fsops_set_wait_timeout_ns(1_000_000_000)
    r.ws.zero_()
    r.out.fill_(-7.0)
    r.call()
    torch.cuda.synchronize()
    assert r.status() == 0
    _compare(r)


@pytest.mark.parametrize("i", range(len(CASES)))
def test_waits_of_almost_no_time(fs, short, i):
    """A limit of one try: whichever wait runs out, or none, the call ends and the
    next one is right."""
    import torch

    new, ctx, Hkv, G = CASES[i]
    bt = Batch(new, ctx, Hkv, 16, 420 + i)
    _finite_cache(bt)
    r = Run(fs, bt, G)
    for ns in (1, 2000, 20000):
        fs.fsops_set_wait_timeout_ns(ns)
        for _ in range(3):
            r.ws.zero_()
            r.call()
            torch.cuda.synchronize()
            assert r.status() >> 24 in (0, fs.ERR_TIMEOUT)
    fs.fsops_set_wait_timeout_ns(1_000_000_000)
    r.ws.zero_()
    r.out.fill_(-7.0)
    r.call()
    torch.cuda.synchronize()
    assert r.status() == 0
    _compare(r)
