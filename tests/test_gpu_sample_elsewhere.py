"""Top-p's cut where the counts do not say it: logits so far below the largest one
that their distance leaves fp32, but heavy, as the temperature is as high."""
import numpy as np
import pytest

from tests.test_gpu_sample import Run, fs  # noqa: F401

pytestmark = pytest.mark.gpu


# a row in several blocks, a row in one, few and many equals of the largest logit
@pytest.mark.parametrize("V", [400, 5000, 41000, 150001])
@pytest.mark.parametrize("tops", [1, 200, 257, 0.1])
def test_the_cut_lies_among_the_lowest(fs, V, tops):  # noqa: F811
    rng = np.random.default_rng(V)
    A = int(V * tops) if isinstance(tops, float) else min(tops, V // 2)
    N = 9
    x = np.full((N, V), -3.3e38, np.float32)
    for row in x:
        row[rng.permutation(V)[:A]] = 3.3e38
        row[rng.permutation(V)[:V // 7]] = -np.inf
    p = np.linspace(0.5013, 0.9717, N).astype(np.float32)  # (equals make borders at simple fractions: none of these)
    for par in (dict(), dict(top_k=V - V // 5), dict(min_p=0.05)):
        for T in (3e38, np.inf):
            r = Run(fs, x, False, rng.random(N), temperature=T, top_p=p, **par)
            for _ in range(3):
                r.call()
            r.check()


def test_the_cut_lies_between_logits_that_the_counts_tell_apart(fs):  # noqa: F811
    """Three and more heights, the middle ones within fp32's reach of the largest."""
    rng = np.random.default_rng(4)
    x = rng.choice(np.array([3.3e38, 1e38, 0.0, -5e36, -1e38, -3.3e38], np.float32), (24, 30011))
    r = Run(fs, x, False, rng.random(24), temperature=2.5e38, top_p=np.linspace(0.02, 0.995, 24))
    for _ in range(3):
        r.call()
    r.check()
