"""Tokens from logits at temperatures at which log2(e) / T leaves fp32's normal
numbers, with u next to a border.

Borders are good to 2^-36 of the mass at any temperature (tests/test_gpu_sample.py
has why), so u may be 2^-35 from one.  The oracle's own borders are sums of 501
float64 weights and lie within 2^-43."""
import numpy as np
import pytest

from tests.test_gpu_sample import Run, fs  # noqa: F401

pytestmark = pytest.mark.gpu
NEAR, FAR = 2.0 ** -35, 2.0 ** -30


def _borders(x, T, k=0):
    """Shares of the mass up to each token, by index, of the k largest (0: all)."""
    x = x.astype(np.float64)
    w = np.exp((x - x.max()) / min(float(np.float32(T)), 3.4028234663852886e38))  # (of the fp32 temperature)
    if k:
        w[np.argsort(-x, kind="stable")[k:]] = 0.0
    s = np.cumsum(w)
    return s / s[-1]


def _next_to(shares):
    """The fp32 number in (0, 1) that is nearest to one of the shares, but not nearer than NEAR; its distance."""
    u = shares.astype(np.float32)
    u = np.concatenate([u, np.nextafter(u, np.float32(0)), np.nextafter(u, np.float32(1))])
    d = np.abs(u.astype(np.float64) - np.tile(shares, 3))
    d[(d < NEAR) | (u <= 0) | (u >= 1)] = 1.0
    # (nor may another border be nearer)
    for i in np.argsort(d):
        if np.abs(shares - float(u[i])).min() >= NEAR:
            return u[i], d[i]


def _rows(seed, N, V, T, k=0):
    """N rows of V logits across the temperature, each with such a u."""
    rng = np.random.default_rng(seed)
    x = rng.uniform(-1.0, 1.0, (N, V)) * min(T, 3.3e38)
    x = x.astype(np.float32)
    at = [_next_to(_borders(r, T, k)[:-1]) for r in x]
    u, d = (np.array(v) for v in zip(*at))
    near = d < FAR
    assert near.sum() > N // 2
    return x[near], u[near].astype(np.float32)


@pytest.mark.parametrize("k", [0, 60, 400])
@pytest.mark.parametrize("T", [2e29, 1e31, 1e35, 1e37, 1.2e38, 3e38, np.inf])
def test_next_to_a_border(fs, T, k):  # noqa: F811
    x, u = _rows(5, 120, 501, T, k)
    r = Run(fs, x, False, u, temperature=T, top_k=k)
    r.call()
    r.check()


@pytest.mark.parametrize("T", [1e37, 3e38])
def test_top_p_next_to_a_border(fs, T):  # noqa: F811
    """What is ahead of a token in the order of falling logits is all but top-p of the mass."""
    rng = np.random.default_rng(6)
    x = (rng.uniform(-1.0, 1.0, (120, 501)) * T).astype(np.float32)
    p, d = (np.array(v) for v in zip(*[_next_to(_borders(-np.sort(-r), T)[:-1]) for r in x]))
    near = d < FAR
    assert near.sum() > 60
    # (a u just below 1 is drawn from the last of the kept tokens, by index: half of them change with the cut)
    r = Run(fs, x[near], False, np.full(int(near.sum()), 0.99999, np.float32), temperature=T, top_p=p[near])
    r.call()
    r.check()


@pytest.mark.parametrize("k", [0, 60])
def test_many_long_rows_next_to_a_border(fs, k):  # noqa: F811
    x, u = _rows(7, 300, 40001, 3e38, k)
    assert len(x) >= 128  # (a block a row, then the clusters)
    r = Run(fs, x, False, u, temperature=3e38, top_k=k)
    r.call()
    r.check()


# logits on both sides of 2^109, from where on such a temperature's weights are taken in fp64, and ordinary ones;
# forbidden logits are none of them
@pytest.mark.parametrize("V", [501, 40001])
@pytest.mark.parametrize("T,size", [(6e32, 6.4e32), (6e32, 7e32), (1e35, 6.4e32), (1.2e38, 6.4e32), (3e38, 6.4e32), (np.inf, 6.4e32),
                                    (np.inf, 1e20), (np.inf, 3.0)])
def test_logits_smaller_than_the_temperature(fs, T, size, V):  # noqa: F811
    rng = np.random.default_rng(8)
    x = (rng.uniform(-1.0, 1.0, (40, V)) * size).astype(np.float32)
    x[:, 3::5] = -np.inf
    u, d = (np.array(v) for v in zip(*[_next_to(_borders(r, T)[:-1]) for r in x]))
    near = d < FAR
    assert near.sum() > 20
    r = Run(fs, x[near], False, u[near].astype(np.float32), temperature=T)
    r.call()
    r.check()
