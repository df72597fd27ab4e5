"""How near u may come to a border.

A weight is a whole number of units, 2^-45 of the largest one: it is off by a unit
at most, and by 2^-37 of itself (its power of two is good to half a unit of 2^-38 in
each of two parts and the exponent to 2^-39 in the rest).  Where many weights are
alike, they are all rounded alike: V of them move a border by V units.  So a border
lies within 2^-36 + V 2^-45 (largest weight / mass) of the mass of the exact one."""
import numpy as np
import pytest

from tests.test_gpu_sample import Run, fs  # noqa: F401

pytestmark = pytest.mark.gpu


def _next_to(x, T):
    """The fp32 number nearest to a border of the unfiltered row, but no nearer than the bound."""
    w = np.exp((x.astype(np.float64) - x.max()) / T)
    s = np.cumsum(w)
    shares, near = s[:-1] / s[-1], 2.0 ** -36 + len(x) * 2.0 ** -45 / s[-1]
    u = shares.astype(np.float32)
    u = np.unique(np.concatenate([u, np.nextafter(u, np.float32(0)), np.nextafter(u, np.float32(1))]))
    u = u[(u > 0) & (u < 1)]
    at = np.searchsorted(shares, u.astype(np.float64))
    d = np.minimum(np.abs(shares[np.minimum(at, len(shares) - 1)] - u), np.abs(shares[np.maximum(at - 1, 0)] - u))
    d[d < near] = 2.0
    i = int(np.argmin(d))
    assert d[i] < 8 * near
    return u[i]


# (few rows, and as many as have a block each; one block a row and several)
@pytest.mark.parametrize("N,V", [(24, 43060), (24, 5000), (130, 43060)])
def test_many_weights_alike(fs, N, V):  # noqa: F811
    """One token has nearly all of the mass, the others some 10^6 units each, rounded to the same whole number."""
    rng = np.random.default_rng(V + N)
    x = np.broadcast_to(np.float32(-17.4) + np.arange(N, dtype=np.float32)[:, None] * 2.0 ** -12, (N, V)).astype(np.float32).copy()
    x[np.arange(N), rng.integers(0, V, N)] = 0.0
    r = Run(fs, x, False, np.array([_next_to(row, 1.0) for row in x]))
    r.call()
    r.check()


@pytest.mark.parametrize("half", [True, False], ids=["bf16", "fp32"])
@pytest.mark.parametrize("T,shift", [(1.0, 0.0), (0.7, 0.0), (0.25, 300.0), (1.0, -1300.0)])
def test_next_to_a_border(fs, half, T, shift):  # noqa: F811
    """Also where powers are near the largest that the table's way takes."""
    from tests._util import bf16_bits_to_f64
    from workloads import inputs

    rng = np.random.default_rng(int(T * 8 + abs(shift)))
    x = (rng.standard_normal((60, 3001)) * 0.5 + shift).astype(np.float32)
    if half:
        x = bf16_bits_to_f64(inputs.bf16_bits_from_f32(x)).astype(np.float32)
    r = Run(fs, x, half, np.array([_next_to(row, float(np.float32(T))) for row in x]), temperature=T)
    r.call()
    r.check()
