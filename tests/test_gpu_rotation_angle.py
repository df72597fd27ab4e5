"""The rotation's angle at far positions: within 2^-25 turns at any position, for
frequencies up to 2^40.  Shown where it can be seen through a bf16 result: at
positions that come back to nearly a whole number of turns, where the sine is a
millionth or so.  The pair (1, 0) is turned, so the second element is the sine:
off by at most 2 pi 2^-25, its rounding to bf16 (2^-8) and 2^-21 relative for
the sine itself."""
from fractions import Fraction
import math

import numpy as np
import pytest

from tests._util import to_dev_u16, from_dev_bf16, bf16_bits_to_f64

BITS = 300


def _arctan_inverse(x):
    term = (1 << BITS) // x
    total, n = term, 1
    while term:
        term //= -x * x
        n += 2
        total += term // n
    return total


def _turns_per_radian():
    """1 / (2 pi) by Machin's formula, to some 290 bits."""
    pi = 4 * (4 * _arctan_inverse(5) - _arctan_inverse(239))
    return Fraction(1 << BITS, 2 * pi)


def _fraction(f):
    """f / 2 pi without its whole turns, in 2^-64 turns."""
    t = Fraction(float(f)) * _turns_per_radian()
    return round((t - round(t)) * 2 ** 64) % 2 ** 64


def test_turns_per_radian():
    assert abs(float(_turns_per_radian()) * 2 * math.pi - 1) < 1e-15


FREQ = np.array([1.0, 0.9375, 0.87, 0.5, 0.25, 0.1, 1e-3, 3.7, 10.0, 99.0, 1000.0, 65536.3, 1e6, 2.0 ** 30 + 2 ** 10, 2.0 ** 40,
                 -7.3], np.float32)


@pytest.mark.gpu
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("top", [2 ** 31 - 1, 2 ** 24, -2 ** 31 + 2 ** 22])
def test_angles_of_far_positions(top, interleaved):
    import torch

    import mxfp8_swiglu_mlp_gb300 as fs

    p = np.arange(top - 2 ** 22 + 1, top + 1, dtype=np.int64)
    positions, which, angle = [], [], []
    for i, f in enumerate(FREQ):
        turns = (p.astype(np.uint64) * np.uint64(_fraction(f))).astype(np.int64)  # modulo a turn, signed; off by p 2^-65
        best = np.argpartition(np.abs(turns), 6)[:6]
        positions += p[best].tolist()
        which += [i] * len(best)
        angle += (turns[best] * (2 * math.pi / 2 ** 64)).tolist()
    T = len(positions)
    x = np.zeros((T, 32), np.uint16)
    first = np.array(which) * 2 if interleaved else np.array(which)
    second = first + (1 if interleaved else 16)
    x[np.arange(T), first] = 0x3F80
    d = to_dev_u16(x)
    y = torch.empty_like(d)
    pos, fr = torch.tensor(positions, dtype=torch.int32, device="cuda"), torch.from_numpy(FREQ).cuda()
    fs.fsops_qk_norm_rope(d, 32, None, 0, None, None, 0.0, pos, (fr, 32, interleaved), y, 32, None, 0, T, 1, 0, 32)
    torch.cuda.synchronize()
    got = bf16_bits_to_f64(from_dev_bf16(y))[np.arange(T), second]
    want = np.sin(angle)
    tol = 2 * math.pi * 2.0 ** -25 + (2.0 ** -8 + 2.0 ** -21) * np.abs(want)
    assert np.all(np.abs(got - want) <= tol), (np.abs(got - want) / tol).reshape(len(FREQ), -1).max(1)
