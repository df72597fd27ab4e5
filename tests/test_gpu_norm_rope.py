"""Per-head norm and rotation, and the append to the paged MXFP8 cache, against
the float64 oracle.

Tolerances.  In fp32 the kernels add up to 256 squares (20 sequential and
shuffled additions a lane, so the mean is good to 2^-19.7 and its root to
2^-20.7), take rsqrt (2^-22), three products and one fused pair; the angle is
good to 2^-23 turns of a half and sine and cosine to 2 ulp, 2^-22 together.
All of it stays below 2^-19 of the pair's length (of the value itself where
nothing is rotated).  A bf16 result then adds its rounding, 2^-8 relative; an
E4M3 code half a step, 2^-4 relative or 2^-10 of the block's scale."""
import numpy as np
import pytest

import oracle
from workloads import inputs
from tests._util import to_dev_u16, from_dev_bf16, bf16_bits_to_f64

pytestmark = pytest.mark.gpu
FP32 = 2.0 ** -19


@pytest.fixture(scope="module")
def fs():
    import mxfp8_swiglu_mlp_gb300 as fs

    return fs


def _bits(rng, *shape, spread=1.0):
    x = rng.standard_normal(shape) * np.exp(spread * rng.standard_normal(shape[:-1] + (1,)))
    return inputs.bf16_bits_from_f32(x.astype(np.float32))


def _freq(R, theta=1e4):
    return (theta ** (-np.arange(0, R, 2) / max(R, 1))).astype(np.float32)


def _pair_length(x, R, interleaved):
    """|(u, w)| at both elements of each rotated pair, |x| elsewhere."""
    m = np.abs(x)
    if R:
        first = slice(0, R, 2) if interleaved else slice(0, R // 2)
        second = slice(1, R, 2) if interleaved else slice(R // 2, R)
        h = np.hypot(x[..., first], x[..., second])
        m[..., first], m[..., second] = h, h
    return m


def _dev(a):
    import torch

    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


# T, Hq, Hkv, D, R, interleaved, norm, highest position
CASES = [(1, 32, 8, 128, 128, False, True, 5000), (3, 5, 1, 64, 64, False, True, 100), (70, 7, 3, 96, 96, True, True, 900),
         (130, 14, 2, 64, 32, True, False, 2 ** 31 - 1), (9, 3, 2, 192, 128, False, True, 10 ** 6), (5, 2, 1, 256, 256, False, False, 40),
         (33, 1, 1, 80, 64, False, True, 70), (4, 3, 0, 16, 0, False, True, 1), (2, 0, 3, 48, 32, True, True, 9),
         (700, 16, 4, 128, 64, False, True, 131072), (4099, 4, 2, 128, 128, True, True, 4100)]


def _norm_rope(fs, c, seed, in_place=False, stream=None):
    import torch

    T, Hq, Hkv, D, R, inter, norm, far = c
    rng = np.random.default_rng(seed)
    H = Hq + Hkv
    ld = H * D + 24  # rows of one buffer, with a gap
    buf = np.zeros((T, ld), np.uint16)
    buf[:, :H * D] = _bits(rng, T, H, D).reshape(T, -1)
    gam = inputs.bf16_bits_from_f32((1 + 0.2 * rng.standard_normal((2, D))).astype(np.float32))
    pos = rng.integers(0, far, T, endpoint=True).astype(np.int32)
    pos[0] = far
    f = _freq(R)
    d, gd = to_dev_u16(buf), to_dev_u16(gam)
    q, k = (d[:, :Hq * D] if Hq else None), (d[:, Hq * D:] if Hkv else None)
    if in_place:
        qo, ko, ldqo, ldko = q, k, ld, ld
    else:
        ldqo, ldko = Hq * D + 8, Hkv * D
        qo = torch.full((T, ldqo), -7.0, dtype=torch.bfloat16, device="cuda") if Hq else None
        ko = torch.full((T, ldko), -7.0, dtype=torch.bfloat16, device="cuda") if Hkv else None
    fs.fsops_qk_norm_rope(q, ld, k, ld, gd[0] if norm else None, gd[1] if norm else None, 1e-5, _dev(pos) if R else None,
                          (_dev(f), R, inter) if R else None, qo, ldqo, ko, ldko, T, Hq, Hkv, D, stream)
    torch.cuda.synchronize()
    x = bf16_bits_to_f64(buf[:, :H * D]).reshape(T, H, D)
    g = bf16_bits_to_f64(gam)
    for out, h0, h1, gi in ((qo, 0, Hq, 0), (ko, Hq, H, 1)):
        if out is None:
            continue
        args = (g[gi] if norm else None, 1e-5, pos)
        want = oracle.norm_rope(x[:, h0:h1], *args, f, R, inter)
        size = _pair_length(oracle.norm_rope(x[:, h0:h1], *args, f, 0, inter), R, inter)
        bits = from_dev_bf16(out)
        got = bf16_bits_to_f64(bits[:, :(h1 - h0) * D]).reshape(want.shape)
        err = np.abs(got - want) - 2.0 ** -8 * np.abs(want) - 2 * FP32 * size
        assert np.all(err <= 0), (float(err.max()), np.unravel_index(err.argmax(), err.shape))
        if out is qo and not in_place:
            assert np.all(bits[:, Hq * D:] == 0xC0E0)  # the gap between rows: -7 as it was
    if in_place:
        assert np.all(from_dev_bf16(d)[:, H * D:] == 0)


@pytest.mark.parametrize("c", CASES, ids=lambda c: "-".join(map(str, c)))
def test_norm_rope_matches_oracle(fs, c):
    _norm_rope(fs, c, seed=sum(map(int, c[:6])))


@pytest.mark.parametrize("c", [CASES[2], CASES[9]], ids=lambda c: "-".join(map(str, c)))
def test_norm_rope_in_place(fs, c):
    _norm_rope(fs, c, seed=7, in_place=True)


def test_norm_rope_negative_position_turns_back(fs):
    """Position -p undoes position p, to the two bf16 roundings."""
    import torch

    rng = np.random.default_rng(3)
    x = _bits(rng, 5, 2, 128, spread=0.0)
    f = _dev(_freq(128))
    pos = np.array([1, 5, 77, 4096, 2 ** 30], np.int32)
    d = to_dev_u16(x.reshape(5, 256))
    y, z = torch.empty_like(d), torch.empty_like(d)
    fs.fsops_qk_norm_rope(d, 256, None, 0, None, None, 0.0, _dev(pos), (f, 128, False), y, 256, None, 0, 5, 2, 0, 128)
    fs.fsops_qk_norm_rope(y, 256, None, 0, None, None, 0.0, _dev(-pos), (f, 128, False), z, 256, None, 0, 5, 2, 0, 128)
    torch.cuda.synchronize()
    x = bf16_bits_to_f64(x)
    size = _pair_length(x, 128, False)
    got = bf16_bits_to_f64(from_dev_bf16(z)).reshape(x.shape)
    assert np.all(np.abs(got - x) <= (2 * 2.0 ** -8 + 4 * FP32) * np.sqrt(2) * size)


# ---------------------------------------------------------------- append
class Batch:
    def __init__(self, new, ctx, Hkv, P, seed, pad=0, extra_pages=3):
        rng = np.random.default_rng(seed)
        self.new, self.lens = np.array(new), np.array(new) + np.array(ctx)
        self.B, self.Hkv, self.P = len(new), Hkv, P
        self.cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.T = int(self.cu[-1]) + pad
        npg = [-(-int(n) // P) for n in self.lens]
        self.pages = sum(npg) + extra_pages
        perm = rng.permutation(self.pages).astype(np.int32)
        self.table = np.full((self.B, max(max(npg), 1) + 1), -1, np.int32)
        at = 0
        for b, n in enumerate(npg):
            self.table[b, :n] = perm[at:at + n]
            at += n
        self.max_pages = self.table.shape[1]
        shape = (self.pages, Hkv, P)
        self.codes = [rng.integers(0, 255, shape + (128,)).astype(np.uint8) for _ in range(2)]
        self.scales = [rng.integers(100, 140, shape + (4,)).astype(np.uint8) for _ in range(2)]
        self.k, self.v = (_bits(rng, self.T, Hkv, 128) for _ in range(2))
        self.gamma = inputs.bf16_bits_from_f32((1 + 0.2 * rng.standard_normal(128)).astype(np.float32))
        self.rng = rng

    def where(self):
        """Sequence, place, page and slot of each row in use."""
        b = np.repeat(np.arange(self.B), self.new)
        place = np.concatenate([np.arange(L - n, L) for n, L in zip(self.new, self.lens)]).astype(np.int64)
        return b, place, self.table[b, place // self.P], place % self.P


def _append(fs, bt, norm, R, inter, positions=None, stream=None, graph=False):
    import torch

    HD = bt.Hkv * 128
    rows = np.zeros((bt.T, 2 * HD + 8), np.uint16)
    rows[:, :HD], rows[:, HD:2 * HD] = bt.k.reshape(bt.T, -1), bt.v.reshape(bt.T, -1)
    d = to_dev_u16(rows)
    cache = [_dev(x) for x in (bt.codes[0], bt.scales[0], bt.codes[1], bt.scales[1])]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    keep = [_dev(bt.table), _dev(bt.cu), _dev(bt.lens.astype(np.int32)), _dev(_freq(R)), to_dev_u16(bt.gamma),
            _dev(positions) if positions is not None else None]
    torch.cuda.synchronize()
    fs.fsops_mxfp8_kv_append(d, rows.shape[1], d[:, HD:], rows.shape[1], keep[4] if norm else None, 1e-6, keep[5],
                             (keep[3], R, inter) if R else None, *cache, bt.pages, keep[0], bt.max_pages, keep[1], keep[2],
                             bt.T, bt.B, bt.Hkv, 128, bt.P, status, stream)
    torch.cuda.synchronize()
    return [x.cpu().numpy() for x in cache], fs.fsops_read_kernel_status(status)


APPENDS = [([1], [0], 1, 16, 0), ([1] * 7, [0, 15, 16, 17, 100, 31, 63], 8, 16, 0), ([5, 0, 130, 1, 0], [0, 9, 33, 64, 0], 3, 64, 9),
           ([300, 17], [1, 900], 5, 128, 1), ([0, 0], [5, 0], 2, 32, 4), ([1] * 70 + [0] * 40 + [2] * 3, list(range(113)), 2, 32, 0)]


@pytest.mark.parametrize("norm,R,inter", [(True, 128, False), (True, 64, True), (False, 96, False), (False, 0, False), (True, 0, False)])
@pytest.mark.parametrize("i", range(len(APPENDS)))
def test_append_matches_oracle(fs, i, norm, R, inter):
    new, ctx, Hkv, P, pad = APPENDS[i]
    bt = Batch(new, ctx, Hkv, P, 10 * i + R, pad)
    (kc, ks, vc, vs), status = _append(fs, bt, norm, R, inter)
    assert status == 0
    b, place, page, slot = bt.where()
    n = len(b)
    # V: the plain quantiser's bits
    c, s = oracle.quantize_bf16(bt.v[:n].reshape(-1, 128))
    assert np.array_equal(vc[page, :, slot], c.reshape(n, Hkv, 128))
    assert np.array_equal(vs[page, :, slot], s.reshape(n, Hkv, 4))
    gk, gs = kc[page, :, slot], ks[page, :, slot]
    if not norm and not R:
        c, s = oracle.quantize_bf16(bt.k[:n].reshape(-1, 128))
        assert np.array_equal(gk, c.reshape(n, Hkv, 128)) and np.array_equal(gs, s.reshape(n, Hkv, 4))
    elif n:
        g = bf16_bits_to_f64(bt.gamma) if norm else None
        x = bf16_bits_to_f64(bt.k[:n])
        want = oracle.norm_rope(x, g, 1e-6, place, _freq(R), R, inter)
        size = _pair_length(oracle.norm_rope(x, g, 1e-6, place, _freq(R), 0, inter), R, inter)
        err = 2 * FP32 * size
        # the scale byte is one of those that values this near can have
        am, slack = np.abs(want).reshape(n, Hkv, 4, 32).max(-1), err.reshape(n, Hkv, 4, 32).max(-1)
        for side, sign in ((am - slack, 1), (am + slack, -1)):
            e = np.frexp(np.maximum(side, 0))[1] - 9 + 127
            e = np.where(side > 0, e, 0)
            assert np.all(sign * (gs.astype(np.int64) - np.clip(e, 0, 254)) >= 0)
        unit = np.repeat(np.ldexp(1.0, gs.astype(np.int64) - 127), 32, axis=-1)
        got = oracle.dequantize(gk.reshape(-1, 128), gs.reshape(-1, 4)).reshape(want.shape)
        clipped = np.clip(want, -448 * unit, 448 * unit)
        assert np.all(np.abs(got - clipped) <= np.maximum(2.0 ** -4 * np.abs(clipped), 2.0 ** -10 * unit) + err)
    # every other slot is as it was
    for got, was in ((kc, bt.codes[0]), (ks, bt.scales[0]), (vc, bt.codes[1]), (vs, bt.scales[1])):
        was = was.copy()
        was[page, :, slot] = got[page, :, slot]
        assert np.array_equal(got, was)


def test_append_given_positions(fs):
    """Positions apart from the places (the rotation follows them)."""
    bt = Batch([40, 3], [0, 50], 2, 32, 5)
    pos = bt.rng.integers(0, 2 ** 20, bt.T).astype(np.int32)
    (kc, ks, _, _), status = _append(fs, bt, True, 128, False, positions=pos)
    assert status == 0
    b, place, page, slot = bt.where()
    want = oracle.norm_rope(bf16_bits_to_f64(bt.k), bf16_bits_to_f64(bt.gamma), 1e-6, pos, _freq(128), 128, False)
    got = oracle.dequantize(kc[page, :, slot].reshape(-1, 128), ks[page, :, slot].reshape(-1, 4)).reshape(want.shape)
    # E4M3 of normal values, saturation included: 448 stands for up to 512, an eighth
    big = np.abs(want) >= np.repeat(np.ldexp(1.0, ks[page, :, slot].astype(np.int64) - 127 - 6), 32, axis=-1)
    assert np.all(np.abs(got - want)[big] <= (0.125 + 2.0 ** -16) * np.abs(want)[big])


def test_append_reports_bad_metadata(fs):
    """A length too short for its rows and a page id out of range are reported,
    not followed; the other sequences are appended."""
    bt = Batch([2, 3, 4], [20, 20, 20], 2, 16, 6)
    good, _ = _append(fs, bt, False, 0, False)
    bt.lens[1] = 2
    got, status = _append(fs, bt, False, 0, False)
    assert status >> 16 == (fs.ERR_INVALID_ARG << 8 | 1) and status & 0xFFFF == 1
    for x, y in zip(good, got):
        page, slot = bt.table[0, 1], [4, 5]
        assert np.array_equal(x[page][:, slot], y[page][:, slot])
    bt.lens[1] = 23
    bt.table[1, 1] = bt.pages
    _, status = _append(fs, bt, False, 0, False)
    assert status >> 16 == (fs.ERR_INVALID_ARG << 8 | 2) and status & 0xFFFF == 1
    bt.table[1, 1] = -5
    _, status = _append(fs, bt, False, 0, False)
    assert status >> 16 == (fs.ERR_INVALID_ARG << 8 | 2)


def test_append_of_zeros_and_extremes(fs):
    """All-zero blocks (scale byte 0, codes 0) and the largest and smallest bf16."""
    bt = Batch([6], [3], 2, 16, 8)
    bt.k[:] = 0
    bt.v[0], bt.v[1], bt.v[2] = 0x8000, 0x7F7F, 0x0001
    (kc, ks, vc, vs), status = _append(fs, bt, False, 0, False)
    b, place, page, slot = bt.where()
    assert status == 0 and not ks[page, :, slot].any() and not kc[page, :, slot].any()
    c, s = oracle.quantize_bf16(bt.v.reshape(-1, 128))
    assert np.array_equal(vc[page, :, slot].reshape(-1, 128), c) and np.array_equal(vs[page, :, slot].reshape(-1, 4), s)
