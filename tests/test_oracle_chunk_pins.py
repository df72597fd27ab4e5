"""The oracle's rotation and chunk attention against closed forms and against
the decode attention that the other pins cover."""
import numpy as np

import oracle
from workloads import inputs


def test_rotation_is_a_rotation():
    """Pairs keep their length, position 0 changes nothing, and the dot
    product of two rotated vectors depends on the distance of their positions."""
    rng = np.random.default_rng(1)
    f = 1e4 ** (-np.arange(0, 64, 2) / 64)
    for inter in (False, True):
        x = rng.standard_normal((4, 2, 96))
        y = oracle.norm_rope(x, None, 0.0, [0, 1, 17, 100000], f, 64, inter)
        assert np.array_equal(y[0], x[0]) and np.array_equal(y[..., 64:], x[..., 64:])
        assert np.allclose(np.linalg.norm(y, axis=-1), np.linalg.norm(x, axis=-1), rtol=1e-14)
        a, b = x[:1], x[1:2]
        dot = [np.sum(oracle.norm_rope(a, None, 0.0, [p], f, 64, inter) * oracle.norm_rope(b, None, 0.0, [p + 5], f, 64,
                                                                                              inter)) for p in (0, 777)]
        assert abs(dot[0] - dot[1]) < 1e-9


def test_rotation_pairs_by_hand():
    x = np.zeros((1, 1, 32))
    x[0, 0, 0] = 1.0
    f = np.zeros(16)
    f[0] = np.pi / 2
    assert np.allclose(oracle.norm_rope(x, None, 0.0, [1], f, 32, False)[0, 0, 16], 1.0)
    assert np.allclose(oracle.norm_rope(x, None, 0.0, [1], f, 32, True)[0, 0, 1], 1.0)
    y = oracle.norm_rope(3.0 * np.ones((1, 1, 32)), 2.0 * np.ones(32), 0.0, [0], f, 32, True)
    assert np.allclose(y, 2.0)


def _cache(seed):
    wl = inputs.AttnWorkload("t", 3, 8, 2, 128, 16, 20, 90, seed)
    d = inputs.make_attention(wl)
    n = d["k"].shape[0]
    c = {}
    for name in ("k", "v"):
        codes, scales = oracle.quantize_bf16(d[name].reshape(-1, 128))
        c[name] = (codes.reshape(n, 2, 16, 128), scales.reshape(n, 2, 16, 4))
    return wl, d, c


def test_chunk_of_one_is_the_decode_step():
    wl, d, c = _cache(3)
    want = oracle.paged_decode_attention(d["q"], *c["k"], *c["v"], d["block_table"], d["seq_lens"], 0.1)["out"]
    q = oracle.bf16_bits_to_f64(d["q"])
    got = oracle.paged_chunk_attention(q, *c["k"], *c["v"], d["block_table"], np.arange(4), d["seq_lens"], 0, 0.1)["out"]
    assert np.allclose(got, want, rtol=1e-12, atol=1e-14)


def test_chunk_rows_are_decode_steps_of_their_own_length():
    """Row i of a chunk is the decode step of the sequence cut after its token;
    a window of 1 returns the token's own value."""
    wl, d, c = _cache(4)
    rng = np.random.default_rng(5)
    n, L = 4, int(d["seq_lens"][1])
    q = rng.standard_normal((n, 8, 128)).astype(np.float32)
    bits = inputs.bf16_bits_from_f32(q)
    q = oracle.bf16_bits_to_f64(bits)
    table, lens = d["block_table"][1:2], np.array([L])
    got = oracle.paged_chunk_attention(q, *c["k"], *c["v"], table, [0, n], lens, 0, 0.1)["out"]
    for i in range(n):
        want = oracle.paged_decode_attention(bits[i:i + 1], *c["k"], *c["v"], table, [L - n + i + 1], 0.1)["out"]
        assert np.allclose(got[i], want[0], rtol=1e-12, atol=1e-14)
    one = oracle.paged_chunk_attention(q, *c["k"], *c["v"], table, [0, n], lens, 1, 0.1)["out"]
    t = np.arange(L - n, L)
    v = oracle.dequantize(*(x[table[0, t // 16], :, t % 16].reshape(n * 2, -1) for x in c["v"])).reshape(n, 2, 128)
    assert np.array_equal(one, np.repeat(v, 4, axis=1))
