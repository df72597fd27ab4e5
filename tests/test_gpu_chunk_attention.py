"""Attention of a chunk of new tokens over the paged MXFP8 cache against the
float64 oracle, and the four attention-side operators run one after another.

Tolerances, per element, with A = softmax average of |V|: the output's rounding
to bf16 (2^-8 |out|), the probabilities' (each off by 2^-8 at most in numerator
and divisor alike: 2^-8 (A + |out|)), and fp32 scores: a sum of 128 products is
off by 2^-17 of its magnitude, which moves every probability by that (with
2^-18 for the base-2 exponential and its argument), twice for numerator and
divisor.  Over a whole output the two roundings are independent and uniform:
2^-8 sqrt(2 / 3) = 3.2e-3 of the norm at most."""
import math

import numpy as np
import pytest

import oracle
from workloads import inputs
from tests._util import to_dev_u16, from_dev_bf16, bf16_bits_to_f64, rel_l2
from tests.test_gpu_norm_rope import Batch, _bits, _dev, _freq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fs():
    import mxfp8_swiglu_mlp_gb300 as fs

    return fs


def _finite_cache(bt):
    """Cache contents quantised from normal draws; slots of no token hold NaN
    codes and NaN scales."""
    for i in range(2):
        c, s = oracle.quantize_bf16(_bits(bt.rng, bt.pages * bt.Hkv * bt.P, 128, spread=0.3))
        bt.codes[i] = c.reshape(bt.codes[i].shape)
        bt.scales[i] = s.reshape(bt.scales[i].shape)
    used = np.zeros((bt.pages, bt.P), bool)
    for b in range(bt.B):
        t = np.arange(bt.lens[b])
        used[bt.table[b, t // bt.P], t % bt.P] = True
    for i in range(2):
        bt.codes[i].transpose(0, 2, 1, 3)[~used] = 0x7F
        bt.scales[i].transpose(0, 2, 1, 3)[~used] = 0xFF


class Run:
    def __init__(self, fs, bt, G, window=0, sm=None, qgap=0):
        import torch

        self.fs, self.bt, self.G, self.window = fs, bt, G, window
        self.Hq = G * bt.Hkv
        self.sm = 1 / math.sqrt(128) if sm is None else sm
        self.qbits = _bits(bt.rng, bt.T, self.Hq, 128, spread=0.3)
        rows = np.zeros((bt.T, self.Hq * 128 + qgap), np.uint16)
        rows[:, :self.Hq * 128] = self.qbits.reshape(bt.T, -1)
        self.q, self.ld = to_dev_u16(rows), rows.shape[1]
        self.cache = [_dev(x) for x in (bt.codes[0], bt.scales[0], bt.codes[1], bt.scales[1])]
        self.meta = [_dev(bt.table), _dev(bt.cu), _dev(bt.lens.astype(np.int32))]
        self.n = fs.fsops_paged_chunk_attention_workspace_bytes(bt.T, bt.B, self.Hq, bt.Hkv, 128, bt.P, bt.max_pages)
        assert self.n > 0
        self.ws = torch.zeros(self.n, dtype=torch.uint8, device="cuda")
        self.out = torch.full((bt.T, self.ld), -7.0, dtype=torch.bfloat16, device="cuda")
        torch.cuda.synchronize()

    def call(self, stream=None):
        bt = self.bt
        self.fs.fsops_mxfp8_paged_chunk_attention(
            self.q, self.ld, *self.cache, bt.pages, self.meta[0], bt.max_pages, self.meta[1], self.meta[2], self.out,
            self.ld, bt.T, bt.B, self.Hq, bt.Hkv, 128, bt.P, self.window, self.sm, self.ws, self.n, stream)

    def status(self):
        return self.fs.fsops_read_kernel_status(self.ws)

    def got(self):
        return from_dev_bf16(self.out)

    def want(self):
        bt = self.bt
        return oracle.paged_chunk_attention(bf16_bits_to_f64(self.qbits), bt.codes[0], bt.scales[0], bt.codes[1],
                                            bt.scales[1], bt.table, bt.cu, bt.lens, self.window, self.sm)


def _compare(r, bits=None, ref=None):
    bt, bits, ref = r.bt, r.got() if bits is None else bits, r.want() if ref is None else ref
    n = int(bt.cu[-1])
    got = bf16_bits_to_f64(bits[:n, :r.Hq * 128]).reshape(n, r.Hq, 128)
    out, A, mag = ref["out"][:n], ref["absv"][:n], ref["mag"][:n, :, None]
    tol = 2.0 ** -8 * np.abs(out) + (2.0 ** -8 + 2 * (2.0 ** -17 * mag + 2.0 ** -18)) * (A + np.abs(out))
    err = np.abs(got - out) - tol
    assert np.all(err <= 0), (float(err.max()), np.unravel_index(err.argmax(), err.shape))
    if n:
        assert rel_l2(got, out) <= 3.5e-3, rel_l2(got, out)
    # padding rows and the gaps between rows stay as they were
    assert np.all(bits[n:] == 0xC0E0) and np.all(bits[:, r.Hq * 128:] == 0xC0E0)


def _check(fs, new, ctx, Hkv, P, G, window=0, pad=0, seed=0, qgap=0, sm=None):
    import torch

    bt = Batch(new, ctx, Hkv, P, seed, pad)
    _finite_cache(bt)
    r = Run(fs, bt, G, window, sm, qgap)
    r.call()
    torch.cuda.synchronize()
    assert r.status() == 0
    _compare(r)
    # the counters are back at zero: a second call gives the same bits
    first = r.got()
    r.out.fill_(-7.0)
    r.call()
    torch.cuda.synchronize()
    assert r.status() == 0 and np.array_equal(first, r.got())


# single tokens at the edges of key tiles and pages
@pytest.mark.parametrize("G", [1, 4, 7])
@pytest.mark.parametrize("P", [16, 128])
def test_single_tokens(fs, P, G):
    lens = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 500]
    _check(fs, [1] * len(lens), [n - 1 for n in lens], 2, P, G, seed=P + G)


CHUNKS = [
    ([5, 0, 64, 130, 1], [0, 40, 7, 250, 300], 2, 16, 4, 3),
    ([33, 2, 200], [0, 0, 1], 1, 64, 7, 0),
    ([256, 1, 257], [128, 127, 129], 2, 32, 1, 1),
    ([3, 70], [600, 60], 3, 128, 8, 40),
    ([20, 21], [100, 0], 1, 16, 12, 0),
    ([5], [40], 1, 16, 64, 0),
    ([128], [0], 4, 64, 2, 0),
    ([0, 0, 9], [5, 0, 0], 2, 16, 3, 2),
    ([600], [700], 1, 32, 5, 0),
]


@pytest.mark.parametrize("i", range(len(CHUNKS)))
def test_chunks(fs, i):
    new, ctx, Hkv, P, G, pad = CHUNKS[i]
    _check(fs, new, ctx, Hkv, P, G, pad=pad, seed=20 + i, qgap=8 * i)


@pytest.mark.parametrize("window", [1, 2, 17, 64, 100, 128, 300, 100000])
def test_windows(fs, window):
    _check(fs, [1, 90, 300, 4], [500, 20, 260, 0], 2, 16, 3, window=window, seed=window % 97)


def test_window_skips_stale_pages(fs):
    """Page-table entries that no row's window reaches are never followed."""
    import torch

    bt = Batch([3, 50], [900, 700], 2, 16, 4)
    _finite_cache(bt)
    r = Run(fs, bt, 4, window=100)
    ref = r.want()
    for b in range(2):
        first = bt.lens[b] - bt.new[b] - 100 + 1
        bt.table[b, :first // 16] = -9
    r.meta[0].copy_(_dev(bt.table))
    r.call()
    torch.cuda.synchronize()
    assert r.status() == 0
    _compare(r, ref=ref)


def test_long_cache_split_over_blocks(fs):
    """Few rows over long caches: partial results of many splits."""
    _check(fs, [1, 3], [9000, 5003], 2, 16, 4, seed=1)
    _check(fs, [40], [12345], 1, 128, 2, seed=2)


def test_many_sequences(fs):
    """More than 32 sequences (the plan walks them in groups), empty ones among them."""
    rng = np.random.default_rng(0)
    new = [int(x) for x in rng.choice([0, 1, 1, 2, 30], 75)]
    _check(fs, new, [int(x) for x in rng.integers(0, 200, 75)], 2, 16, 2, pad=5, seed=3)


@pytest.mark.parametrize("sm", [0.0, 3.0, -0.2])
def test_softmax_scales(fs, sm):
    """Uniform weights, nearly one-hot weights (maxima that keep growing), a
    negative scale."""
    _check(fs, [70, 1], [200, 300], 2, 32, 4, sm=sm, seed=9)


def test_key_scales_far_apart(fs):
    """Keys and values whose block scales lie 2^30 apart, and zero blocks."""
    import torch

    bt = Batch([40, 2], [150, 400], 2, 16, 12)
    _finite_cache(bt)
    for i in range(2):
        s = bt.scales[i]
        fine = s != 0xFF
        s[fine] = np.clip(s[fine].astype(int) + bt.rng.choice([0, 0, 0, -30, -3, 2], int(fine.sum())), 1, 250)
        bt.codes[i][:, :, 3::7, 32:64] = np.where(bt.codes[i][:, :, 3::7, 32:64] == 0x7F, 0x7F, 0)
    r = Run(fs, bt, 4)
    r.call()
    torch.cuda.synchronize()
    assert r.status() == 0
    _compare(r)


def test_graph_replay_follows_new_lengths(fs):
    """A captured call replayed with other offsets, lengths and tables; two
    graphs that share a workspace, one after the other."""
    import torch

    bts = [Batch(n, c, 2, 16, 30 + i, p) for i, (n, c, p) in enumerate((([4, 60, 1], [90, 5, 3], 2), ([1, 1, 65], [7, 1, 41], 0)))]
    for bt in bts:
        bt.k = bt.v = None
        _finite_cache(bt)
    T = max(bt.T for bt in bts)
    for bt in bts:
        bt.T = T
    runs = [Run(fs, bt, 4) for bt in bts]
    width = max(bt.max_pages for bt in bts)
    a, b = runs
    s = torch.cuda.Stream()
    graphs = []
    for r in runs:
        r.ws = a.ws
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            r.call(stream=s)
        graphs.append(g)
    for _ in range(2):
        for r, g in zip(runs, graphs):
            r.out.fill_(-7.0)
            g.replay()
            torch.cuda.synchronize()
            assert r.status() == 0
            _compare(r)
    # the first graph with fewer tokens in the same buffers
    bt = a.bt
    bt.new, bt.lens = np.array([2, 0, 50]), np.array([94, 65, 50])
    bt.table[2, :4] = bt.table[1, :4]
    bt.cu = np.array([0, 2, 2, 52], np.int32)
    for x, y in zip(a.meta, (bt.table, bt.cu, bt.lens.astype(np.int32))):
        x.copy_(_dev(y))
    a.out.fill_(-7.0)
    graphs[0].replay()
    torch.cuda.synchronize()
    assert a.status() == 0 and width
    _compare(a)


def test_bad_metadata_is_reported(fs):
    """A chunk longer than its sequence, offsets behind the buffer and a page id
    out of range: reported, never followed; the other sequences are right."""
    import torch

    bt = Batch([4, 5, 6], [100, 50, 30], 2, 16, 40)
    _finite_cache(bt)
    for what in ("length", "table", "long", "offset"):
        r = Run(fs, bt, 4)
        ref = r.want()
        table, cu, lens = bt.table.copy(), bt.cu.copy(), bt.lens.astype(np.int32)
        if what == "length":
            lens[1] = 4
        elif what == "long":
            lens[1] = bt.max_pages * 16 + 1
        elif what == "offset":
            cu[3] = bt.T + 1
        else:
            table[1, 2] = bt.pages
        for x, y in zip(r.meta, (table, cu, lens)):
            x.copy_(_dev(y))
        r.call()
        torch.cuda.synchronize()
        word = r.status()
        assert word >> 24 == fs.ERR_INVALID_ARG and (word >> 16) & 0xFF == (2 if what == "table" else 1), hex(word)
        assert word & 0xFFFF == (2 if what == "offset" else 1)
        got = bf16_bits_to_f64(r.got()[:4, :r.Hq * 128]).reshape(4, r.Hq, 128)
        assert rel_l2(got, ref["out"][:4]) <= 3.5e-3


def test_workspace_too_small_is_refused(fs):
    bt = Batch([3], [40], 2, 16, 41)
    _finite_cache(bt)
    r = Run(fs, bt, 4)
    r.n -= 256
    with pytest.raises(fs.FsopsError) as e:
        r.call()
    assert e.value.status == fs.ERR_INVALID_ARG


def test_layer_step_by_step(fs):
    """A prompt in two chunks, then decode steps: rotation of q, append, chunk
    attention, on a side stream; the decode operator agrees with a chunk of
    one.  The cache the kernels built is what the oracle attends over."""
    import torch

    Hkv, G, P, D, R = 2, 4, 16, 128, 128
    Hq, B, MP, pages = Hkv * G, 2, 20, 40
    rng = np.random.default_rng(50)
    table = rng.permutation(pages).astype(np.int32).reshape(B, MP)
    kc, vc = (torch.full((pages, Hkv, P, D), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.full((pages, Hkv, P, D // 32), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(2))
    gam = to_dev_u16(inputs.bf16_bits_from_f32((1 + 0.1 * rng.standard_normal((2, D))).astype(np.float32)))
    f, td = _dev(_freq(R)), _dev(table)
    side = torch.cuda.Stream()
    lens = np.zeros(B, np.int64)
    width = (Hq + 2 * Hkv) * D
    for new in ([100, 37], [61, 150], [1, 1], [1, 1], [1, 0], [5, 5]):
        new = np.array(new)
        cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        T = int(cu[-1])
        pos = np.concatenate([np.arange(n) + L for n, L in zip(new, lens)]).astype(np.int32)
        lens += new
        qkv = to_dev_u16(_bits(rng, T, width, spread=0.2))
        q = torch.empty(T, Hq * D, dtype=torch.bfloat16, device="cuda")
        out = torch.full((T, Hq * D), -7.0, dtype=torch.bfloat16, device="cuda")
        n = fs.fsops_paged_chunk_attention_workspace_bytes(T, B, Hq, Hkv, D, P, MP)
        ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
        meta = [_dev(pos), _dev(cu), _dev(lens.astype(np.int32))]
        side.wait_stream(torch.cuda.current_stream())
        fs.fsops_qk_norm_rope(qkv, width, None, 0, gam[0], None, 1e-6, meta[0], (f, R, False), q, Hq * D, None, 0, T, Hq,
                              0, D, side)
        fs.fsops_mxfp8_kv_append(qkv[:, Hq * D:], width, qkv[:, (Hq + Hkv) * D:], width, gam[1], 1e-6, None, (f, R, False),
                                 kc, ks, vc, vs, pages, td, MP, meta[1], meta[2], T, B, Hkv, D, P, ws, side)
        fs.fsops_mxfp8_paged_chunk_attention(q, Hq * D, kc, ks, vc, vs, pages, td, MP, meta[1], meta[2], out, Hq * D, T, B,
                                             Hq, Hkv, D, P, 0, 1 / math.sqrt(D), ws, n, side)
        side.synchronize()
        assert fs.fsops_read_kernel_status(ws) == 0
        qf = bf16_bits_to_f64(from_dev_bf16(q)).reshape(T, Hq, D)
        ref = oracle.paged_chunk_attention(qf, *(x.cpu().numpy() for x in (kc, ks, vc, vs)), table, cu, lens, 0,
                                           1 / math.sqrt(D))["out"]
        got = bf16_bits_to_f64(from_dev_bf16(out)).reshape(T, Hq, D)
        assert rel_l2(got, ref) <= 3.5e-3
        if np.all(new == 1):
            wn = fs.fsops_paged_attention_workspace_bytes(B, Hq, Hkv, D, P, MP)
            dw = torch.zeros(wn, dtype=torch.uint8, device="cuda")
            dec = torch.empty_like(out)
            fs.fsops_mxfp8_paged_decode_attention(q, kc, ks, vc, vs, pages, td, MP, meta[2], dec, B, Hq, Hkv, D, P,
                                                  1 / math.sqrt(D), dw, wn)
            torch.cuda.synchronize()
            # each is within its own roundings of the exact result
            assert rel_l2(bf16_bits_to_f64(from_dev_bf16(dec)), got.reshape(T, -1)) <= 3.5e-3 + 2.0 ** -8
