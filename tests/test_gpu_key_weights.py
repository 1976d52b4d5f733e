"""Key weights on the GPU against float64 over the dequantized cache.

Tolerance of a key's weight, the sum of p = exp(s - lse) over rows: each p is off by a factor of
d + 2^-21 + 2^-22 (|s| + |lse|) (the score's accumulator, cut at each of D / 16 steps, twice for pairs, and
subnormal low parts as in chunk_cases.py; the exponential; the rounding of the exponent's terms to float32),
the sum by (64 + row tiles) 2^-24 of itself (64 additions of pairs a tile, then the tiles), and keep * old by 2^-23.
"""
import numpy as np
import pytest

from oracle import chunked

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from chunk_cases import PAIRS, Chunk, dev     # noqa: E402


@pytest.fixture(scope="module")
def memra():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from decode_attention_block_memra_gb300 import _build
    _build.build()
    import decode_attention_block_memra_gb300 as m
    m.lib()
    return m


class Weights(Chunk):
    def __init__(self, *a, stride=0, **kw):
        super().__init__(*a, **kw)
        rng = np.random.default_rng(7)
        self.old = rng.random((len(self.new), self.Hkv, stride or max(max(self.lens), 1))).astype(np.float32)
        self.weights = dev(self.old)
        lse = np.full((len(self.buf), self.Hq), np.nan, np.float32)       # (rows of no sequence are not read)
        G = self.Hq // self.Hkv
        for b, n in enumerate(self.new):
            for h in range(self.Hkv):
                _, k, _ = self.keys(b, h)
                s = chunked.logits(self.rows_of(b)[:, h * G:(h + 1) * G], k[:, None], chunked.chunk_sees(n, self.lens[b]),
                                   self.D ** -0.5)
                lse[self.starts[b]:self.starts[b + 1], h * G:(h + 1) * G] = chunked.logits_lse(s)
        self.lse_in = lse

    def rows_of(self, b):
        return self.q[self.starts[b]:self.starts[b + 1]]

    def call(self, keep=1.0, **kw):
        a = dict(q=self.buf[:, :self.Hq], lse=dev(self.lse_in), cu_seqlens=dev(self.starts), page_table=dev(self.table),
                 seq_lens=dev(np.array(self.lens, np.int32)), max_seq_len=max(self.lens), weights=self.weights, keep=keep)
        self.memra.key_weights(self.cache, **{**a, **kw})
        return self.memra.read_status(self.cache)

    def check(self, keep, hidden=None, sequences=None):
        got, G = self.weights.cpu().numpy().astype(np.float64), self.Hq // self.Hkv
        worst = 0.0
        for b in range(len(self.new)) if sequences is None else sequences:
            T, n = self.lens[b], self.new[b]
            assert np.array_equal(got[b, :, T:], self.old[b, :, T:])
            if n == 0:
                assert np.array_equal(got[b], self.old[b])
                continue
            for h in range(self.Hkv):
                _, k, _ = self.keys(b, h)
                q = self.rows_of(b)[:, h * G:(h + 1) * G].astype(np.float64)
                sees = chunked.chunk_sees(n, T)
                if hidden is not None:
                    sees = sees & ~hidden[b]
                s = chunked.logits(q, k[:, None], sees, self.D ** -0.5)
                lse = self.lse_in[self.starts[b]:self.starts[b + 1], h * G:(h + 1) * G].astype(np.float64)
                p = np.exp(s - lse.T[..., None])
                d = np.einsum("ngd,td->gnt", np.abs(q), np.abs(k)) * self.D ** -0.5 * 2.0 ** -23 * (self.D / 8)
                d += np.abs(q).sum(-1).T[..., None] * self.D ** -0.5 * 2.0 ** -24
                e = p * (d + 2.0 ** -21 + 2.0 ** -22 * (np.abs(np.where(np.isfinite(s), s, 0)) + np.abs(lse.T[..., None])))
                total = p.sum((0, 1))
                old = keep * self.old[b, h, :T].astype(np.float64) if keep else 0.0
                tol = 1.05 * e.sum((0, 1)) + (64 + n * G / 32 + 1) * 2.0 ** -24 * total + 2.0 ** -23 * np.abs(old + total) + 1e-37
                err = np.abs(got[b, h, :T] - (old + total))
                assert (err <= tol).all(), f"sequence {b} head {h}: {(err / tol).max()} of the tolerance"
                worst = max(worst, float((err / tol).max()))
        return worst


@pytest.mark.parametrize("kf,vf", PAIRS[:4])
@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("keep", [1.0, 0.0, 0.75])
def test_formats_and_ragged_chunks(memra, kf, vf, D, keep):
    c = Weights(memra, kf, vf, D, 8, 2, [33, 1, 200, 0, 5, 1], [100, 700, 3, 50, 0, 1500], pad=3, seed=D)
    assert c.call(keep) == 0
    c.check(keep)


@pytest.mark.parametrize("new,past", [([1], [0]), ([1], [15]), ([1], [127]), ([1], [128]), ([17], [0]), ([64], [64]), ([128], [1])])
@pytest.mark.parametrize("D", [128, 256])
def test_small(memra, new, past, D):
    c = Weights(memra, "q8_0", "q5_1", D, 8, 2, new, past)
    assert c.call() == 0
    c.check(1.0)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (5, 1), (4, 4), (12, 4), (40, 8), (128, 1), (96, 1), (65, 1), (192, 2), (3, 3)])
@pytest.mark.parametrize("D", [128, 256])
def test_head_layouts(memra, Hq, Hkv, D):
    c = Weights(memra, "q8_0", "q4_0", D, Hq, Hkv, [3, 40, 1], [90, 10, 333], seed=Hq)
    assert c.call(0.5) == 0
    c.check(0.5)


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("new,past", [([1], [9000]), ([300], [2000]), ([1, 700], [20000, 100]), ([1500], [0])])
def test_long_contexts_and_long_chunks(memra, D, new, past):
    c = Weights(memra, "q8_0", "q5_1", D, 4, 1, new, past, seed=1)
    assert c.call() == 0
    c.check(1.0)


def test_many_sequences(memra):
    rng = np.random.default_rng(3)
    new = [int(x) for x in rng.integers(0, 4, 150)]
    past = [int(x) for x in rng.integers(0, 400, 150)]
    c = Weights(memra, "fp8", "fp8", 128, 8, 2, new, past, pad=1, stride=500)
    assert c.call() == 0
    c.check(1.0)


def test_keep_zero_overwrites_what_was_not_written(memra):
    c = Weights(memra, "q8_0", "q5_1", 128, 8, 2, [5], [200], stride=300)
    c.weights.fill_(float("nan"))
    assert c.call(0.0) == 0
    assert torch.isnan(c.weights[..., 205:]).all()
    c.weights[..., 205:] = dev(c.old[..., 205:])
    c.check(0.0)


def test_weights_of_a_row_sum_to_one(memra):
    c = Weights(memra, "q8_0", "q5_1", 128, 32, 4, [40], [3000])
    c.memra.chunk_attn(c.cache, **{**c.args(), "lse": c.lse})
    assert c.call(0.0, lse=c.lse) == 0
    assert (c.weights.sum(-1) - 40 * 8).abs().max() <= 40 * 8 * 1e-5


def test_strided_queries(memra):
    c = Weights(memra, "fp8", "q4_0", 128, 8, 2, [30, 2], [40, 99], stride_heads=4)
    assert c.call() == 0
    c.check(1.0)


def test_same_call_same_bytes_and_adds_up(memra):
    c = Weights(memra, "q8_0", "q5_1", 128, 32, 4, [200, 1, 1], [1000, 4000, 100])
    c.call(0.0)
    once = c.weights.clone()
    c.call(0.0)
    assert torch.equal(c.weights[0, :, :1200], once[0, :, :1200])
    c.call(1.0)
    assert torch.allclose(c.weights[1, :, :4001], 2 * once[1, :, :4001], rtol=1e-6, atol=0)


def test_bad_pages_collect_nothing(memra):
    c = Weights(memra, "q8_0", "q5_1", 128, 8, 2, [30, 2], [200, 90])
    table = c.table.copy()
    table[0, 3], table[1, 0] = -1, c.cache.num_pages
    assert c.call(page_table=dev(table)) == memra.DEVERR_BAD_PAGE
    hidden = [np.zeros(T, bool) for T in c.lens]
    hidden[0][48:64] = hidden[1][:16] = True
    c.check(1.0, hidden)


def test_bad_lengths(memra):
    M = memra
    c = Weights(memra, "q8_0", "q5_1", 128, 8, 2, [30, 20, 5], [200, 90, 60])
    for lens in ([230, 8, 65], [230, -5, 65], [230, 0, 65], [230, 2 ** 31 - 1, 65]):
        c.weights.copy_(dev(c.old))
        assert c.call(seq_lens=dev(np.array(lens, np.int32))) & M.DEVERR_BAD_SEQ_LEN
        c.check(1.0, sequences=[0, 2])
    for starts in ([0, 30, 50, 56], [-3, 30, 50, 55], [0, 30, 2 ** 31 - 1, 55], [0, 30, 10, 55]):
        assert c.call(cu_seqlens=dev(np.array(starts, np.int32))) & M.DEVERR_BAD_SEQ_LEN


def test_empty_calls(memra):
    c = Weights(memra, "q8_0", "q5_1", 128, 8, 2, [0, 0], [40, 0], pad=2)
    assert c.call() == 0
    c.check(1.0)


def test_captured_and_replayed(memra):
    c = Weights(memra, "q8_0", "q5_1", 128, 32, 4, [20, 1, 1], [3000, 4000, 100])
    a = dict(q=c.buf, lse=dev(c.lse_in), cu_seqlens=dev(c.starts), page_table=dev(c.table),
             seq_lens=dev(np.array(c.lens, np.int32)), max_seq_len=max(c.lens), weights=c.weights)
    memra.key_weights(c.cache, **a)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        memra.key_weights(c.cache, **a)
    c.weights.copy_(dev(c.old))
    graph.replay()
    assert memra.read_status(c.cache) == 0
    c.check(1.0)


@pytest.mark.parametrize("kf,D", [("q8_0", 128), ("fp8", 128), ("q8_0", 256), ("nvfp4", 256)])
def test_a_chunk_among_many_single_tokens(memra, kf, D):
    """On average few rows a sequence, so that row tiles are small; one sequence has more than the ring and the kept log-sum-exps hold."""
    c = Weights(memra, kf, "q5_1", D, 8, 1, [1] * 31 + [140] + [1] * 32, [100] * 31 + [300] + [20] * 32, seed=D)
    assert c.call(0.5) == 0
    c.check(0.5)


def test_thousands_of_calls_in_a_row(memra):
    cases = [Weights(memra, kf, "q5_1", D, 8, 2, [70, 1, 9], [500, 1200, 0], seed=D)
             for D in (128, 256) for kf in ("q8_0", "fp8")]
    args, want = [], []
    for c in cases:
        assert c.call(0.0) == 0
        c.check(0.0)
        want.append(c.weights.clone())
        args.append(dict(q=c.buf, lse=dev(c.lse_in), cu_seqlens=dev(c.starts), page_table=dev(c.table),
                         seq_lens=dev(np.array(c.lens, np.int32)), max_seq_len=max(c.lens), weights=c.weights, keep=0.0))
    for _ in range(1500):
        for c, a in zip(cases, args):
            memra.key_weights(c.cache, **a)
    for c, w in zip(cases, want):
        assert memra.read_status(c.cache) == 0 and torch.equal(c.weights, w)


def test_refusals_of_the_binding(memra):
    c = Weights(memra, "q8_0", "q5_1", 128, 8, 2, [30, 2], [40, 99])
    for bad in (dict(q=c.buf.float()), dict(lse=c.lse.half()), dict(lse=c.lse[:5]), dict(weights=c.weights[:, :1]),
                dict(weights=c.weights.double()), dict(max_seq_len=102), dict(keep=float("nan")), dict(sm_scale=0.0),
                dict(cu_seqlens=dev(c.starts).long()), dict(seq_lens=dev(c.starts)[:1]), dict(page_table=dev(c.table).long()),
                dict(weights=c.weights.cpu()), dict(max_seq_len=-1)):
        with pytest.raises(memra.MemraError):
            c.call(**bad)
    assert c.call() == 0
    c.check(1.0)


@pytest.mark.parametrize("kf,D", [("q8_0", 128), ("fp8", 128), ("q8_0", 256), ("nvfp4", 256)])
@pytest.mark.parametrize("new,past", [
    ([40, 1, 300], [3000, 4000, 100]),       # large row tiles; log-sum-exps kept for a run, and not
    ([1] * 6, [3000, 5000, 700, 4000, 1, 900]),                                       # small ones
    ([1] * 15 + [140], [300] * 15 + [2000]),
])
@pytest.mark.parametrize("first", [True, False])
def test_a_wait_that_runs_out(memra, kf, D, new, past, first):
    """The copies of CTA 0's first chunk are declared 16 bytes too long: the keys of its share become NaN, the others keep their bytes."""
    import time
    if not first:                            # CTA 0 begins in the longest chunk
        new, past = new[::-1], past[::-1]
    c = Weights(memra, kf, "q5_1", D, 8, 2, new, past, stride=max(n + p for n, p in zip(new, past)) + 7)
    assert c.call(0.5) == 0
    c.check(0.5)
    good, pool = c.weights.clone(), c.cache.k_pool.clone()
    c.weights.copy_(dev(c.old))
    begin = time.monotonic()
    memra.testing_key_weights_short_page(
        c.cache, c.buf, dev(c.lse_in), dev(c.starts), dev(c.table), dev(np.array(c.lens, np.int32)), max(c.lens), c.weights, 0.5)
    assert memra.read_status(c.cache) == memra.DEVERR_TIMEOUT
    assert time.monotonic() - begin < 20
    nan = torch.isnan(c.weights)
    assert nan[0, 0, 0] and not nan.all(-1).all()
    # whole tiles of keys, and nothing behind a sequence's last
    for b, T in enumerate(c.lens):
        assert not nan[b, :, T:].any()
        for h in range(2):
            x = nan[b, h, :T].cpu().numpy()
            assert all(x[lo:lo + 128].all() or not x[lo:lo + 128].any() for lo in range(0, T, 128))
    assert torch.equal(c.weights[~nan], good[~nan]) and torch.equal(c.cache.k_pool, pool)
    c.weights.copy_(dev(c.old))
    assert c.call(0.5) == 0
    assert torch.equal(c.weights, good)


def test_no_keys_and_no_weights(memra):
    c = Weights(memra, "fp8", "fp8", 128, 8, 2, [2, 0], [5, 0])
    empty = torch.empty(2, 2, 0, device="cuda")
    lens, starts = dev(np.zeros(2, np.int32)), dev(np.zeros(3, np.int32))
    assert c.call(weights=empty, max_seq_len=0, seq_lens=lens, cu_seqlens=starts) == 0
    # rows of a sequence without a key, and a length past the bound of 0: flagged, nothing is read or written
    assert c.call(weights=empty, max_seq_len=0, seq_lens=lens) == memra.DEVERR_BAD_SEQ_LEN
    assert c.call(weights=empty, max_seq_len=0) == memra.DEVERR_BAD_SEQ_LEN
    assert c.call() == 0
    c.check(1.0)
