"""Chunk attention on the GPU against float64 over the dequantized cache; tolerances from the roundings (chunk_cases.py)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from chunk_cases import PAIRS, Chunk, dequantized, dev     # noqa: E402


@pytest.fixture(scope="module")
def memra():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from decode_attention_block_memra_gb300 import _build
    _build.build()
    import decode_attention_block_memra_gb300 as m
    m.lib()
    return m


@pytest.mark.parametrize("new,past", [([1], [0]), ([1], [15]), ([1], [63]), ([17], [0]), ([64], [64]), ([5], [300])])
@pytest.mark.parametrize("D", [128, 256])
def test_small(memra, new, past, D):
    c = Chunk(memra, "q8_0", "q5_1", D, 8, 2, new, past)
    assert c.call() == 0
    c.check()


@pytest.mark.parametrize("kf,vf", PAIRS)
@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("lse", [False, True])
def test_formats_and_ragged_chunks(memra, kf, vf, D, lse):
    c = Chunk(memra, kf, vf, D, 8, 2, [33, 1, 200, 0, 5, 1], [100, 700, 3, 50, 0, 1500], pad=3, seed=D)
    assert c.call(lse) == 0
    c.check(lse)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (5, 1), (4, 4), (12, 4), (40, 8), (128, 1), (96, 2), (3, 3)])
@pytest.mark.parametrize("D", [128, 256])
def test_head_layouts(memra, Hq, Hkv, D):
    c = Chunk(memra, "fp8", "q4_0", D, Hq, Hkv, [3, 40, 1], [90, 10, 333], seed=Hq)
    assert c.call() == 0
    c.check()


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("new,past", [([1], [9000]), ([300], [5000]), ([1, 700], [20000, 100]), ([2000], [0]), ([129], [16383])])
def test_long_contexts_are_cut_and_joined(memra, D, new, past):
    c = Chunk(memra, "q8_0", "q5_1", D, 4, 1, new, past, seed=1)
    assert c.call() == 0
    c.check()


def test_many_sequences(memra):
    rng = np.random.default_rng(3)
    new = [int(x) for x in rng.integers(0, 4, 150)]
    past = [int(x) for x in rng.integers(0, 400, 150)]
    c = Chunk(memra, "fp8", "fp8", 128, 8, 2, new, past, pad=1)
    assert c.call() == 0
    c.check()


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("window", [1, 5, 16, 63, 64, 65, 300])
def test_windows_over_rings(memra, D, window):
    c = Chunk(memra, "q8_0", "q5_1", D, 8, 2, [40, 1, 130, 7], [1000, 2000, 0, 3], window=window)
    assert c.call() == 0
    c.check()
    # a table of all pages is a ring that never wraps
    c = Chunk(memra, "fp8", "fp8", D, 8, 2, [40, 1], [300, 200], window=window, extra_columns=30)
    assert c.call() == 0
    c.check()


def test_pages_before_the_window_need_not_exist(memra):
    c = Chunk(memra, "q8_0", "q5_1", 128, 8, 2, [20], [1000], window=50, extra_columns=80)
    first = (1000 - 50 + 1) // 16
    gone = [p % c.table.shape[1] for p in range(0, first)]
    c.table[0, gone] = -1
    assert c.call() == 0
    c.check()


def test_strided_queries_and_scale(memra):
    c = Chunk(memra, "q8_0", "q5_1", 128, 8, 2, [30, 2], [40, 99], stride_heads=4)
    assert c.call() == 0
    c.check()
    # keys a thousand times smaller under queries a thousand times larger; and the reverse
    for gain in (1000.0, 0.001):
        c = Chunk(memra, "q8_0", "q5_1", 128, 8, 2, [30, 2], [40, 99], k_gain=1 / gain, q_gain=gain)
        assert c.call() == 0
        c.check()


def test_peaked_rows(memra):
    # scores of up to 100: one key has nearly all the weight, and which one changes along the keys
    c = Chunk(memra, "fp8", "fp8", 128, 8, 2, [60, 3], [900, 4000], q_gain=10.0)
    assert c.call() == 0
    c.check()


def test_large_values(memra):
    c = Chunk(memra, "q8_0", "q5_1", 128, 4, 2, [20], [100],
              v_of=lambda *s: np.random.default_rng(0).choice([-60000.0, 60000.0, 1.0], s))
    assert c.call() == 0
    c.check()


def test_long_sums(memra):
    """Each CTA takes over 7,680 keys of a block: its sums are joined in float32."""
    for new in ([1], [130]):
        c = Chunk(memra, "fp8", "q4_0", 128, 160, 160, new, [16384 - new[0]], fill=False,
                  v_of=lambda *s: 1 + np.random.default_rng(1).random(s))
        c.buf.mul_(0.1)
        c.q = c.buf.cpu().numpy()[:, :160]
        assert c.call() == 0
        c.check(heads=[0, 1, 77, 159])


def test_long_sums_at_head_dim_256(memra):
    c = Chunk(memra, "fp8", "fp8", 256, 160, 160, [2], [16382], fill=False, v_of=lambda *s: 1 + np.random.default_rng(1).random(s))
    assert c.call() == 0
    c.check(heads=[0, 80, 159])


def test_the_longest_context_means(memra):
    """Queries of zeros: the mean of V over 262,144 keys, all of one sign."""
    c = Chunk(memra, "q8_0", "q5_1", 128, 8, 1, [3], [262141], q_gain=0.0, fill=False,
              v_of=lambda *s: 1 + np.random.default_rng(1).random(s))
    assert c.call() == 0
    c.check()


def test_same_call_same_bytes(memra):
    c = Chunk(memra, "q8_0", "q5_1", 128, 32, 4, [200, 1, 1], [3000, 4000, 100])
    c.call()
    first, first_lse = c.out.clone(), c.lse.clone()
    c.ws.fill_(0)
    c.out.fill_(-7)
    c.call()
    assert torch.equal(c.out, first) and torch.equal(c.lse, first_lse)


def test_agrees_with_decode(memra):
    c = Chunk(memra, "q8_0", "q5_1", 128, 8, 2, [4, 4], [700, 3000])
    c.call()
    out = torch.empty(2, 4, 8, 128, dtype=torch.float16, device="cuda")
    ws = torch.empty(memra.decode_attn_workspace_bytes(2, 4, 8, 128, 3004), dtype=torch.uint8, device="cuda")
    memra.decode_attn(c.cache, c.buf.view(2, 4, 8, 128), dev(c.table), dev(np.array(c.lens, np.int32)), 3004, out, ws)
    assert (out.view(8, 8, 128).float() - c.out.float()).abs().max() <= 2e-3


def test_not_finite_queries_and_keys(memra):
    c = Chunk(memra, "fp8", "fp8", 128, 4, 1, [40, 3], [100, 50])
    c.buf[5, 2, 7] = float("nan")
    c.buf[6, 1, 0] = float("inf")
    # the key at position 120 of the first sequence: an fp8 NaN in its row
    pages = c.cache.k_pool.view(-1, 1, 2048)
    slot = c.table[0, 120 // 16]
    from oracle import layout, quant
    row = quant.quantize_rows(c.rows[0][1][120:121, 0], "fp8", c.scales[0])
    seg = np.zeros((1, 1, 2048), np.uint8)
    layout.write_rows(seg, "k", row, np.array([120 % 16]), 0, 128)
    at = int(np.nonzero(seg[0, 0])[0][0])
    pages[int(slot), 0, at] = 0x7F
    assert c.call() == 0
    nan = torch.isnan(c.out).any(-1).cpu().numpy()
    want = np.zeros((43, 4), bool)
    want[5, 2] = want[6, 1] = True
    want[20:40] = True                       # tokens from position 120 on
    assert np.array_equal(nan, want) and np.array_equal(torch.isnan(c.lse).cpu().numpy(), want)
    whole = c.out.cpu().numpy().astype(np.float64)
    out, tol, _, _ = c.expected(1, 0)
    assert (np.abs(whole[40:] - out) <= tol).all()


def test_bad_pages_are_left_out(memra):
    c = Chunk(memra, "q8_0", "q5_1", 128, 8, 2, [30, 2], [200, 90])
    table = c.table.copy()
    table[0, 3], table[1, 0] = -1, c.cache.num_pages
    assert c.call(page_table=dev(table)) == memra.DEVERR_BAD_PAGE
    got = c.out.cpu().numpy().astype(np.float64)
    from oracle import attention, chunked
    for b, page in ((0, 3), (1, 0)):
        sees = chunked.chunk_sees(c.new[b], c.lens[b])
        sees[:, 16 * page:16 * page + 16] = False
        for h in range(2):
            _, k, v = c.keys(b, h)
            rows = slice(c.starts[b], c.starts[b + 1])
            want = attention.masked_rows(c.q[rows, 4 * h:4 * h + 4], k[:, None], v[:, None], sees, 128 ** -0.5)
            assert np.abs(got[rows, 4 * h:4 * h + 4] - want).max() <= 2e-3


def test_bad_lengths(memra):
    M = memra
    c = Chunk(memra, "q8_0", "q5_1", 128, 8, 2, [30, 20, 5], [200, 90, 60])
    # shorter than its chunk: the rows at positions below 0 are zeros, the others see their keys
    assert c.call(seq_lens=dev(np.array([230, 8, 65], np.int32))) == M.DEVERR_BAD_SEQ_LEN
    assert not c.out[30:42].any() and torch.isinf(c.lse[30:42]).all() and c.out[42:50].any()
    c.check(sequences=[0, 2])
    for lens in ([230, -5, 65], [230, 2 ** 31 - 1, 65], [230, 0, 65]):
        assert c.call(seq_lens=dev(np.array(lens, np.int32))) & M.DEVERR_BAD_SEQ_LEN
        c.check(sequences=[0, 2])
    for starts in ([0, 30, 50, 56], [-3, 30, 50, 55], [0, 30, 2 ** 31 - 1, 55], [0, 30, 10, 55]):
        assert c.call(cu_seqlens=dev(np.array(starts, np.int32))) & M.DEVERR_BAD_SEQ_LEN
    assert c.call() == 0
    c.check()
    # a ring too small for the window
    c = Chunk(memra, "q8_0", "q5_1", 128, 8, 2, [30], [400], window=100)
    assert c.call(page_table=dev(c.table[:, :5])) == M.DEVERR_BAD_SEQ_LEN


def test_empty_calls(memra):
    c = Chunk(memra, "q8_0", "q5_1", 128, 8, 2, [0, 0], [40, 0], pad=2)
    assert c.call() == 0
    c.check()
    c = Chunk(memra, "q8_0", "q5_1", 128, 8, 2, [3], [40])
    q = c.buf[:0]
    c.memra.chunk_attn(c.cache, **{**c.args(), "q": q, "out": c.out[:0], "lse": c.lse[:0]})
    assert memra.read_status(c.cache) == 0


def test_captured_and_replayed_on_other_lengths(memra):
    c = Chunk(memra, "q8_0", "q5_1", 128, 32, 4, [200, 1, 1], [3000, 4000, 100], pad=4)
    a = c.args()
    c.call(**a)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        memra.chunk_attn(c.cache, **a)
    for new, past in (([200, 1, 1], [3000, 4000, 100]), ([3, 150, 40], [3100, 3851, 61]), ([0, 0, 1], [0, 0, 100])):
        c.new, c.past, c.lens = new, past, [n + p for n, p in zip(new, past)]
        c.starts = np.concatenate(([0], np.cumsum(new))).astype(np.int32)
        a["cu_seqlens"].copy_(dev(c.starts))
        a["seq_lens"].copy_(dev(np.array(c.lens, np.int32)))
        rows = c.rows
        c.rows = [(f, k[:T], v[:T]) for (f, k, v), T in zip(rows, c.lens)]
        c.out.fill_(-7)
        c.lse.fill_(-7)
        graph.replay()
        assert memra.read_status(c.cache) == 0
        c.check()
        c.rows = rows


def test_calls_side_by_side(memra):
    cases = [Chunk(memra, "q8_0", "q5_1", 128, 32, 4, [300, 1], [2000, 5000], seed=s) for s in range(3)]
    alone = []
    for c in cases:
        c.call()
        alone.append(c.out.clone())
        c.out.fill_(-7)
    streams = [torch.cuda.Stream() for _ in cases]
    args = [c.args() for c in cases]
    torch.cuda.synchronize()
    for _ in range(5):
        for c, a, s in zip(cases, args, streams):
            memra.chunk_attn(c.cache, **a, stream=s)
    torch.cuda.synchronize()
    for c, want in zip(cases, alone):
        assert memra.read_status(c.cache) == 0
        assert torch.equal(c.out, want)


def test_thousands_of_calls_in_a_row(memra):
    cases = [Chunk(memra, "q8_0", "q5_1", D, 8, 2, [70, 1, 9], [500, 1200, 0], seed=D) for D in (128, 256)]
    want = []
    for c in cases:
        assert c.call() == 0
        c.check()
        want.append(c.out.clone())
    args = [c.args() for c in cases]
    for _ in range(1500):
        for c, a in zip(cases, args):
            memra.chunk_attn(c.cache, **a)
    for c, w in zip(cases, want):
        assert memra.read_status(c.cache) == 0 and torch.equal(c.out, w)


def test_offsets_past_32_bits(memra):
    """Pages whose bytes lie past 4 GiB of the pools."""
    c = Chunk(memra, "q8_0", "q5_1", 128, 8, 2, [5], [100])
    n = c.cache.num_pages
    big = memra.KVCache("q8_0", "q5_1", 1_200_000, 2, 128)
    shift = 1_200_000 - n
    for src, dst, seg in ((c.cache.k_pool, big.k_pool, 2 * 2176), (c.cache.v_pool, big.v_pool, 2 * 1536)):
        dst[shift * seg:] = src
    assert shift * 2 * 2176 > 2 ** 32
    out = c.out.clone()
    a = c.args()
    a.update(out=out, page_table=dev(c.table + shift))
    memra.chunk_attn(big, **a)
    assert memra.read_status(big) == 0
    c.call()
    assert torch.equal(out, c.out)


def test_refusals_of_the_binding(memra):
    c = Chunk(memra, "q8_0", "q5_1", 128, 8, 2, [30, 2], [40, 99])
    good = c.args()
    for bad in (dict(q=good["q"].float()), dict(q=good["q"][:, :7]), dict(out=c.out[:5]), dict(out=c.out.float()),
                dict(cu_seqlens=good["cu_seqlens"].long()), dict(cu_seqlens=good["cu_seqlens"][:2]),
                dict(page_table=good["page_table"].long()), dict(seq_lens=good["seq_lens"][:1]),
                dict(lse=c.lse.half()), dict(lse=c.lse[:, :4]), dict(workspace=c.ws[:-1]), dict(workspace=None),
                dict(workspace=c.ws.cpu()), dict(sm_scale=0.0), dict(sm_scale=-1.0), dict(window=-1),
                dict(max_seq_len=-1), dict(q=good["q"].cpu())):
        with pytest.raises(memra.MemraError):
            c.call(**bad)
    assert c.call() == 0
    c.check()


@pytest.mark.parametrize("D", [128, 256])
def test_a_wait_that_runs_out(memra, D):
    """The copies of CTA 0's first chunk are declared 16 bytes too long: its rows become NaN, the others keep their bytes."""
    import time
    c = Chunk(memra, "q8_0", "q5_1", D, 8, 2, [40, 1, 300], [3000, 4000, 100])
    assert c.call() == 0
    good, good_lse = c.out.clone(), c.lse.clone()
    pools = c.cache.k_pool.clone(), c.cache.v_pool.clone()
    begin = time.monotonic()
    memra.testing_chunk_attn_short_page(c.cache, **c.args())
    assert memra.read_status(c.cache) == memra.DEVERR_TIMEOUT
    assert time.monotonic() - begin < 20
    nan = torch.isnan(c.out).all(-1)
    assert nan[0].any() and not nan.all()
    assert torch.equal(torch.isnan(c.out).any(-1), nan) and torch.equal(torch.isnan(c.lse), nan)
    assert torch.equal(c.out[~nan], good[~nan]) and torch.equal(c.lse[~nan], good_lse[~nan])
    assert torch.equal(c.cache.k_pool, pools[0]) and torch.equal(c.cache.v_pool, pools[1])
    assert c.call() == 0
    assert torch.equal(c.out, good) and torch.equal(c.lse, good_lse)


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("kf,vf", [("fp8", "fp8"), ("q8_0", "q5_1"), ("nvfp4", "nvfp4")])
@pytest.mark.parametrize("new,past", [([3, 1, 140], [0, 0, 200]), ([1], [9000]), ([2, 1], [20000, 500])])
@pytest.mark.parametrize("value", [-np.inf, np.inf])
def test_infinite_queries_whose_scores_have_one_sign(memra, kf, vf, D, new, past, value):
    """Every key is positive in the channel where a query is infinite: its scores are all -inf, or all inf."""
    c = Chunk(memra, kf, vf, D, 4, 1, new, past)
    for b, T in enumerate(c.lens):
        k = np.abs(c.rows[b][1])
        k[..., [7, D - 1]] += 1
        pos = np.arange(T)
        memra.kv_append(c.cache, dev(k), dev(c.rows[b][2]),
                        dev((c.table[b, pos // 16] * 16 + pos % 16).astype(np.int32)))
        c.rows[b] = (0, k, c.rows[b][2])
    assert c.call() == 0
    c.check()
    good, good_lse = c.out.clone(), c.lse.clone()
    want = torch.zeros(c.lse.shape, dtype=torch.bool, device="cuda")
    for t in range(sum(new)):                # (a channel of each part of a row: the last dims may lie elsewhere)
        c.buf[t, t % 4, 7 if t % 2 else D - 1] = float(value)
        want[t, t % 4] = True
    assert c.call() == 0
    assert torch.equal(c.out.isnan().all(-1), want) and torch.equal(c.lse.isnan(), want)
    assert torch.equal(c.out[~want], good[~want]) and torch.equal(c.lse[~want], good_lse[~want])


@pytest.mark.parametrize("tail", [22.5, 24.6, 25.1, 27.0, 31.0])
@pytest.mark.parametrize("kf,vf,D,T,n", [("q8_0", "q5_1", 128, 262144, 4864), ("fp8", "fp8", 128, 131072, 4864),
                                         ("fp8", "q4_0", 256, 131072, 2432)])
def test_a_dominant_key_over_a_long_even_tail(memra, kf, vf, D, T, n, tail):
    """The first key's score is `tail` log2 units above the others', whose values have one sign; blocks enough that most CTAs take all
    keys of theirs.  A row at position p is r sum(v_1 .. v_p) / (1 + p r), r = e^-s.

    Tolerance: r is off by the score's accumulator (D / 16 steps, twice for pairs) and 2^-19 for the exponential, once in the sum
    above and once below; weights by 2^-11 of themselves or 2^-32 of the first's; the accumulator's cut bits and the output's
    rounding as in Chunk.expected; the sum of weights by a rounding of 2^-24 for each 64 keys.
    """
    c = Chunk(memra, kf, vf, D, 8, 1, [n], [T - n], fill=False,
              v_of=lambda *s: (1 + np.random.default_rng(1).random(s)) * (np.arange(s[0]) > 0)[:, None, None])
    k = np.zeros((T, 1, D), np.float16)
    k[0, 0, 0] = 5.0
    for lo in range(0, T, 65536):
        pos = np.arange(lo, lo + 65536)
        memra.kv_append(c.cache, dev(k[pos]), dev(c.rows[0][2][pos]), dev((c.table[0, pos // 16] * 16 + pos % 16).astype(np.int32)))
    k0 = dequantized(k[:1, 0], kf, c.scales[0])[0, 0]
    c.buf.zero_()
    c.buf[..., 0] = float(tail * np.log(2) * D ** 0.5 / k0)
    s = float(c.buf[0, 0, 0]) * k0 * D ** -0.5
    assert c.call() == 0
    p, r = np.arange(T - n, T)[:, None], np.exp(-s)
    v = np.cumsum(dequantized(c.rows[0][2][:, 0], vf, c.scales[1]), 0)[T - n:]
    want, want_lse = r * v / (1 + p * r), s + np.log1p(p * r)
    r_off, l_off = 1.05 * s * 2.0 ** -23 * (D / 8) + 2.0 ** -19, T / 64 * 2.0 ** -24
    tol = want * (2 * r_off + l_off + 2 * 2.0 ** -11 + 960 * 2.0 ** -23) + T * 2.0 ** -32 * 2 + 2.0 ** -25
    err = np.abs(c.out.cpu().numpy().astype(np.float64) - want[:, None]) / tol[:, None]
    assert err.max() <= 1, f"{err.max()} of the tolerance"
    lse = c.lse.cpu().numpy().astype(np.float64)
    assert (np.abs(lse - want_lse) <= r_off + l_off + 2.0 ** -22 * want_lse).all()


@pytest.mark.parametrize("vf", ["q5_1", "fp8"])
@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("new,past", [([3], [700]), ([1, 200], [9000, 40])])
@pytest.mark.parametrize("k0", [200.0, 2200.0, 60000.0])
def test_scores_so_large_that_float32_has_no_digits_left(memra, vf, D, new, past, k0):
    """Scores of 2^20 to 2^29 log2 units that differ by up to 16: float32 holds them to 2^-3 .. 64 units, so that a row may weigh its keys
    anyhow, but it is a mean of them: V between 1 and 2 (to a step of its format and of fp16) gives rows between 1 and 2."""
    def some(c, b):
        T = c.lens[b]
        k = np.zeros((T, 1, D), np.float16)
        k[:, 0, 0] = k0
        k[:, 0, 32] = np.random.default_rng(b).random(T) * 16 * D ** 0.5 / 1.4427
        return k

    c = Chunk(memra, "q8_0", vf, D, 4, 1, new, past, v_of=lambda *s: 1 + np.random.default_rng(1).random(s))
    for b, T in enumerate(c.lens):
        pos = np.arange(T)
        memra.kv_append(c.cache, dev(some(c, b)), dev(c.rows[b][2]),
                        dev((c.table[b, pos // 16] * 16 + pos % 16).astype(np.int32)))
        c.rows[b] = (0, some(c, b), c.rows[b][2])
    c.buf.zero_()
    c.buf[..., 0], c.buf[..., 32] = 60000.0, 1.0
    assert c.call() == 0
    score = 60000.0 * dequantized(c.rows[0][1][:1, 0], "q8_0", 1.0)[0, 0] * D ** -0.5
    # (a row's reference is off by half a step of float32, 2^-24 of itself, the score by D / 8 of 2^-23)
    assert (c.lse - score).abs().max() <= 16 + 11 + score * (2.0 ** -22 + D / 8 * 2.0 ** -23)
    for b in range(len(new)):
        v = dequantized(c.rows[b][2][:, 0], vf, c.scales[1])
        out = c.out[c.starts[b]:c.starts[b + 1]].float().cpu().numpy()
        # (weights rounded to fp16: 2^-11; sums cut by the tensor cores: 960 * 2^-23; the output's own 2^-11)
        assert (out >= v.min(0) * (1 - 2.0 ** -9)).all() and (out <= v.max(0) * (1 + 2.0 ** -9)).all()


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("q_gain,k_gain", [(1e3, 1e3), (1e4, 2e3), (1.2e4, 1.2e4)])
def test_large_queries_and_keys_pick_one_key(memra, D, q_gain, k_gain):
    """Random scores of 10^6 to 10^8: a row is the value of its largest score."""
    c = Chunk(memra, "q8_0", "q4_0", D, 4, 2, [30, 2], [2000, 300], q_gain=q_gain, k_gain=k_gain)
    assert c.call() == 0 and torch.isfinite(c.out).all() and torch.isfinite(c.lse).all()
    picked = 0
    for b in range(2):
        T, n = c.lens[b], c.new[b]
        for h in range(2):
            _, k, v = c.keys(b, h)
            q = c.q[c.starts[b]:c.starts[b + 1], 2 * h:2 * h + 2].astype(np.float64)
            s = np.einsum("ngd,td->ngt", q, k) * D ** -0.5
            s[np.broadcast_to(~(np.arange(T) <= np.arange(T - n, T)[:, None])[:, None], s.shape)] = -np.inf
            off = np.einsum("ngd,td->ngt", np.abs(q), np.abs(k)).max(-1) * D ** -0.5 * (D / 8 + 2) * 2.0 ** -23
            two = np.sort(s, -1)[..., -2:]
            sure = two[..., 1] - two[..., 0] > 2 * off + 40        # the second weighs below 2^-57
            out = c.out[c.starts[b]:c.starts[b + 1], 2 * h:2 * h + 2].float().cpu().numpy()
            want = v[s.argmax(-1)]
            assert (np.abs(out - want)[sure] <= 2.0 ** -9 * np.abs(want[sure]) + 2.0 ** -24).all()
            picked += sure.sum()
    assert picked > 100
