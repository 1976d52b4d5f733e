"""Tree attention on the GPU against its definition in float64 over the oracle's dequantized cache.

Tolerance, per output element, from the arithmetic (u = 2^-11, half a step of
fp16, relative): the output's rounding u |o|; each weight's rounding to fp16,
u sum p |v| / sum p, or 2^-25 absolute for a weight below fp16's normal range
(the largest weight of a split is at least 1); the float32 scores, each K = 16
step of a product (hi and lo parts: twice head_dim / 16 of them) off by at most
2^-22 of the absolute products so far, and 2^-19 for exponentials, sums and the
merge: a relative error of twice that on every weight; and 2^-21 of the largest
value for a dequantized pair hi + lo, with its share on the scores.
"""
import numpy as np
import pytest

import workloads as W
from oracle import attention, quant

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = 2.0 ** -11
PAIRS = [(k, v) for k in W.K_FORMATS for v in W.V_FORMATS]


@pytest.fixture(scope="module")
def memra():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from decode_attention_block_memra_gb300 import _build
    _build.build()
    import decode_attention_block_memra_gb300 as m
    m.lib()
    return m


def random_tree(rng, nodes):
    """Words of a random tree: bit j of word i, node j is on node i's path from a root (i included)."""
    words = np.zeros(nodes, np.uint64)
    for i in range(nodes):
        parent = rng.integers(-1, i) if i else -1
        words[i] = np.uint64(1 << i) | (words[parent] if parent >= 0 else np.uint64(0))
    return words


def chain(nodes):
    return np.array([(1 << (i + 1)) - 1 for i in range(nodes)], np.uint64)


def reference(w, words, lens=None, missing_pages=()):
    """(o, tolerance) float64 [B, N, Hq, D] of the workload's rows under the mask words."""
    cache = attention.quantize_cache(w)
    B, N, Hq, D = w.q.shape
    G = w.group
    o, tol = np.zeros(w.q.shape), np.zeros(w.q.shape)
    for b in range(B):
        T = int(w.seq_lens[b])
        rows = attention.sequence_rows(w, b)
        key = np.arange(T) - (T - N)
        sees = np.ones((N, T), bool)
        for i in range(N):
            for j in range(N):
                sees[i, T - N + j] = bool(int(words[b, i]) >> j & 1)
        for col in missing_pages:
            sees[:, 16 * col:16 * col + 16] = False
        assert key[-1] == N - 1
        for h in range(w.n_kv_heads):
            k = quant.dequantize_rows(quant.select_rows(cache["k"][h], rows)).astype(np.float64)
            v = quant.dequantize_rows(quant.select_rows(cache["v"][h], rows)).astype(np.float64)
            q = w.q[b, :, h * G:(h + 1) * G].astype(np.float64)
            s = np.einsum("igd,td->igt", q, k) * w.sm_scale
            mass = np.einsum("igd,td->igt", np.abs(q), np.abs(k)) * w.sm_scale
            s = np.where(sees[:, None], s, -np.inf)
            top = s.max(-1, keepdims=True)
            p = np.exp(s - np.where(np.isfinite(top), top, 0))
            l = p.sum(-1, keepdims=True)
            p = np.divide(p, l, out=np.zeros_like(p), where=l > 0)
            mass = np.where(sees[:, None], mass, 0).max(-1, keepdims=True)
            step = 2 * ((D // 8 + 2) * 2.0 ** -22 * mass + 2.0 ** -21 * mass + 2.0 ** -19)
            heads = slice(h * G, (h + 1) * G)
            o[b, :, heads] = p @ v
            tol[b, :, heads] = (U * np.abs(p @ v) + (U + step) * (p @ np.abs(v)) +
                                (T * 2.0 ** -25 + 2.0 ** -21) * np.abs(v).max())
    return o, tol


def run(memra, w, words, mask_extra=None, max_seq_len=None, sm_scale=None, seed=3, sentinel=True):
    from decode_attention_block_memra_gb300.runner import upload
    dw = upload(w, fill_seed=seed)
    memra.kv_append(dw.cache, dw.step_k, dw.step_v, dw.step_slots)
    B, N, Hq, D = w.q.shape
    M = max_seq_len or w.max_seq_len
    n = memra.tree_attn_workspace_bytes(B, N, Hq, D, M)
    ws = torch.full((max(n, 16),), 0xFF, dtype=torch.uint8, device="cuda")      # NaN everywhere
    mask = torch.from_numpy(words.view(np.int64).copy()).cuda()
    dw.out.fill_(float("nan"))
    args = (dw.cache, dw.q, dw.page_table, dw.seq_lens, M, mask, dw.out, ws, sm_scale or w.sm_scale)
    memra.tree_attn(*args)
    return dw, args


def check(memra, w, words, **kw):
    dw, args = run(memra, w, words, **kw)
    assert memra.read_status(dw.cache) == 0
    want, tol = reference(w, words)
    got = dw.out.cpu().numpy().astype(np.float64)
    assert np.isfinite(got).all()
    worst = float((np.abs(got - want) / tol).max())
    assert worst <= 1, worst
    return dw, args, got


def words_for(w, seed=0, make=random_tree):
    rng = np.random.default_rng(seed)
    return np.stack([make(rng, w.q_len) for _ in range(w.batch)])


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("kf,vf", PAIRS)
def test_formats(memra, kf, vf, D):
    w = W.random_case(50 + D, batch=3, q_len=9, n_heads=16, n_kv_heads=2, head_dim=D, k_fmt=kf, v_fmt=vf,
                      ctx=(9, 1700))
    check(memra, w, words_for(w, 1))


@pytest.mark.parametrize("kf,vf", PAIRS)
def test_formats_at_two_row_tiles(memra, kf, vf):
    w = W.random_case(51, batch=2, q_len=19, n_heads=16, n_kv_heads=2, head_dim=128, k_fmt=kf, v_fmt=vf,
                      ctx=(19, 2900))
    check(memra, w, words_for(w, 3))


@pytest.mark.parametrize("T", [20, 63, 64, 65, 128, 129, 191, 193, 256, 300, 1029])
def test_length_edges_at_two_row_tiles(memra, T):
    # 160 rows; T = 20: the tree alone
    w = W.make_workload(f"e{T}", batch=1, q_len=20, n_heads=8, n_kv_heads=1, head_dim=128, k_fmt="q8_0", v_fmt="q5_1",
                        seed=T, seq_lens=[T], permute_pages=True, extra_pages=2)
    check(memra, w, words_for(w, T))


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("nodes,n_heads,n_kv_heads", [
    (1, 8, 2), (2, 4, 4), (16, 32, 4), (17, 32, 4),      # 128 rows, then two tiles
    (33, 16, 2), (64, 8, 2), (64, 16, 2),                # 264, 256 and 512 rows of a KV head
    (5, 6, 2), (13, 10, 2), (64, 3, 3), (3, 128, 1), (64, 12, 1), (64, 128, 1)])
def test_shapes(memra, nodes, n_heads, n_kv_heads, D):
    w = W.random_case(nodes * 7 + n_heads, batch=2, q_len=nodes, n_heads=n_heads, n_kv_heads=n_kv_heads, head_dim=D,
                      ctx=(nodes, 700))
    check(memra, w, words_for(w, nodes))


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("T", [4, 5, 15, 16, 17, 31, 32, 33, 63, 64, 65, 68, 127, 128, 132, 511, 512, 513, 516, 1024,
                               1027])
def test_length_edges(memra, T, D):
    # T = 4: the tree alone, no key before it
    w = W.make_workload(f"t{T}", batch=1, q_len=4, n_heads=8, n_kv_heads=1, head_dim=D, k_fmt="q8_0", v_fmt="q5_1",
                        seed=T, seq_lens=[T], permute_pages=True, extra_pages=2)
    check(memra, w, words_for(w, T))


def test_rows_that_see_nothing(memra):
    w = W.make_workload("empty", batch=2, q_len=6, n_heads=8, n_kv_heads=2, head_dim=128, k_fmt="q8_0", v_fmt="q5_1",
                        seed=1, seq_lens=[6, 40], permute_pages=True, extra_pages=2)
    words = np.zeros((2, 6), np.uint64)
    words[0, 3] = 1 << 5                     # one row of the first sequence sees one node, a later one
    dw, _, got = check(memra, w, words)
    assert (got[0, [0, 1, 2, 4, 5]] == 0).all() and (got[1] != 0).any()


@pytest.mark.parametrize("D,nodes", [(128, 9), (256, 9), (128, 40)])
@pytest.mark.parametrize("kf,vf", PAIRS)
def test_unnamed_rows_may_hold_anything(memra, kf, vf, D, nodes):
    """Rows of a padded tree that no word names, whose bytes stand for NaN."""
    w = W.random_case(60 + D, batch=2, q_len=nodes, n_heads=8, n_kv_heads=2, head_dim=D, k_fmt=kf, v_fmt=vf,
                      ctx=(nodes + 60, nodes + 90))
    words = words_for(w, 17)
    used = np.array([nodes - 4, 3])
    for b, n in enumerate(used):
        words[b, n:] = 0
        words[b, :n] &= np.uint64((1 << int(n)) - 1)
    want, tol = reference(w, words)
    dw, args = run(memra, w, words)
    unnamed = set()
    for b, n in enumerate(used):
        for t in range(int(w.seq_lens[b]) - nodes + int(n), int(w.seq_lens[b])):
            unnamed.add(int(w.page_table[b, t // 16]) * 16 + t % 16)
    keep = [i for i, s in enumerate(dw.step_slots.tolist()) if s not in unnamed]
    assert len(keep) == used.sum()
    for pool in (dw.cache.k_pool, dw.cache.v_pool):
        pool.fill_(0xFF)
    before = w.prefill_rows
    memra.kv_append(dw.cache, *(torch.from_numpy(np.ascontiguousarray(x[before])).cuda()
                                for x in (w.k_rows, w.v_rows, w.slots)))
    memra.kv_append(dw.cache, dw.step_k[keep].contiguous(), dw.step_v[keep].contiguous(),
                    dw.step_slots[keep].contiguous())
    dw.out.fill_(float("nan"))
    memra.tree_attn(*args)
    assert memra.read_status(dw.cache) == 0
    worst = float((np.abs(dw.out.cpu().numpy().astype(np.float64) - want) / tol).max())
    assert worst <= 1, worst


def test_bits_past_the_tree_are_ignored(memra):
    w = W.random_case(5, batch=2, q_len=7, n_heads=8, n_kv_heads=2, ctx=(7, 90))
    words = words_for(w, 2)
    _, _, want = check(memra, w, words)
    dw, _ = run(memra, w, words | np.uint64(0xFFFFFFFFFFFFFF80))
    assert np.array_equal(dw.out.cpu().numpy().astype(np.float64), want)


def test_a_chain_is_the_causal_verify(memra):
    w = W.random_case(6, batch=3, q_len=5, n_heads=16, n_kv_heads=4, ctx=(100, 2600))
    words = np.stack([chain(5)] * 3)
    dw, _, got = check(memra, w, words)
    out = torch.empty_like(dw.out)
    memra.decode_attn(dw.cache, dw.q, dw.page_table, dw.seq_lens, w.max_seq_len, out, dw.workspace, w.sm_scale)
    assert np.abs(out.cpu().numpy().astype(np.float64) - got).max() <= 4e-3     # 2e-3 from the definition each


@pytest.mark.parametrize("D,lens", [(128, [40000]), (256, [21000, 530]), (128, [9000, 70, 2049])])
def test_many_splits(memra, D, lens):
    w = W.make_workload("long", batch=len(lens), q_len=4, n_heads=8, n_kv_heads=2, head_dim=D, k_fmt="q8_0",
                        v_fmt="q5_1", seed=7, seq_lens=lens, permute_pages=True)
    check(memra, w, words_for(w, 3))


def test_splits_at_their_largest(memra):
    # 16 KV heads x 16 row tiles leave a wave one split: more than 2 x 7,680 keys make three
    w = W.make_workload("wide", batch=1, q_len=64, n_heads=16 * 32, n_kv_heads=16, head_dim=128, k_fmt="fp8",
                        v_fmt="fp8", seed=8, seq_lens=[8192 + 8192 + 70])
    words = words_for(w, 4)
    dw, args = run(memra, w, words)
    assert memra.read_status(dw.cache) == 0
    got = dw.out.cpu().numpy().astype(np.float64)
    # two KV heads of the sixteen, against the definition
    for h in (0, 15):
        one = W.Workload(**{**w.__dict__})
        one.n_heads, one.n_kv_heads = 32, 1
        one.q = w.q[:, :, 32 * h:32 * h + 32]
        one.k_rows, one.v_rows = w.k_rows[:, h:h + 1], w.v_rows[:, h:h + 1]
        want, tol = reference(one, words)
        assert (np.abs(got[:, :, 32 * h:32 * h + 32] - want) <= tol).all()


@pytest.mark.parametrize("kf,vf", [("q8_0", "q5_1"), ("fp8", "q4_0"), ("nvfp4", "nvfp4")])
def test_long_sums_keep_their_precision(memra, kf, vf):
    """Means over 15,000 keys in one split are a hundredth of the values: what nearly cancels in the sums
    must not cost precision.  Relative in the 2-norm the output's rounding and the weights' (independent of
    the values' signs) are at most u each."""
    w = W.make_workload("long_sums", batch=1, q_len=64, n_heads=16 * 32, n_kv_heads=16, head_dim=128, k_fmt=kf,
                        v_fmt=vf, seed=19, seq_lens=[15_000])
    w.q = (w.q.astype(np.float32) * 0.5).astype(np.float16)
    words = words_for(w, 19)
    dw, _ = run(memra, w, words)
    assert memra.read_status(dw.cache) == 0
    got = dw.out.cpu().numpy().astype(np.float64)
    one = W.Workload(**{**w.__dict__})
    one.n_heads, one.n_kv_heads = 32, 1
    one.q, one.k_rows, one.v_rows = w.q[:, :, 64:96], w.k_rows[:, 2:3], w.v_rows[:, 2:3]
    want, _ = reference(one, words)
    err = np.linalg.norm(got[:, :, 64:96] - want) / np.linalg.norm(want)
    assert err <= 2 * U, err


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("kf,vf", [("q8_0", "q5_1"), ("fp8", "q4_0"), ("fp8", "fp8"), ("nvfp4", "nvfp4")])
def test_long_means_keep_their_precision(memra, kf, vf, D):
    """Equal scores over 15,000 keys, in splits of up to 7,680: every weight is 1 exactly, every row a mean.

    Left are the output's rounding (half a step of fp16 at its value, which
    V^'s rounding can bring above 2) and the float32 sums: 480 steps of 16 keys in
    a split, two products each where V^ is a pair, every one off by at most
    2^-21 of the sum so far, half of its end on average: 2^-12 relative.
    """
    w = W.make_workload("long_means", batch=1, q_len=64, n_heads=16 * 4, n_kv_heads=16, head_dim=D, k_fmt=kf,
                        v_fmt=vf, seed=20, seq_lens=[15_000])
    w.q[:] = 0
    rng = np.random.default_rng(20)
    w.v_rows[:] = (1.9 + 0.09 * rng.random(w.v_rows.shape)).astype(np.float16)
    words = np.stack([chain(64)])
    dw, _ = run(memra, w, words)
    assert memra.read_status(dw.cache) == 0
    got = dw.out.cpu().numpy().astype(np.float64)
    rows = attention.sequence_rows(w, 0)
    for h in (0, 15):
        cache = quant.quantize_rows(w.v_rows[:, h], vf, w.v_scale)
        v = quant.dequantize_rows(quant.select_rows(cache, rows)).astype(np.float64)
        want = np.cumsum(v, 0)[-64:] / np.arange(len(v) - 63, len(v) + 1)[:, None]
        tol = np.spacing(want.astype(np.float16)).astype(np.float64) / 2 + 2.0 ** -12 * want
        assert (np.abs(got[0, :, 4 * h:4 * h + 4] - want[:, None]) <= tol[:, None]).all()


@pytest.mark.parametrize("D", [128, 256])
def test_alone_and_batched(memra, D):
    """A sequence alone (cut into other splits) within the tolerance; the same call twice, the same bytes."""
    w = W.random_case(9, batch=3, q_len=6, n_heads=16, n_kv_heads=2, head_dim=D, ctx=(300, 3000))
    words = words_for(w, 5)
    dw, args, got = check(memra, w, words)
    want, tol = reference(w, words)
    again = torch.empty_like(dw.out)
    memra.tree_attn(*args[:6], again, *args[7:])
    assert torch.equal(again, dw.out)
    for b in range(3):
        out = torch.empty_like(dw.out[b:b + 1])
        memra.tree_attn(dw.cache, dw.q[b:b + 1], dw.page_table[b:b + 1].contiguous(), dw.seq_lens[b:b + 1].clone(),
                        int(w.seq_lens[b]), args[5][b:b + 1].contiguous(), out, args[7], w.sm_scale)
        assert (np.abs(out[0].cpu().numpy().astype(np.float64) - want[b]) <= tol[b]).all()


@pytest.mark.parametrize("batch,n_heads,n_kv_heads", [(33, 8, 2), (70, 4, 4), (400, 8, 4)])
def test_many_sequences(memra, batch, n_heads, n_kv_heads):
    # more than a warp's worth of lengths, empty ones among them; the last fills the GPU without any cut
    rng = np.random.default_rng(batch)
    lens = rng.integers(3, 200, batch)
    lens[::7] = 3
    w = W.make_workload("many", batch=batch, q_len=3, n_heads=n_heads, n_kv_heads=n_kv_heads, head_dim=128,
                        k_fmt="q8_0", v_fmt="q5_1", seed=batch, seq_lens=lens, permute_pages=True)
    check(memra, w, words_for(w, batch), max_seq_len=3000 if batch > 100 else None)


def test_peaked_scores_and_a_negative_scale(memra):
    w = W.random_case(10, batch=2, q_len=8, n_heads=16, n_kv_heads=2, ctx=(500, 1500))
    w.q = (w.q.astype(np.float32) * 40).astype(np.float16)
    check(memra, w, words_for(w, 6))
    w2 = W.random_case(11, batch=2, q_len=8, n_heads=16, n_kv_heads=2, ctx=(500, 1500))
    words = words_for(w2, 7)
    dw, _ = run(memra, w2, words, sm_scale=-w2.sm_scale)
    w2.q = -w2.q
    want, tol = reference(w2, words)
    assert (np.abs(dw.out.cpu().numpy().astype(np.float64) - want) <= tol).all()


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("D,nodes,ctx", [(128, 9, 200), (128, 9, 2600), (128, 40, 200), (128, 40, 2600), (256, 9, 200),
                                         (256, 9, 2600)])
def test_a_query_that_is_not_finite_makes_its_row_nan(memra, D, nodes, ctx, value):
    # one split, then several; no other row changes
    w = W.random_case(70 + D, batch=2, q_len=nodes, n_heads=8, n_kv_heads=2, head_dim=D, ctx=(ctx - 30, ctx))
    dw, args, _ = check(memra, w, words_for(w, 21))
    want = dw.out.clone()
    for b, i, h in ((0, 3, 2), (1, nodes - 1, 7)):
        dw.q[b, i, h, 5] = value
        want[b, i, h] = float("nan")
    memra.tree_attn(*args)
    assert memra.read_status(dw.cache) == 0
    assert torch.equal(torch.isnan(dw.out), torch.isnan(want))
    assert torch.equal(dw.out.nan_to_num(7.0), want.nan_to_num(7.0))


@pytest.mark.parametrize("D,nodes,ctx", [(128, 9, 200), (128, 9, 2600), (128, 40, 2600), (256, 9, 200), (256, 9, 2600)])
def test_a_key_that_is_nan_reaches_the_rows_that_see_it(memra, D, nodes, ctx):
    """fp8's NaN code in one key of one KV head: before the tree (every row sees it), then in the tree's row of a node."""
    w = W.random_case(71 + D, batch=2, q_len=nodes, n_heads=8, n_kv_heads=2, head_dim=D, k_fmt="fp8", v_fmt="q5_1",
                      ctx=(ctx - 30, ctx))
    words = words_for(w, 22)
    dw, args, _ = check(memra, w, words)
    clean, h, group, node = dw.out.clone(), 1, 4, nodes // 2
    pool = dw.cache.k_pool.view(w.num_pages, 2, -1)
    T = int(w.seq_lens[1])
    for pos, sees in ((37, np.ones(nodes, bool)), (T - nodes + node, (words[1] >> np.uint64(node)) & np.uint64(1) != 0)):
        page, t = int(w.page_table[1, pos // 16]), pos % 16
        byte = ((t // 8 * (D // 64)) * 32 + 4 * (t % 8)) * 16               # element 0 of token t
        held = pool[page, h, byte].clone()
        pool[page, h, byte] = 0x7F
        memra.tree_attn(*args)
        pool[page, h, byte] = held
        want = clean.clone()
        want[1, torch.from_numpy(sees).cuda(), h * group:(h + 1) * group] = float("nan")
        assert memra.read_status(dw.cache) == 0
        assert torch.equal(torch.isnan(dw.out), torch.isnan(want))
        assert torch.equal(dw.out.nan_to_num(7.0), want.nan_to_num(7.0))


@pytest.mark.parametrize("D,nodes,ctx", [(128, 7, 200), (128, 40, 2600), (256, 7, 2600)])
def test_a_scale_of_zero(memra, D, nodes, ctx):
    # means over the keys that a row sees; zeros where it sees none
    w = W.random_case(72 + D, batch=2, q_len=nodes, n_heads=8, n_kv_heads=2, head_dim=D, ctx=(ctx - 30, ctx))
    w2 = W.random_case(73 + D, batch=1, q_len=nodes, n_heads=8, n_kv_heads=2, head_dim=D, ctx=(nodes, nodes))
    for x, seed in ((w, 23), (w2, 24)):
        words = words_for(x, seed)
        if x is w2:
            words[0, ::2] = 0                            # the tree alone: these rows see nothing
        dw, args = run(memra, x, words)
        dw.out.fill_(float("nan"))
        memra.tree_attn(*args[:8], 0.0)
        assert memra.read_status(dw.cache) == 0
        flat = type("Flat", (W.Workload,), {"sm_scale": 0.0})(**x.__dict__)
        want, tol = reference(flat, words)
        got = dw.out.cpu().numpy().astype(np.float64)
        assert np.isfinite(got).all() and (np.abs(got - want) <= tol).all()
        if x is w2:
            assert (got[0, ::2] == 0).all() and (got[0, 1::2] != 0).any()


def test_bad_pages_are_left_out(memra):
    w = W.random_case(12, batch=1, q_len=4, n_heads=8, n_kv_heads=2, ctx=(300, 300))
    words = words_for(w, 8)
    dw, args = run(memra, w, words)
    memra.read_status(dw.cache)
    table = dw.page_table.clone()
    table[0, 3], table[0, 5] = w.num_pages, -1
    memra.tree_attn(dw.cache, dw.q, table, *args[3:])
    assert memra.read_status(dw.cache) == memra.DEVERR_BAD_PAGE
    want, tol = reference(w, words, missing_pages=(3, 5))
    assert (np.abs(dw.out.cpu().numpy().astype(np.float64) - want) <= tol).all()


def test_pages_past_32_bit_offsets(memra):
    # 8 KV heads: page 250,000 of q8_0 K starts past 4 GiB
    w = W.random_case(17, batch=2, q_len=4, n_heads=16, n_kv_heads=8, ctx=(100, 300))
    high = 250_000 - w.num_pages
    w.page_table = (w.page_table + high).astype(np.int32)
    w.slots = (w.slots + 16 * high).astype(np.int32)
    w.num_pages = 250_000
    from decode_attention_block_memra_gb300.runner import upload
    dw = upload(w)
    memra.kv_append(dw.cache, dw.step_k, dw.step_v, dw.step_slots)
    words = words_for(w, 17)
    mask = torch.from_numpy(words.view(np.int64).copy()).cuda()
    ws = torch.empty(memra.tree_attn_workspace_bytes(2, 4, 16, 128, w.max_seq_len), dtype=torch.uint8, device="cuda")
    memra.tree_attn(dw.cache, dw.q, dw.page_table, dw.seq_lens, w.max_seq_len, mask, dw.out, ws, w.sm_scale)
    assert memra.read_status(dw.cache) == 0
    want, tol = reference(w, words)
    assert (np.abs(dw.out.cpu().numpy().astype(np.float64) - want) <= tol).all()
    kept = torch.tensor([[1, 3]] * 2, dtype=torch.int32, device="cuda")
    pool = dw.cache.k_pool.view(w.num_pages, 8, -1)
    before = pool[high:].clone()
    memra.kv_compact(dw.cache, dw.page_table, dw.seq_lens, w.max_seq_len, kept,
                     torch.full((2,), 2, dtype=torch.int32, device="cuda"), 4)
    assert memra.read_status(dw.cache) == 0
    assert not torch.equal(pool[high:], before) and not bool(pool[:high].any())


def test_binding_refuses_other_tensors(memra):
    w = W.random_case(18, batch=2, q_len=4, n_heads=8, n_kv_heads=2, ctx=(40, 60))
    dw, args = run(memra, w, words_for(w, 18))
    cache, q, table, lens, M, mask, out, ws, scale = args
    on_host = memra.KVCache("q8_0", "q5_1", cache.num_pages, cache.n_kv_heads, cache.head_dim, device="cpu")
    for bad in ((cache, q.float(), table, lens, M, mask, out, ws), (cache, q, table[:1], lens, M, mask, out, ws),
                (cache, q, table, lens.long(), M, mask, out, ws), (cache, q, table, lens, M, mask.int(), out, ws),
                (cache, q, table, lens, M, mask[:, :3], out, ws), (cache, q, table.cpu(), lens, M, mask, out, ws),
                (cache, q, table, lens, M, mask, out[:1], ws), (cache, q.transpose(1, 2), table, lens, M, mask, out, ws),
                (cache, q, table, lens, M, mask, out, ws.cpu()), (on_host, q, table, lens, M, mask, out, ws)):
        with pytest.raises(memra.MemraError):
            memra.tree_attn(*bad)
    kept, count = torch.zeros(2, 3, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    for bad in ((table[:1], lens, M, kept, count), (table, lens[:1], M, kept, count), (table, lens, M, kept.long(), count),
                (table, lens, M, kept, count[:1]), (table, lens, M, kept.cpu(), count)):
        with pytest.raises(memra.MemraError):
            memra.kv_compact(cache, *bad, 4)
    with pytest.raises(memra.MemraError):
        memra.kv_compact(on_host, table, lens, M, kept, count, 4)
    pages = torch.zeros(1, dtype=torch.int32, device="cuda")
    with pytest.raises(memra.MemraError):
        memra.kv_copy_pages(on_host, pages, pages + 1)


def test_lengths_out_of_range(memra):
    w = W.random_case(13, batch=2, q_len=6, n_heads=8, n_kv_heads=2, ctx=(100, 100))
    words = words_for(w, 9)
    dw, args = run(memra, w, words)
    for lens, M in (([100, 4], 100), ([100, 10 ** 9], 10 ** 9), ([-7, 0], 100)):
        dw.out.fill_(float("nan"))
        n = memra.tree_attn_workspace_bytes(2, 6, 8, 128, min(M, 112))
        M = min(M, 112)
        ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
        memra.tree_attn(dw.cache, dw.q, dw.page_table, torch.tensor(lens, dtype=torch.int32, device="cuda"), M,
                        args[5], dw.out, ws, w.sm_scale)
        assert memra.read_status(dw.cache) == memra.DEVERR_BAD_SEQ_LEN
        assert bool(torch.isfinite(dw.out).all())
        for b, T in enumerate(lens):
            if T < 6:                        # nodes at positions below 0
                assert bool((dw.out[b, :6 - max(T, 0)] == 0).all())


def test_captured_call_reads_new_lengths_and_words(memra):
    w = W.random_case(14, batch=2, q_len=4, n_heads=8, n_kv_heads=2, ctx=(900, 1300))
    words = words_for(w, 10)
    dw, args, got = check(memra, w, words)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        memra.tree_attn(*args)
    dw.out.zero_()
    g.replay()
    assert np.array_equal(dw.out.cpu().numpy().astype(np.float64), got)
    other = words_for(w, 11)
    args[5].copy_(torch.from_numpy(other.view(np.int64).copy()))
    g.replay()
    want, tol = reference(w, other)
    assert (np.abs(dw.out.cpu().numpy().astype(np.float64) - want) <= tol).all()


@pytest.mark.parametrize("D,nodes", [(128, 5), (256, 5), (128, 30)])
def test_many_calls_in_a_row(memra, D, nodes):
    """No wait runs out and no byte changes over thousands of calls (a wait that names the wrong phase would)."""
    w = W.random_case(16, batch=4, q_len=nodes, n_heads=16, n_kv_heads=2, head_dim=D, k_fmt="fp8", v_fmt="fp8",
                      ctx=(300, 2500))
    dw, args, got = check(memra, w, words_for(w, 13))
    want = dw.out.clone()
    same = torch.ones((), dtype=torch.bool, device="cuda")
    for _ in range(3000):
        dw.out.zero_()
        memra.tree_attn(*args)
        same &= (dw.out == want).all()
    assert memra.read_status(dw.cache) == 0 and bool(same)


def test_two_streams_with_their_own_workspaces(memra):
    w = W.random_case(15, batch=2, q_len=8, n_heads=32, n_kv_heads=4, ctx=(3000, 5000))
    words = words_for(w, 12)
    dw, args, got = check(memra, w, words)
    outs, streams = [], [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        out, ws = torch.empty_like(dw.out), torch.empty_like(args[7])
        outs.append((out, ws))
    torch.cuda.synchronize()
    for _ in range(3):
        for s, (out, ws) in zip(streams, outs):
            memra.tree_attn(*args[:6], out, ws, args[8], stream=s)
    torch.cuda.synchronize()
    for out, _ in outs:
        assert torch.equal(out, dw.out)
