"""Eviction on the GPU against the CPU oracle: indices, weights and pool bytes, every comparison exact."""
import numpy as np
import pytest

from oracle import chunked, layout

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

PAIRS = [("q8_0", "q5_1"), ("q8_0", "q4_0"), ("fp8", "fp8"), ("nvfp4", "nvfp4"), ("fp8", "q5_1"), ("nvfp4", "q4_0")]


@pytest.fixture(scope="module")
def memra():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from decode_attention_block_memra_gb300 import _build
    _build.build()
    import decode_attention_block_memra_gb300 as m
    m.lib()
    return m


def dev(a, dtype=np.int32):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=dtype)).cuda()


def token_bytes(side, fmt, D):
    """bool [16, segment]: the bytes of a segment that hold token t, found by writing rows and looking."""
    from oracle import quant
    seg = layout.segment_bytes(side, fmt, D)
    rng = np.random.default_rng(0)
    mine = np.zeros((16, seg), bool)
    for t in range(16):
        for start in (0, 255):
            for _ in range(12):
                pool = np.full((1, 1, seg), start, np.uint8)
                row = quant.quantize_rows((rng.standard_normal((1, D)) * 3).astype(np.float16), fmt, 0.01)
                layout.write_rows(pool, side, row, np.array([t]), 0, D)
                mine[t] |= pool[0, 0] != start
    assert (mine.sum(0) == 1).all(), "every byte belongs to one token"
    return mine


class Case:
    def __init__(self, memra, kf, vf, D, heads, lens, budgets, sink, recent, weights=None, seed=0, spare=2, stride=0):
        rng = np.random.default_rng(seed)
        self.memra, self.D, self.fmt, self.heads = memra, D, (kf, vf), heads
        self.lens, self.budgets, self.sink, self.recent = lens, budgets, sink, recent
        B, most = len(lens), max(max(budgets), 1)
        used = [max(1, -(-n // 16)) for n in lens]
        per = -(-most // 16)
        self.pages = sum(used) + B * per + spare
        order = rng.permutation(self.pages)
        self.table = np.full((B, max(used)), 2 ** 30, np.int32)          # (columns past the end are not read)
        for b, n in enumerate(used):
            self.table[b, :n] = order[sum(used[:b]):sum(used[:b + 1])]
        self.to = order[sum(used):sum(used) + B * per].reshape(B, per).astype(np.int32)
        self.raw = [rng.integers(0, 256, (self.pages, heads, layout.segment_bytes(s, f, D)), dtype=np.uint8)
                    for s, f in (("k", kf), ("v", vf))]
        self.cache = memra.KVCache(kf, vf, self.pages, heads, D, k_pool=torch.from_numpy(self.raw[0]).cuda().flatten(),
                                   v_pool=torch.from_numpy(self.raw[1]).cuda().flatten())
        stride = stride or max(max(lens), 1)
        self.weights = rng.random((B, heads, stride)).astype(np.float32) if weights is None else weights
        self.kept = torch.full((B, heads, most), 77, dtype=torch.int32, device="cuda")
        self.new_w = torch.full((B, heads, most + 3), -5.0, device="cuda")
        self.new_lens = torch.full((B,), 77, dtype=torch.int32, device="cuda")

    def call(self, **kw):
        a = dict(page_table=dev(self.table), seq_lens=dev(self.lens), max_seq_len=max(max(self.lens), 0),
                 weights=dev(self.weights, np.float32), budgets=dev(self.budgets), dst_table=dev(self.to),
                 kept=self.kept, sink=self.sink, recent=self.recent, new_weights=self.new_w, new_lens=self.new_lens)
        self.memra.kv_evict(self.cache, **{**a, **kw})
        return self.memra.read_status(self.cache)

    def check(self, lens=None, budgets=None):
        lens, budgets = lens or self.lens, budgets or self.budgets
        want = [x.copy() for x in self.raw]
        kept, new_w = np.full(self.kept.shape, -1), np.full(self.new_w.shape, -5.0, np.float32)
        marks = [token_bytes(s, f, self.D) for s, f in zip("kv", self.fmt)]
        for b, (T, budget) in enumerate(zip(lens, budgets)):
            for h in range(self.heads):
                rows = chunked.kept_tokens(self.weights[b, h, :T], budget, self.sink, self.recent)
                kept[b, h, :len(rows)] = rows
                new_w[b, h, :len(rows)] = self.weights[b, h, rows]
                for j, i in enumerate(rows):
                    src, dst = self.table[b, i // 16], self.to[b, j // 16]
                    for raw, pool, mark in zip(self.raw, want, marks):
                        pool[dst, h, mark[j % 16]] = raw[src, h, mark[i % 16]]
        assert np.array_equal(self.kept.cpu().numpy(), kept)
        assert np.array_equal(self.new_w.cpu().numpy(), new_w, equal_nan=True)
        assert self.new_lens.tolist() == [min(a, b) for a, b in zip(lens, budgets)]
        for got, pool in zip((self.cache.k_pool, self.cache.v_pool), want):
            assert np.array_equal(got.cpu().numpy().reshape(pool.shape), pool)


@pytest.mark.parametrize("kf,vf", PAIRS)
@pytest.mark.parametrize("D", [128, 256])
def test_formats(memra, kf, vf, D):
    c = Case(memra, kf, vf, D, 2, [100, 37, 16, 1], [40, 37, 5, 1], 3, 7)
    assert c.call() == 0
    c.check()


@pytest.mark.parametrize("lens,budgets,sink,recent", [
    ([1], [1], 0, 0), ([1], [0], 4, 4), ([0, 5], [3, 3], 1, 1), ([64], [64], 0, 0), ([65], [64], 0, 0),
    ([300], [17], 4, 100),                   # the recent ones alone pass the budget
    ([300], [17], 100, 5), ([300], [17], 0, 0), ([300, 299, 17], [16, 15, 17], 2, 2),
    ([5000, 4097], [1000, 2049], 5, 64), ([9000], [8999], 1, 0), ([20000], [33], 0, 16), ([33000], [20000], 64, 64),
])
def test_lengths_and_budgets(memra, lens, budgets, sink, recent):
    c = Case(memra, "fp8", "fp8", 128, 1 if max(lens) > 4000 else 3, lens, budgets, sink, recent)
    assert c.call() == 0
    c.check()


@pytest.mark.parametrize("kind", ["equal", "zeros", "few", "steps", "negative", "special", "denormal"])
@pytest.mark.parametrize("T,budget", [(700, 301), (5000, 123)])
def test_ties_and_special_weights(memra, kind, T, budget):
    rng = np.random.default_rng(T)
    w = {"equal": lambda: np.full(T, 0.25), "zeros": lambda: np.where(rng.random(T) < 0.5, 0.0, -0.0),
         "few": lambda: rng.choice([0.0, 0.5, 0.5 + 2.0 ** -25], T), "steps": lambda: 1 + rng.integers(0, 3, T) * 2.0 ** -23,
         "negative": lambda: rng.standard_normal(T), "denormal": lambda: rng.integers(-3, 4, T) * 1.4e-45,
         "special": lambda: rng.choice([np.nan, np.inf, -np.inf, 1.0, 0.0, -1.0], T)}[kind]().astype(np.float32)
    c = Case(memra, "q8_0", "q5_1", 128, 1, [T], [budget], 2, 3, weights=w[None, None])
    assert c.call() == 0
    c.check()


def test_optional_outputs_and_wider_weights(memra):
    c = Case(memra, "q8_0", "q5_1", 128, 2, [50, 40], [20, 30], 1, 2, stride=77)
    assert c.call(new_weights=None, new_lens=None) == 0
    assert (c.new_w == -5).all() and (c.new_lens == 77).all()
    assert c.call() == 0
    c.check()


def test_bad_lengths_budgets_and_pages(memra):
    c = Case(memra, "q8_0", "q5_1", 128, 2, [64, 48, 30], [20, 20, 20], 1, 2)
    M = memra
    assert c.call(seq_lens=dev([64, -4, 1000])) & M.DEVERR_BAD_SEQ_LEN        # (and its columns past the end hold no page)
    assert c.new_lens.tolist() == [20, 0, 20]
    c = Case(memra, "q8_0", "q5_1", 128, 2, [64, 48, 30], [20, 20, 20], 1, 2)
    assert c.call(budgets=dev([-1, 21, 20])) == M.DEVERR_BAD_SEQ_LEN
    c.check(budgets=[0, 20, 20])
    # a source page outside the pool: its rows do not move; the indices still say what was kept
    c = Case(memra, "q8_0", "q5_1", 128, 1, [64], [64], 0, 0)
    table = c.table.copy()
    table[0, 1], table[0, 2] = -1, c.pages
    assert c.call(page_table=dev(table)) == M.DEVERR_BAD_PAGE
    got = c.cache.k_pool.cpu().numpy().reshape(c.raw[0].shape)
    assert np.array_equal(got[c.to[0, [0, 3]]], c.raw[0][c.table[0, [0, 3]]])
    assert np.array_equal(got[c.to[0, [1, 2]]], c.raw[0][c.to[0, [1, 2]]])
    c = Case(memra, "q8_0", "q5_1", 128, 1, [64], [64], 0, 0)
    to = c.to.copy()
    to[0, 1], to[0, 2] = -1, c.pages
    assert c.call(dst_table=dev(to)) == M.DEVERR_BAD_PAGE
    got = c.cache.k_pool.cpu().numpy().reshape(c.raw[0].shape)
    assert np.array_equal(got[c.to[0, [0, 3]]], c.raw[0][c.table[0, [0, 3]]])
    assert np.array_equal(got[c.to[0, [1, 2]]], c.raw[0][c.to[0, [1, 2]]])


def test_a_shared_prefix_may_be_read_by_several(memra):
    c = Case(memra, "q8_0", "q5_1", 128, 2, [80, 80], [32, 48], 2, 2)
    c.table[1, :3] = c.table[0, :3]
    assert c.call() == 0
    c.check()


def test_the_longest_context(memra):
    T, budget = 262144, 16384
    rng = np.random.default_rng(5)
    w = (rng.random((1, 2, T)) ** 8 * (rng.random((1, 2, T)) > 0.1)).astype(np.float32)
    cache = memra.KVCache("fp8", "fp8", T // 16 + budget // 16, 2, 128)
    g = torch.Generator(device="cuda").manual_seed(0)
    for pool in (cache.k_pool, cache.v_pool):
        pool.copy_(torch.randint(0, 256, pool.shape, dtype=torch.uint8, device="cuda", generator=g))
    before = cache.k_pool.clone().view(-1, 2, 2048)
    pages = rng.permutation(T // 16 + budget // 16).astype(np.int32)
    kept = torch.empty(1, 2, budget, dtype=torch.int32, device="cuda")
    memra.kv_evict(cache, dev(pages[None, :T // 16]), dev([T]), T, dev(w, np.float32), dev([budget]),
                   dev(pages[None, T // 16:]), kept, sink=64, recent=1024)
    assert memra.read_status(cache) == 0
    after = cache.k_pool.view(-1, 2, 2048).cpu().numpy()
    before, mark = before.cpu().numpy(), token_bytes("k", "fp8", 128)
    where = np.stack([np.nonzero(m)[0] for m in mark])
    for h in range(2):
        middle = np.arange(64, T - 1024)
        best = middle[np.lexsort((middle, -w[0, h, middle]))][:budget - 1088]
        rows = np.concatenate((np.arange(64), np.sort(best), np.arange(T - 1024, T)))
        assert np.array_equal(kept[0, h].cpu().numpy(), rows)
        j = np.arange(budget)
        got = after[pages[T // 16 + j // 16][:, None], h, where[j % 16]]
        assert np.array_equal(got, before[pages[rows // 16][:, None], h, where[rows % 16]])


def test_refusals_of_the_binding(memra):
    c = Case(memra, "q8_0", "q5_1", 128, 2, [50, 40], [20, 30], 1, 2)
    i32 = torch.int32
    for bad in (dict(page_table=dev(c.table).long()), dict(seq_lens=dev([50])), dict(weights=dev(c.weights, np.float64)),
                dict(weights=dev(c.weights[:, :1], np.float32)), dict(max_seq_len=51), dict(budgets=dev([20, 30], np.int64)),
                dict(dst_table=dev(c.to[:, :1])), dict(kept=torch.empty(2, 3, 30, dtype=i32, device="cuda")),
                dict(new_weights=torch.empty(2, 2, 29, device="cuda")), dict(new_lens=torch.empty(3, dtype=i32, device="cuda")),
                dict(sink=-1), dict(recent=-1), dict(kept=torch.empty(2, 2, 30, dtype=i32)), dict(max_seq_len=-1)):
        with pytest.raises(memra.MemraError):
            c.call(**bad)
    assert c.call() == 0
    c.check()


@pytest.mark.parametrize("lens,budgets,heads", [
    ([700 - 9 * b for b in range(64)], [40 + b % 3 for b in range(64)], 8),          # more rows than run at once
    ([9000, 5000, 1, 4097], [300, 1000, 1, 64], 2),                                   # clusters
    ([70000], [500], 4), ([5, 0, 30, 16], [3, 3, 0, 16], 3),
])
@pytest.mark.parametrize("which", ["seq_lens", "budgets"])
def test_lengths_updated_in_place(memra, lens, budgets, heads, which):
    c = Case(memra, "fp8", "fp8", 128, heads, lens, budgets, 1, 4)
    c.new_lens = dev(lens if which == "seq_lens" else budgets)
    assert c.call(**{which: c.new_lens}) == 0
    c.check()


def test_lengths_updated_in_place_by_a_replayed_graph(memra):
    """Two evictions of a cache to half, then to a quarter, by one pair of captured calls: the second reads what the first left."""
    c = Case(memra, "q8_0", "q5_1", 128, 2, [3000, 1200], [1500, 600], 2, 8)
    lens, weights, first, second = dev(c.lens), dev(c.weights, np.float32), dev(c.budgets), dev([750, 300])
    kept, w2 = torch.empty(2, 2, 750, dtype=torch.int32, device="cuda"), torch.zeros(2, 2, 1500, device="cuda")
    to = dev(np.arange(2 * 47).reshape(2, 47) + c.pages)
    cache = memra.KVCache("q8_0", "q5_1", c.pages + 94, 2, 128)
    cache.k_pool[:c.cache.k_pool.numel()], cache.v_pool[:c.cache.v_pool.numel()] = c.cache.k_pool, c.cache.v_pool
    table, half = dev(c.table), dev(c.to)

    def calls():
        memra.kv_evict(cache, table, lens, 3000, weights, first, half, c.kept, 2, 8, new_weights=w2, new_lens=lens)
        memra.kv_evict(cache, half, lens, 1500, w2, second, to, kept, 2, 8, new_lens=lens)

    calls()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for _ in range(3):
        lens.copy_(dev(c.lens))
        kept.fill_(77)
        graph.replay()
        assert memra.read_status(cache) == 0 and lens.tolist() == [750, 300]
        for b in range(2):
            for h in range(2):
                rows = chunked.kept_tokens(c.weights[b, h, :c.lens[b]], c.budgets[b], 2, 8)
                again = chunked.kept_tokens(c.weights[b, h, rows], lens[b].item(), 2, 8)
                assert np.array_equal(kept[b, h].cpu().numpy()[:len(again)], again)
                assert (kept[b, h, len(again):] == -1).all()


@pytest.mark.parametrize("on", ["current", "stream", "handle"])
def test_budgets_of_nothing(memra, on):
    """kept has no column: no sequence keeps a token, and new_lens says so."""
    c = Case(memra, "fp8", "fp8", 128, 2, [50, 0, 7], [0, 0, 0], 1, 2)
    c.kept, c.to, c.new_w = c.kept[..., :0], c.to[:, :0], c.new_w[..., :0]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert c.call(stream={"current": None, "stream": side, "handle": side.cuda_stream}[on]) == 0
    torch.cuda.synchronize()
    c.check()
    lens = dev(c.lens)
    assert c.call(seq_lens=lens, new_lens=lens, new_weights=None) == 0 and lens.tolist() == [0, 0, 0]
    with pytest.raises(memra.MemraError):
        c.call(new_lens=torch.zeros(2, dtype=torch.int32, device="cuda"))


def test_sequences_without_a_token_and_no_weights(memra):
    c = Case(memra, "fp8", "fp8", 128, 2, [0, 0], [3, 3], 1, 2)
    empty = torch.empty(2, 2, 0, device="cuda")
    for new_weights in (c.new_w, None):
        assert c.call(weights=empty, max_seq_len=0, new_weights=new_weights) == 0
        c.check()
    # a length past the bound of 0 is clamped
    assert c.call(weights=empty, max_seq_len=0, seq_lens=dev([5, 0])) == memra.DEVERR_BAD_SEQ_LEN
    c.check()


def best(w, T, n, sink, recent):
    """kept_tokens of float32 weights without NaN, by numpy's sort."""
    recent = min(recent, n)
    sink = min(sink, n - recent)
    middle = np.arange(sink, T - recent)
    first = middle[np.lexsort((middle, -w[middle]))][:n - sink - recent]
    return np.concatenate((np.arange(sink), np.sort(first), np.arange(T - recent, T))).astype(np.int64)


@pytest.mark.parametrize("kind", ["random", "few", "rising"])
@pytest.mark.parametrize("batch,heads,T,budget", [(40, 8, 40000, 3000),      # one CTA to a row, three rounds of its registers
                                                  (24, 4, 50000, 700),       # two to a row
                                                  (1, 2, 700000, 30000)])    # sixteen
def test_rows_that_pass_a_cta_s_registers(memra, batch, heads, T, budget, kind):
    rng = np.random.default_rng(T)
    shape = (batch, heads, T)
    w = {"random": lambda: rng.random(shape), "few": lambda: rng.choice([0.0, 0.25, 0.5], shape),
         "rising": lambda: np.broadcast_to(np.arange(T) % 60000, shape)}[kind]().astype(np.float32)
    lens = [T - 1000 * b for b in range(batch)] if batch < 30 else [T - 300 * b for b in range(batch)]
    pages = T // 16 + 1                      # every sequence reads the same pages
    cache = memra.KVCache("fp8", "fp8", pages + batch * (-(-budget // 16)), heads, 128)
    g = torch.Generator(device="cuda").manual_seed(0)
    for pool in (cache.k_pool, cache.v_pool):
        pool.copy_(torch.randint(0, 256, pool.shape, dtype=torch.uint8, device="cuda", generator=g))
    before = cache.k_pool.view(-1, heads, 2048)[:pages].cpu().numpy()
    table = np.tile(rng.permutation(pages).astype(np.int32), (batch, 1))
    to = (pages + rng.permutation(batch * (-(-budget // 16)))).astype(np.int32).reshape(batch, -1)
    kept, new = torch.empty(batch, heads, budget, dtype=torch.int32, device="cuda"), torch.zeros(batch, heads, budget, device="cuda")
    new_lens = dev(lens)
    memra.kv_evict(cache, dev(table), new_lens, T, dev(w, np.float32), dev([budget] * batch), dev(to), kept, 5, 100,
                   new_weights=new, new_lens=new_lens)
    assert memra.read_status(cache) == 0 and new_lens.tolist() == [budget] * batch
    after = cache.k_pool.view(-1, heads, 2048).cpu().numpy()
    where = np.stack([np.nonzero(m)[0] for m in token_bytes("k", "fp8", 128)])
    kept, new, j = kept.cpu().numpy(), new.cpu().numpy(), np.arange(budget)
    for b in range(batch):
        for h in range(heads):
            rows = best(w[b, h], lens[b], budget, 5, 100)
            assert np.array_equal(kept[b, h], rows) and np.array_equal(new[b, h], w[b, h, rows])
            got = after[to[b, j // 16][:, None], h, where[j % 16]]
            assert np.array_equal(got, before[table[b, rows // 16][:, None], h, where[rows % 16]])


def test_many_calls_in_a_row_and_side_by_side(memra):
    cases = [Case(memra, "q8_0", "q5_1", 128, 2, [700, 40], [301, 40], 2, 3, seed=1),
             Case(memra, "fp8", "fp8", 256, 3, [5000, 4097], [1000, 2049], 5, 64, seed=2),
             Case(memra, "nvfp4", "q4_0", 128, 1, [70000], [900], 0, 16, seed=3)]
    calls, want = [], []
    for c in cases:
        assert c.call() == 0
        c.check()
        want.append([t.clone() for t in (c.kept, c.new_w, c.new_lens, c.cache.k_pool, c.cache.v_pool)])
        a = dict(page_table=dev(c.table), seq_lens=dev(c.lens), max_seq_len=max(c.lens), weights=dev(c.weights, np.float32),
                 budgets=dev(c.budgets), dst_table=dev(c.to), kept=c.kept, sink=c.sink, recent=c.recent, new_weights=c.new_w,
                 new_lens=c.new_lens)
        calls.append((c.cache, a))
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for turn in range(600):
        for (cache, a), stream in zip(calls, streams):
            memra.kv_evict(cache, **a, stream=stream if turn < 300 else None)
        if turn == 299:
            torch.cuda.synchronize()
    for c, w in zip(cases, want):
        assert memra.read_status(c.cache) == 0
        assert all(torch.equal(t, u) for t, u in zip((c.kept, c.new_w, c.new_lens, c.cache.k_pool, c.cache.v_pool), w))
