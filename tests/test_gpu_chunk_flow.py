"""A long prompt in a cache of bounded size, as the four operators are used together.

Each round: the new tokens' rows are normalized, turned and appended, attend over what the
cache still holds, add to its keys' weights, and an eviction leaves the budget in the other
half of the pages.  Every stage is held against float64 given what the stage before it made:
the rows against the formula; attention and weights against the cache's rows (those of k_out,
quantized) with the tolerances of chunk_cases.py and test_gpu_key_weights.py; the kept tokens
exactly, by the weights that the GPU has.
"""
import numpy as np
import pytest

from oracle import chunked

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from chunk_cases import Chunk, dequantized, dev     # noqa: E402
from test_gpu_key_weights import Weights, memra     # noqa: E402, F401
from test_gpu_norm_rope import check as check_rows     # noqa: E402

PAGES = 24                                   # of a sequence in each half of the pool


class Flow(Weights):
    """`lens` tokens of every sequence in the cache, each KV head its own; the next `new` come in."""

    def __init__(self, memra, kf, vf, D, Hq, Hkv, batch, budgets, sink, recent, seed):
        self.memra, self.kf, self.vf, self.D, self.Hq, self.Hkv, self.window = memra, kf, vf, D, Hq, Hkv, 0
        self.budgets, self.sink, self.recent, self.B = budgets, sink, recent, batch
        self.rng = np.random.default_rng(seed)
        self.scales = [16.0 / 448 if f == "fp8" else 16.0 / 2688 if f == "nvfp4" else 1.0 for f in (kf, vf)]
        self.cache = memra.KVCache(kf, vf, 2 * batch * PAGES, Hkv, D, *self.scales)
        self.tables = self.rng.permutation(2 * batch * PAGES).astype(np.int32).reshape(2, batch, PAGES)
        self.half = 0
        self.seen, self.lens, self.new = [0] * batch, [0] * batch, [0] * batch
        self.k = [[np.zeros((0, D), np.float16) for _ in range(Hkv)] for _ in range(batch)]
        self.v = [[np.zeros((0, D), np.float16) for _ in range(Hkv)] for _ in range(batch)]
        self.freq = (1e4 ** (-np.arange(D // 4) / (D // 4))).astype(np.float32)
        self.qw, self.kw = ((1 + 0.2 * self.rng.standard_normal(D)).astype(np.float32) for _ in range(2))
        self.weights = torch.zeros(2, batch, Hkv, PAGES * 16, device="cuda")
        self.ws = torch.empty(memra.chunk_attn_workspace_bytes(D), dtype=torch.uint8, device="cuda")

    @property
    def table(self):
        return self.tables[self.half]

    def keys(self, b, h):
        return 0, dequantized(self.k[b][h], self.kf, self.scales[0]), dequantized(self.v[b][h], self.vf, self.scales[1])

    def step(self, new):
        """The chunk's tensors, and the lists behind them brought up to date."""
        self.new = new
        self.starts = np.concatenate(([0], np.cumsum(new))).astype(np.int32)
        total, T0 = sum(new), list(self.lens)
        self.lens = [T + n for T, n in zip(T0, new)]
        self.raw = self.rng.standard_normal((total, self.Hq + 2 * self.Hkv, self.D)).astype(np.float16)
        at = [np.arange(t, t + n) for t, n in zip(T0, new)]
        self.slots = np.concatenate([self.table[b][p // 16] * 16 + p % 16 for b, p in enumerate(at)]).astype(np.int32)
        # positions of the text, not of the cache
        self.pos = np.concatenate([np.arange(s, s + n) for s, n in zip(self.seen, new)]).astype(np.int32)
        self.seen = [s + n for s, n in zip(self.seen, new)]
        self.fused, Hq, Hkv = dev(self.raw), self.Hq, self.Hkv
        self.k_out = torch.empty(total, Hkv, self.D, dtype=torch.float16, device="cuda")
        self.out = torch.empty(total, Hq, self.D, dtype=torch.float16, device="cuda")
        self.lse = torch.empty(total, Hq, device="cuda")
        self.d = dict(starts=dev(self.starts), table=dev(self.table), other=dev(self.tables[1 - self.half]),
                      lens=dev(np.array(self.lens, np.int32)), slots=dev(self.slots), pos=dev(self.pos), freq=dev(self.freq),
                      qw=dev(self.qw), kw=dev(self.kw), budgets=dev(np.array(self.budgets, np.int32)))
        self.kept = torch.empty(self.B, Hkv, max(self.budgets), dtype=torch.int32, device="cuda")
        self.new_lens = torch.empty(self.B, dtype=torch.int32, device="cuda")

    def rope(self):
        f, d, Hq, Hkv = self.fused, self.d, self.Hq, self.Hkv
        self.memra.qk_norm_rope(f[:, :Hq], f[:, Hq:Hq + Hkv], d["pos"], d["freq"], f[:, :Hq], self.k_out, d["qw"], d["kw"],
                                cache=self.cache, v=f[:, Hq + Hkv:], slot_mapping=d["slots"])

    def attend(self, collect=True):
        d, limit = self.d, PAGES * 16
        self.memra.chunk_attn(self.cache, self.fused[:, :self.Hq], d["starts"], d["table"], d["lens"], limit, self.out, self.ws,
                              lse=self.lse)
        if collect:
            self.memra.key_weights(self.cache, self.fused[:, :self.Hq], self.lse, d["starts"], d["table"], d["lens"], limit,
                                   self.weights[self.half])

    def evict(self):
        d = self.d
        self.memra.kv_evict(self.cache, d["table"], d["lens"], PAGES * 16, self.weights[self.half], d["budgets"], d["other"],
                            self.kept, self.sink, self.recent, new_weights=self.weights[1 - self.half], new_lens=self.new_lens)

    def all(self):
        self.rope(), self.attend(), self.evict()

    def take_rows(self):
        """The finished rows, as the cache has them."""
        self.q, k = self.fused[:, :self.Hq].cpu().numpy(), self.k_out.cpu().numpy()
        for b in range(self.B):
            rows = slice(self.starts[b], self.starts[b + 1])
            for h in range(self.Hkv):
                self.k[b][h] = np.concatenate((self.k[b][h], k[rows, h]))
                self.v[b][h] = np.concatenate((self.v[b][h], self.raw[rows, self.Hq + self.Hkv + h]))

    def run_and_check(self, new):
        Hq, Hkv = self.Hq, self.Hkv
        self.step(new)
        self.old = self.weights[self.half].cpu().numpy()
        self.weights[1 - self.half].zero_()          # (a key that comes in has collected nothing)
        self.all()
        assert self.memra.read_status(self.cache) == 0
        q, k = self.fused[:, :Hq], self.k_out
        check_rows(q, self.raw[:, :Hq], self.qw, self.pos, self.freq, False)
        check_rows(k, self.raw[:, Hq:Hq + Hkv], self.kw, self.pos, self.freq, False)
        self.take_rows()
        Chunk.check(self)
        self.lse_in = self.lse.cpu().numpy()
        weights, self.weights_now = self.weights, self.weights[self.half]
        self.weights = self.weights_now
        Weights.check(self, 1.0)
        self.weights = weights
        # what stays
        kept, w = self.kept.cpu().numpy(), self.weights_now.cpu().numpy()
        moved, lens = self.weights[1 - self.half].cpu().numpy(), self.new_lens.cpu().numpy()
        for b in range(self.B):
            n = min(self.lens[b], self.budgets[b])
            assert lens[b] == n
            for h in range(Hkv):
                want = chunked.kept_tokens(w[b, h, :self.lens[b]], n, self.sink, self.recent)
                assert np.array_equal(kept[b, h, :n], want) and (kept[b, h, n:] == -1).all()
                assert np.array_equal(moved[b, h, :n], w[b, h, want]) and not moved[b, h, n:].any()
                self.k[b][h], self.v[b][h] = self.k[b][h][want], self.v[b][h][want]
            self.lens[b] = int(n)
        self.half = 1 - self.half


CASES = [("q8_0", "q5_1", 128, 8, 2), ("fp8", "fp8", 256, 4, 1), ("nvfp4", "nvfp4", 128, 8, 2), ("q8_0", "q4_0", 256, 4, 2)]


@pytest.mark.parametrize("kf,vf,D,Hq,Hkv", CASES)
def test_a_prompt_in_chunks_under_a_budget(memra, kf, vf, D, Hq, Hkv):     # noqa: F811
    f = Flow(memra, kf, vf, D, Hq, Hkv, 3, [100, 64, 0], sink=4, recent=24, seed=D)
    for new in ([70, 33, 5], [130, 1, 64], [1, 100, 0], [1, 1, 1]):
        f.run_and_check(new)
    # the next token, by this attention and by decode attention over what was kept
    f.step([1, 1, 1])
    f.rope()
    f.attend(collect=False)
    out = torch.empty(3, 1, Hq, D, dtype=torch.float16, device="cuda")
    ws = torch.empty(memra.decode_attn_workspace_bytes(3, 1, Hq, D, PAGES * 16), dtype=torch.uint8, device="cuda")
    memra.decode_attn(f.cache, f.fused[:, :Hq].contiguous().view(3, 1, Hq, D), f.d["table"], f.d["lens"], PAGES * 16, out, ws)
    assert memra.read_status(f.cache) == 0
    f.take_rows()
    Chunk.check(f)
    f.out, f.operand = out.view(3, Hq, D), 2.0 ** -11
    Chunk.check(f, lse=False)


def test_a_captured_round_on_another_stream(memra):     # noqa: F811
    f = Flow(memra, "q8_0", "q5_1", 128, 8, 2, 2, [80, 50], sink=2, recent=16, seed=3)
    f.run_and_check([90, 200])
    f.run_and_check([40, 7])
    f.step([33, 64])
    raw, start = f.fused.clone(), f.weights.clone()
    f.all()
    results = (f.fused, f.k_out, f.out, f.lse, f.kept, f.new_lens, f.weights, f.cache.k_pool, f.cache.v_pool)
    want = [t.clone() for t in results]
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        f.all()
    for _ in range(2):
        for t in (f.k_out, f.out, f.lse, f.kept, f.new_lens):
            t.zero_()
        f.weights.copy_(start)
        f.fused.copy_(raw)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph.replay()
        side.synchronize()
        for got, ref in zip(results, want):
            assert torch.equal(got, ref)
    assert memra.read_status(f.cache) == 0


def test_weights_that_must_be_set_are_those_of_new_tokens(memra):     # noqa: F811
    """Zeros where the round's tokens come in, NaN everywhere else: the same tokens stay, with the same weights, as with zeros."""
    flows = [Flow(memra, "q8_0", "q5_1", 128, 8, 2, 3, [100, 64, 9], sink=4, recent=8, seed=5) for _ in range(2)]
    flows[1].weights.fill_(float("nan"))
    for new in ([70, 33, 5], [130, 1, 64], [1, 100, 0], [1, 1, 1]):
        got = []
        for i, f in enumerate(flows):
            before = list(f.lens)
            f.step(new)
            now, other = f.weights[f.half], f.weights[1 - f.half]
            for b, (T, n) in enumerate(zip(before, new)):
                now[b, :, T:T + n] = 0
            other.fill_(float("nan") if i else 0.0)
            f.all()
            assert memra.read_status(f.cache) == 0
            lens = f.new_lens.tolist()
            assert lens == [min(T, n) for T, n in zip(f.lens, f.budgets)]
            got.append([f.kept.clone(), f.out.clone()] + [other[b, :, :n].clone() for b, n in enumerate(lens)])
            f.lens, f.half = lens, 1 - f.half
        assert all(torch.equal(a, b) for a, b in zip(*got))
