"""The format pairs that the other tests of the operators for chunks do not run, by the same checks."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import workloads as W     # noqa: E402
from chunk_cases import PAIRS, Chunk, dev     # noqa: E402
from test_gpu_evict import Case     # noqa: E402
from test_gpu_key_weights import memra     # noqa: E402, F401

OTHERS = [(k, v) for k in W.K_FORMATS for v in W.V_FORMATS if (k, v) not in PAIRS]


def test_all_pairs_are_run():
    assert len(OTHERS) + len(PAIRS) == 12


@pytest.mark.parametrize("kf,vf", OTHERS)
@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("window", [0, 70])
def test_chunks(memra, kf, vf, D, window):     # noqa: F811
    c = Chunk(memra, kf, vf, D, 8, 2, [33, 1, 200, 0, 5, 1], [100, 700, 3, 50, 0, 1500], pad=3, seed=D, window=window)
    assert c.call() == 0
    c.check()


@pytest.mark.parametrize("kf,vf", OTHERS)
@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("new,past", [([1], [9000]), ([300], [5000]), ([1, 700], [20000, 100]), ([129], [16383])])
def test_chunks_that_are_cut_and_joined(memra, kf, vf, D, new, past):     # noqa: F811
    c = Chunk(memra, kf, vf, D, 4, 1, new, past, seed=2)
    assert c.call() == 0
    c.check()


@pytest.mark.parametrize("kf,vf", OTHERS)
@pytest.mark.parametrize("D", [128, 256])
def test_long_sums(memra, kf, vf, D):     # noqa: F811
    """Each CTA takes over 7,680 keys of a block."""
    c = Chunk(memra, kf, vf, D, 160, 160, [2], [16382], fill=False, v_of=lambda *s: 1 + np.random.default_rng(1).random(s))
    assert c.call() == 0
    c.check(heads=[0, 1, 159])


@pytest.mark.parametrize("kf,vf", OTHERS)
@pytest.mark.parametrize("D", [128, 256])
def test_one_kv_head_of_many_rows_and_bad_pages(memra, kf, vf, D):     # noqa: F811
    c = Chunk(memra, kf, vf, D, 96, 2, [3, 40, 1], [90, 10, 333], seed=3)
    assert c.call() == 0
    c.check()
    want = c.out.clone()
    table = c.table.copy()
    table[1, 0] = -1
    assert c.call(page_table=dev(table)) == memra.DEVERR_BAD_PAGE
    assert torch.equal(c.out[:3], want[:3]) and torch.equal(c.out[43:], want[43:]) and torch.isfinite(c.out).all()


@pytest.mark.parametrize("kf,vf", OTHERS)
@pytest.mark.parametrize("D", [128, 256])
def test_many_calls_in_a_row(memra, kf, vf, D):     # noqa: F811
    c = Chunk(memra, kf, vf, D, 8, 2, [70, 1, 9], [500, 1200, 0], seed=D)
    assert c.call() == 0
    c.check()
    want, a = c.out.clone(), c.args()
    for _ in range(500):
        memra.chunk_attn(c.cache, **a)
    assert memra.read_status(c.cache) == 0 and torch.equal(c.out, want)


@pytest.mark.parametrize("kf,vf", OTHERS)
@pytest.mark.parametrize("D", [128, 256])
def test_evictions(memra, kf, vf, D):     # noqa: F811
    c = Case(memra, kf, vf, D, 2, [100, 37, 16, 1], [40, 37, 5, 1], 3, 7)
    assert c.call() == 0
    c.check()


@pytest.mark.parametrize("kf,vf", OTHERS)
@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("T", [5, 650])
def test_rows_stored_as_kv_append_stores_them(memra, kf, vf, D, T):     # noqa: F811
    rng = np.random.default_rng(T)
    x = dev(rng.standard_normal((T, 6, D)).astype(np.float16))
    pages = -(-T // 16) + 3
    slots = dev(rng.permutation(pages * 16)[:T].astype(np.int32))
    pos, freq = dev(np.arange(T, dtype=np.int32)), dev((1e4 ** (-np.arange(D // 2) / (D // 2))).astype(np.float32))
    ours, theirs = (memra.KVCache(kf, vf, pages, 2, D, 0.02, 0.02) for _ in range(2))
    q_out, k_out = torch.empty(T, 2, D, dtype=torch.float16, device="cuda"), torch.empty(T, 2, D, dtype=torch.float16, device="cuda")
    ones = torch.ones(D, device="cuda")
    memra.qk_norm_rope(x[:, :2], x[:, 2:4], pos, freq, q_out, k_out, ones, ones, cache=ours, v=x[:, 4:], slot_mapping=slots)
    assert memra.read_status(ours) == 0
    memra.kv_append(theirs, k_out, x[:, 4:].contiguous(), slots)
    assert torch.equal(ours.k_pool, theirs.k_pool) and torch.equal(ours.v_pool, theirs.v_pool)
