"""Page copies and tree compaction on the GPU, byte for byte against the CPU layout oracle.

Expected pools are built by the oracle's quantizer and layout (oracle/): the
moved rows are written again at their new slots over the pools' starting bytes,
so a byte that does not belong to a moved row must keep its value.  Nothing is
rounded; every comparison is exact.
"""
import numpy as np
import pytest

from oracle import layout, quant

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


def make_cache(memra, kf, vf, pages, heads, D, seed):
    """A cache whose pools hold random bytes, and copies of them as [pages, heads, segment]."""
    rng = np.random.default_rng(seed)
    kp, vp = (rng.integers(0, 256, (pages, heads, layout.segment_bytes(s, f, D)), dtype=np.uint8)
              for s, f in (("k", kf), ("v", vf)))
    cache = memra.KVCache(kf, vf, pages, heads, D, 0.01, 0.02, k_pool=torch.from_numpy(kp).cuda().flatten(),
                          v_pool=torch.from_numpy(vp).cuda().flatten())
    return cache, kp, vp


def pools(cache, like):
    return [p.cpu().numpy().reshape(x.shape) for p, x in zip((cache.k_pool, cache.v_pool), like)]


def dev(a, dtype=np.int32):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=dtype)).cuda()


# ------------------------------------------------------------------- copies --

@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("kf,vf", PAIRS)
@pytest.mark.parametrize("n,heads", [(1, 1), (7, 2), (33, 5)])
def test_copy_pages(memra, kf, vf, D, n, heads):
    pages = 2 * n + 3
    cache, kp, vp = make_cache(memra, kf, vf, pages, heads, D, n)
    order = np.random.default_rng(n).permutation(pages)
    src, dst = order[:n], order[n:2 * n]
    memra.kv_copy_pages(cache, dev(src), dev(dst))
    assert memra.read_status(cache) == 0
    kp[dst], vp[dst] = kp[src], vp[src]
    for got, want in zip(pools(cache, (kp, vp)), (kp, vp)):
        assert np.array_equal(got, want)


def test_copy_pages_repeated_source_padding_and_bad_ids(memra):
    cache, kp, vp = make_cache(memra, "q8_0", "q5_1", 12, 2, 128, 3)
    src = [4, 4, -1, 5, 12, 0, 2 ** 31 - 1, 6, 7]
    dst = [1, 2, 3, -7, 8, 12, 9, 10, 7]            # a source twice, padding on either side, ids past the pool, onto itself
    memra.kv_copy_pages(cache, dev(src), dev(dst))
    assert memra.read_status(cache) == memra.DEVERR_BAD_PAGE
    for s, d in ((4, 1), (4, 2), (6, 10)):
        kp[d], vp[d] = kp[s], vp[s]
    for got, want in zip(pools(cache, (kp, vp)), (kp, vp)):
        assert np.array_equal(got, want)
    memra.kv_copy_pages(cache, dev([0, 1]), dev([2, 3]), n=0)
    assert memra.read_status(cache) == 0
    with pytest.raises(memra.MemraError):
        memra.kv_copy_pages(cache, dev([0, 1]), dev([2]))


def test_copy_pages_past_32_bit_offsets(memra):
    # 17 * 128 * 8 = 17,408 bytes of K a page: page 250,000 starts past 4 GiB
    pages, heads, D = 250_100, 8, 128
    cache = memra.KVCache("q8_0", "q4_0", pages, heads, D)
    k, v = cache.k_pool.view(pages, -1), cache.v_pool.view(pages, -1)
    src, dst = torch.tensor([3, 250_099], device="cuda"), torch.tensor([250_050, 5], device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    for p in (k, v):
        p[src] = torch.randint(0, 256, p[src].shape, dtype=torch.uint8, device="cuda", generator=g)
    memra.kv_copy_pages(cache, src.int(), dst.int())
    assert memra.read_status(cache) == 0
    for p in (k, v):
        assert torch.equal(p[dst], p[src])
        assert int((p != 0).any(1).sum()) == 4


# --------------------------------------------------------------- compaction --

def compact_case(memra, kf, vf, D, heads, lens, nodes, kept, count, seed, max_seq_len=None, table_cols=None):
    """Runs kv_compact on appended trees and returns (got, want) pools and the status flags."""
    rng = np.random.default_rng(seed)
    B = len(lens)
    cols = table_cols or max(-(-int(t) // 16) for t in lens) + 1
    pages = B * cols + 2
    cache, kp, vp = make_cache(memra, kf, vf, pages, heads, D, seed)
    table = rng.permutation(pages)[:B * cols].reshape(B, cols).astype(np.int32)
    rows = [rng.standard_normal((2, nodes, heads, D)).astype(np.float16) for _ in range(B)]

    def write(b, positions, which):
        """Row which[i] of sequence b at positions[i], by the oracle."""
        slots = table[b, positions // 16].astype(np.int64) * 16 + positions % 16
        for h in range(heads):
            for side, fmt, pool, scale, x in (("k", kf, kp, 0.01, rows[b][0]), ("v", vf, vp, 0.02, rows[b][1])):
                layout.write_rows(pool, side, quant.quantize_rows(x[which, h], fmt, scale), slots, h, D)

    for b, T in enumerate(lens):
        pos = np.arange(T - nodes, T)
        live = pos >= 0
        write(b, pos[live], np.nonzero(live)[0])
    cache.k_pool.copy_(torch.from_numpy(kp).flatten())
    cache.v_pool.copy_(torch.from_numpy(vp).flatten())
    memra.kv_compact(cache, dev(table), dev(lens), max_seq_len or max(lens), dev(kept), dev(count), nodes)
    flags = memra.read_status(cache)
    for b, T in enumerate(lens):
        which = np.array([j for j in kept[b][:max(count[b], 0)]], np.int64)
        to = T - nodes + np.arange(len(which))
        ok = (which >= 0) & (which < nodes)
        ok[ok] &= (T - nodes + which[ok] >= 0) & (to[ok] >= 0)
        write(b, to[ok], which[ok])
    return pools(cache, (kp, vp)), (kp, vp), flags


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("kf,vf", PAIRS)
def test_compact(memra, kf, vf, D):
    nodes, lens = 13, [13, 16, 40, 100, 29]
    rng = np.random.default_rng(D)
    kept = np.stack([np.sort(rng.permutation(nodes)[:6]) for _ in lens])
    count = [6, 0, 3, 6, 1]
    got, want, flags = compact_case(memra, kf, vf, D, 3, lens, nodes, kept, count, 5)
    assert flags == 0
    for g, w in zip(got, want):
        assert np.array_equal(g, w)


@pytest.mark.parametrize("nodes,most", [(1, 1), (2, 2), (64, 64), (64, 5), (17, 16)])
def test_compact_sizes(memra, nodes, most):
    lens = [nodes, nodes + 1, nodes + 15, nodes + 16, nodes + 300]
    rng = np.random.default_rng(nodes)
    kept = np.stack([np.sort(rng.permutation(nodes)[:most]) for _ in lens])
    got, want, flags = compact_case(memra, "q8_0", "q5_1", 128, 2, lens, nodes, kept, [most] * 5, nodes)
    assert flags == 0
    for g, w in zip(got, want):
        assert np.array_equal(g, w)


def test_compact_any_order_and_repeats(memra):
    # a permutation that swaps rows, and one row taken for all: each needs every read before any write
    kept = np.array([[3, 2, 1, 0], [3, 3, 3, 3], [1, 0, 3, 2]])
    got, want, flags = compact_case(memra, "fp8", "q5_1", 128, 2, [20, 30, 18], 4, kept, [4, 4, 4], 9)
    assert flags == 0
    for g, w in zip(got, want):
        assert np.array_equal(g, w)


def test_compact_flags(memra):
    # an index outside the tree, a count above the list, a negative count, a sequence shorter than the tree
    kept = np.array([[1, 6, -1, 5], [2, 3, 4, 5], [1, 2, 3, 4], [2, 5, 3, 4]])
    got, want, flags = compact_case(memra, "q8_0", "q4_0", 128, 2, [20, 30, 25, 3], 6, kept, [4, 9, -2, 4], 11)
    assert flags == memra.DEVERR_BAD_SLOT | memra.DEVERR_BAD_SEQ_LEN
    for g, w in zip(got, want):
        assert np.array_equal(g, w)


def test_compact_bad_pages_skip_their_rows(memra):
    cache, kp, vp = make_cache(memra, "q8_0", "q5_1", 4, 2, 128, 2)
    # nodes at positions 12..19: rows from the second page, whose id is bad, do not move
    memra.kv_compact(cache, dev([[1, 4]]), dev([20]), 20, dev([[4, 5]]), dev([2]), 8)
    assert memra.read_status(cache) == memra.DEVERR_BAD_PAGE
    for got, want in zip(pools(cache, (kp, vp)), (kp, vp)):
        assert np.array_equal(got, want)
    # a length past the table is clamped and flagged
    memra.kv_compact(cache, dev([[1]]), dev([40]), 64, dev([[0]]), dev([1]), 8)
    assert memra.read_status(cache) == memra.DEVERR_BAD_SEQ_LEN


def test_page_calls_captured_and_replayed(memra):
    cache, kp, vp = make_cache(memra, "q8_0", "q5_1", 8, 2, 128, 21)
    src, dst = dev([1]), dev([5])
    table, lens, kept, count = dev([[2, 3]]), dev([20]), dev([[2, 4]]), dev([2])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        memra.kv_copy_pages(cache, src, dst)
        memra.kv_compact(cache, table, lens, 20, kept, count, 6)
    for a, b in ((1, 5), (6, 7)):
        src.fill_(a), dst.fill_(b)
        before = pools(cache, (kp, vp))
        count.zero_()                              # the replay reads the lists anew
        g.replay()
        torch.cuda.synchronize()
        after = pools(cache, (kp, vp))
        for x, y in zip(before, after):
            x[b] = x[a]
            assert np.array_equal(x, y)
    assert memra.read_status(cache) == 0
