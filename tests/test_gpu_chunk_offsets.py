"""The operators for chunks on rows and weights that lie more than 2^31 elements into their tensors: the bytes of a small call."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from chunk_cases import dev     # noqa: E402
from test_gpu_evict import Case     # noqa: E402
from test_gpu_key_weights import Weights, memra     # noqa: E402, F401

T, HEADS, D = 66000, 128, 256                # T * HEADS * D passes 2^31
STRIDE = 2 ** 28 + 8                         # so do the last of 16 rows of weights


@pytest.fixture
def far_rows():
    assert T * HEADS * D > 2 ** 31
    x = torch.zeros(T, HEADS, D, dtype=torch.float16, device="cuda")
    yield x
    del x
    torch.cuda.empty_cache()


def test_rows(memra, far_rows):     # noqa: F811
    rng, n = np.random.default_rng(0), 5
    far_rows[-n:] = dev(rng.standard_normal((n, HEADS, D)).astype(np.float16))
    far_rows[:n] = far_rows[-n:]
    pos, freq = torch.arange(T, dtype=torch.int32, device="cuda"), dev((1e4 ** (-np.arange(64) / 64)).astype(np.float32))
    pos[:n] = pos[-n:]
    w = dev((1 + 0.2 * rng.standard_normal(D)).astype(np.float32))
    want = torch.empty_like(far_rows[:n, :96])
    memra.qk_norm_rope(far_rows[-n:, :96].clone(), None, pos[-n:], freq, want, q_weight=w)
    # in place on a part of the heads; keys and values are the heads behind
    cache = memra.KVCache("q8_0", "q5_1", T // 16 + 1, 2, D)
    q, k, v = far_rows[:, :96], far_rows[:, 96:98], far_rows[:, 98:100]
    slots = torch.arange(T, dtype=torch.int32, device="cuda")
    memra.qk_norm_rope(q, k, pos, freq, q, None, w, w, cache=cache, v=v, slot_mapping=slots)
    assert memra.read_status(cache) == 0
    assert torch.equal(far_rows[-n:, :96], want) and torch.equal(far_rows[:n, :96], want)
    small = memra.KVCache("q8_0", "q5_1", T // 16 + 1, 2, D)
    memra.qk_norm_rope(far_rows[-n:, :1].clone(), k[-n:], pos[-n:], freq, torch.empty_like(far_rows[-n:, :1]), None, None, w,
                       cache=small, v=v[-n:], slot_mapping=slots[-n:])
    last = (T - n) // 16 + 1                 # (the last page, which holds the last tokens alone)
    for a, b in ((cache.k_pool, small.k_pool), (cache.v_pool, small.v_pool)):
        assert torch.equal(a.view(T // 16 + 1, -1)[last:], b.view(T // 16 + 1, -1)[last:])


def test_chunks_and_their_weights(memra, far_rows):     # noqa: F811
    c = Weights(memra, "fp8", "q5_1", D, HEADS, 8, [7, 3], [300, 900])
    n = 10
    a = c.args()
    memra.chunk_attn(c.cache, **a)
    want, want_lse = c.out.clone(), c.lse.clone()
    c.weights.zero_()
    assert c.call(lse=want_lse) == 0
    want_weights = c.weights.clone()
    far_rows[-n:] = c.buf
    out, lse = torch.zeros_like(far_rows), torch.zeros(T, HEADS, device="cuda")
    a.update(q=far_rows, out=out, lse=lse, cu_seqlens=a["cu_seqlens"] + (T - n))
    memra.chunk_attn(c.cache, **a)
    assert memra.read_status(c.cache) == 0
    assert torch.equal(out[-n:], want) and torch.equal(lse[-n:], want_lse)
    assert not out[:100].any() and not out[-n - 100:-n].any()
    del out
    weights = torch.zeros(2, 8, STRIDE, device="cuda")
    assert weights.numel() > 2 ** 31
    assert c.call(q=far_rows, lse=lse, cu_seqlens=a["cu_seqlens"], weights=weights) == 0
    assert torch.equal(weights[..., :want_weights.shape[2]], want_weights)
    assert not weights[..., want_weights.shape[2]:want_weights.shape[2] + 1000].any()


def test_evictions(memra):     # noqa: F811
    c = Case(memra, "fp8", "fp8", 128, 8, [3000, 900], [700, 500], 2, 9)
    weights, new = torch.zeros(2, 8, STRIDE, device="cuda"), torch.full((2, 8, STRIDE), -5.0, device="cuda")
    weights[..., :3000] = dev(c.weights)
    assert c.call(weights=weights, new_weights=new) == 0
    c.new_w.copy_(new[..., :c.new_w.shape[2]])
    c.check()
    assert (new[..., c.new_w.shape[2]:c.new_w.shape[2] + 1000] == -5).all()
    del weights, new
    torch.cuda.empty_cache()
