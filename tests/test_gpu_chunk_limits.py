"""The operators for chunks at the header's limits: 65,535 KV heads, 65,535 sequences, and as many rows of weights.

Heads and sequences repeat a few: every one has the results of the one that it repeats (of a call with those few alone, up to
the order of its sums: chunk attention cuts its keys by the whole call).
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from chunk_cases import dev     # noqa: E402
from oracle import chunked, quant     # noqa: E402
from test_gpu_key_weights import memra     # noqa: E402, F401
from test_gpu_norm_rope import check as check_rows     # noqa: E402

MOST, SOME = 65535, 5


def held(rows, fmt):
    return np.stack([quant.dequantize_rows(quant.quantize_rows(np.ascontiguousarray(rows[:, h]), fmt, 1.0))
                     for h in range(rows.shape[1])], 1)


@pytest.mark.parametrize("D", [128, 256])
def test_heads(memra, D):     # noqa: F811
    rng, n, past = np.random.default_rng(D), 3, 40
    T = n + past
    rows = rng.standard_normal((3, T, SOME, D)).astype(np.float16)
    heads = torch.arange(MOST, device="cuda") % SOME
    q, k, v = (dev(x)[:, heads].contiguous() for x in rows)
    freq = (1e4 ** (-np.arange(D // 2) / (D // 2))).astype(np.float32)
    cache = memra.KVCache("q8_0", "q5_1", 4, MOST, D)
    table = torch.tensor([[2, 0, 3]], dtype=torch.int32, device="cuda")
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    slots = (table[0].long()[pos.long() // 16] * 16 + pos.long() % 16).int()
    k_out = torch.empty_like(k)
    memra.qk_norm_rope(q, k, pos, dev(freq), q, k_out, cache=cache, v=v, slot_mapping=slots)
    assert memra.read_status(cache) == 0
    for got, x in ((q, rows[0]), (k_out, rows[1])):
        check_rows(got[:, :SOME], x, None, pos.cpu().numpy(), freq, False)
        assert torch.equal(got, got[:, :SOME][:, heads])
    pool = cache.k_pool.view(4, MOST, -1)
    assert torch.equal(pool[[0, 2, 3]], pool[[0, 2, 3], :SOME][:, heads])
    starts, lens = dev(np.array([0, n], np.int32)), dev(np.array([T], np.int32))
    out, lse = torch.empty(n, MOST, D, dtype=torch.float16, device="cuda"), torch.empty(n, MOST, device="cuda")
    ws = torch.empty(memra.chunk_attn_workspace_bytes(D), dtype=torch.uint8, device="cuda")
    memra.chunk_attn(cache, q[past:], starts, table, lens, T, out, ws, lse=lse)
    weights = torch.zeros(1, MOST, T, device="cuda")
    memra.key_weights(cache, q[past:], lse, starts, table, lens, T, weights)
    assert memra.read_status(cache) == 0
    few, kh, vh = q[past:, :SOME].cpu().numpy(), held(k_out[:, :SOME].cpu().numpy(), "q8_0"), held(rows[2], "q5_1")
    want, want_lse = chunked.chunk_rows(few, kh, vh, 0, D ** -0.5)
    assert np.abs(out[:, :SOME].cpu().numpy() - want).max() <= 2e-3
    assert (out.float() - out[:, :SOME][:, heads].float()).abs().max() <= 2e-3
    assert (lse - dev(want_lse.astype(np.float32))[:, heads]).abs().max() <= 1e-4
    want = dev(chunked.key_weights(few, kh, want_lse, D ** -0.5).astype(np.float32))
    assert (weights[0] - want[heads]).abs().max() <= 1e-3


def test_sequences(memra):     # noqa: F811
    D, rng = 128, np.random.default_rng(1)
    lens5 = [1, 15, 16, 17, 30]
    rows = rng.standard_normal((2, SOME, 32, D)).astype(np.float16)
    cache = memra.KVCache("fp8", "fp8", 2 * MOST, 1, D, 5 / 448, 5 / 448)
    which = torch.arange(MOST, device="cuda") % SOME
    table = torch.randperm(2 * MOST, device="cuda", generator=torch.Generator("cuda").manual_seed(0)).int().view(MOST, 2)
    for i in range(32):                      # every page full: what lies behind a sequence's length is not seen
        memra.kv_append(cache, dev(rows[0, :, i])[which][:, None].contiguous(), dev(rows[1, :, i])[which][:, None].contiguous(),
                        (table[:, i // 16] * 16 + i % 16).contiguous())
    q = dev(rng.standard_normal((SOME, 2, D)).astype(np.float16))
    lens, starts = dev(np.array(lens5, np.int32))[which].contiguous(), torch.arange(MOST + 1, dtype=torch.int32, device="cuda")
    out, lse = torch.empty(MOST, 2, D, dtype=torch.float16, device="cuda"), torch.empty(MOST, 2, device="cuda")
    ws = torch.empty(memra.chunk_attn_workspace_bytes(D), dtype=torch.uint8, device="cuda")
    memra.chunk_attn(cache, q[which].contiguous(), starts, table, lens, 30, out, ws, lse=lse)
    weights = torch.zeros(MOST, 1, 32, device="cuda")
    memra.key_weights(cache, q[which].contiguous(), lse, starts, table, lens, 30, weights)
    assert memra.read_status(cache) == 0
    for s, T in enumerate(lens5):
        k, v = (quant.dequantize_rows(quant.quantize_rows(rows[i, s, :T], "fp8", float(np.float32(5 / 448))))[:, None] for i in (0, 1))
        want, want_lse = chunked.chunk_rows(q[s:s + 1].cpu().numpy(), k, v, 0, D ** -0.5)
        assert np.abs(out[s].cpu().numpy() - want[0]).max() <= 2e-3 and np.abs(lse[s].cpu().numpy() - want_lse[0]).max() <= 1e-4
        w = chunked.key_weights(q[s:s + 1].cpu().numpy(), k, want_lse, D ** -0.5)
        assert np.abs(weights[s, 0, :T].cpu().numpy() - w[0]).max() <= 1e-4 and not weights[s, 0, T:].any()
    assert (out.float() - out[:SOME][which].float()).abs().max() <= 2e-3
    assert torch.equal(weights, weights[:SOME][which])
    # to 7 tokens each, in pages of another cache's pools (the kept rows go behind the present ones)
    big = memra.KVCache("fp8", "fp8", 3 * MOST, 1, D, 5 / 448, 5 / 448)
    big.k_pool[:cache.k_pool.numel()], big.v_pool[:cache.v_pool.numel()] = cache.k_pool, cache.v_pool
    to = (torch.arange(MOST, dtype=torch.int32, device="cuda") + 2 * MOST).view(MOST, 1)
    kept, budgets = torch.empty(MOST, 1, 7, dtype=torch.int32, device="cuda"), torch.full((MOST,), 7, dtype=torch.int32, device="cuda")
    new, new_lens = torch.zeros(MOST, 1, 7, device="cuda"), torch.empty(MOST, dtype=torch.int32, device="cuda")
    memra.kv_evict(big, table, lens, 32, weights, budgets, to, kept, 1, 2, new_weights=new, new_lens=new_lens)
    assert memra.read_status(big) == 0
    for s, T in enumerate(lens5):
        rows_kept = chunked.kept_tokens(weights[s, 0, :T].cpu().numpy(), min(7, T), 1, 2)
        assert kept[s, 0].tolist() == list(rows_kept) + [-1] * (7 - len(rows_kept)) and new_lens[s] == min(7, T)
    assert torch.equal(kept, kept[:SOME][which]) and torch.equal(new_lens, new_lens[:SOME][which])
    pool = big.v_pool.view(3 * MOST, -1)[2 * MOST:]
    assert torch.equal(pool, pool[:SOME][which]) and torch.equal(new, new[:SOME][which])
