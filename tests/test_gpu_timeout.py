"""The bounded-wait path of the split kernel, driven on the GPU without a fault.

Every pipeline wait of the library is bounded; past the bound the kernel flags
MEMRA_DEVERR_TIMEOUT, waits (bounded) for the copies it issued itself, and
returns.  The test hook of memra_testing.h makes one wait certain to run out:
the first CTA's first page expects 16 bytes more than its copies deliver, and
the page waits give up after a few milliseconds.  Nothing is left in flight
(the short page's copies have landed; only its phase never completes), so the
next call on the same process must be exact again.
"""
import time

import numpy as np
import pytest

import workloads as W
from oracle import attention

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def memra():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from decode_attention_block_memra_gb300 import _build
    _build.build()
    import decode_attention_block_memra_gb300 as m
    m.lib()
    return m


def test_a_wait_that_runs_out_is_flagged_and_the_next_call_is_exact(memra):
    from decode_attention_block_memra_gb300.runner import upload
    w = W.random_case(71, batch=2, q_len=1, n_heads=16, n_kv_heads=2, head_dim=128, ctx=(1500, 3000))
    dw = upload(w, fill_seed=3)
    dw.step()                                         # the step's rows are appended
    assert memra.read_status(dw.cache) == 0
    pools = (dw.cache.k_pool.clone(), dw.cache.v_pool.clone())
    ref = attention.reference(w)

    t0 = time.monotonic()
    memra.testing_decode_attn_short_page(dw.cache, dw.q, dw.page_table, dw.seq_lens, w.max_seq_len, dw.out,
                                         dw.workspace, page_wait_ns=2_000_000, sm_scale=w.sm_scale)
    flags = memra.read_status(dw.cache)              # synchronizes: the call has returned
    elapsed = time.monotonic() - t0
    assert flags & memra.DEVERR_TIMEOUT, f"flags 0x{flags:x}"
    assert elapsed < 30.0
    assert torch.equal(pools[0], dw.cache.k_pool) and torch.equal(pools[1], dw.cache.v_pool)

    # the same process, the same buffers: a normal call is exact and flags nothing
    dw.out.fill_(float("nan"))
    memra.decode_attn(dw.cache, dw.q, dw.page_table, dw.seq_lens, w.max_seq_len, dw.out, dw.workspace, w.sm_scale)
    assert memra.read_status(dw.cache) == 0
    err = np.abs(dw.out.cpu().numpy().astype(np.float64) - ref).max()
    assert err <= 2e-3, err


def test_the_hook_rejects_limits_outside_its_range(memra):
    from decode_attention_block_memra_gb300.runner import upload
    w = W.random_case(72, batch=1, q_len=1, n_heads=8, n_kv_heads=2, head_dim=128, ctx=(40, 80))
    dw = upload(w)
    for bad in (0, 2_000_000_000):
        with pytest.raises(memra.MemraError) as e:
            memra.testing_decode_attn_short_page(dw.cache, dw.q, dw.page_table, dw.seq_lens, w.max_seq_len,
                                                 dw.out, dw.workspace, page_wait_ns=bad)
        assert e.value.status == 1
    assert memra.read_status(dw.cache) == 0


@pytest.mark.parametrize("D,n", [(128, 100), (128, 1500), (256, 40), (256, 1500)])
def test_prompt_rows_of_a_wait_that_runs_out_are_nan(memra, D, n):
    """The last piece of the first prompt, first KV head (2 x 32 tokens of four heads at head_dim 128, 32 at 256): NaN;
    every other row as always; the next call exact."""
    g = torch.Generator(device="cuda").manual_seed(n)
    rows = torch.randn(n + 90, 12, D, device="cuda", generator=g).half()
    q, k, v = rows[:, :8], rows[:, 8:10], rows[:, 10:]
    cu = torch.tensor([0, n, n + 90], dtype=torch.int32, device="cuda")
    want, out = (torch.empty(n + 90, 8, D, dtype=torch.float16, device="cuda") for _ in range(2))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    memra.prompt_attn(q, k, v, cu, want, status=status)
    assert int(status) == 0
    t0 = time.monotonic()
    memra.testing_prompt_attn_short_copy(q, k, v, cu, out, status=status)
    assert int(status) == memra.DEVERR_TIMEOUT
    assert time.monotonic() - t0 < 30.0
    piece = 64 if D == 128 else 32
    lost = torch.zeros(n + 90, 8, dtype=torch.bool, device="cuda")
    lost[(n - 1) // piece * piece:n, :4] = True
    assert bool(torch.isnan(out[lost]).all()) and torch.equal(out[~lost], want[~lost])
    status.zero_()
    memra.prompt_attn(q, k, v, cu, out, status=status)
    assert int(status) == 0 and torch.equal(out, want)


@pytest.mark.parametrize("D,nodes,ctx", [(128, 9, 200), (128, 9, 2600), (128, 40, 200), (128, 40, 2600), (256, 9, 200),
                                         (256, 9, 2600), (256, 40, 2600)])
def test_tree_rows_of_a_wait_that_runs_out_are_nan(memra, D, nodes, ctx):
    """The first sequence's first split, first KV head (four heads; 32 nodes a row tile, two of them at head_dim 128):
    its rows are NaN, also where other splits of theirs are whole; every other row as always; the next call exact."""
    from decode_attention_block_memra_gb300.runner import upload
    w = W.random_case(80 + D, batch=2, q_len=nodes, n_heads=8, n_kv_heads=2, head_dim=D, ctx=(ctx - 30, ctx))
    dw = upload(w)
    memra.kv_append(dw.cache, dw.step_k, dw.step_v, dw.step_slots)
    words = torch.tril(torch.ones(nodes, nodes, dtype=torch.int64)) @ (1 << torch.arange(nodes))
    mask = words.expand(2, nodes).contiguous().cuda()
    ws = torch.empty(memra.tree_attn_workspace_bytes(2, nodes, 8, D, w.max_seq_len), dtype=torch.uint8, device="cuda")
    args = (dw.cache, dw.q, dw.page_table, dw.seq_lens, w.max_seq_len, mask)
    want, out = torch.empty_like(dw.q), torch.empty_like(dw.q)
    memra.tree_attn(*args, want, ws)
    assert memra.read_status(dw.cache) == 0 and bool(torch.isfinite(want).all())
    t0 = time.monotonic()
    memra.testing_tree_attn_short_page(*args, out, ws)
    assert memra.read_status(dw.cache) == memra.DEVERR_TIMEOUT
    assert time.monotonic() - t0 < 30.0
    lost = torch.zeros(2, nodes, 8, dtype=torch.bool, device="cuda")
    lost[0, :64 if D == 128 else 32, :4] = True
    assert bool(torch.isnan(out[lost]).all()) and torch.equal(out[~lost], want[~lost])
    memra.tree_attn(*args, out, ws)
    assert memra.read_status(dw.cache) == 0 and torch.equal(out, want)
