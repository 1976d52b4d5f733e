"""The operators around the decode step in the order a server uses them, against the oracle at every stage.

Two prompts are attended packed and appended to the cache; the first is forked
(its full pages shared, its partial last page copied); each of the three
sequences appends a tree of drafts and verifies it; the accepted branch is
compacted; a decode step follows on the new lengths.  Tolerances: 2e-3 as for
the decode calls (the fp16 rounding of the output, of the weights, and float32
sums) at values of order one.
"""
import numpy as np
import pytest

from oracle import attention, quant

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TOL = 2e-3


@pytest.fixture(scope="module")
def memra():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from decode_attention_block_memra_gb300 import _build
    _build.build()
    import decode_attention_block_memra_gb300 as m
    m.lib()
    return m


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def dequantized(rows, fmt, scale):
    """[T, Hkv, D] fp16 rows as the cache holds them, float64."""
    return np.stack([quant.dequantize_rows(quant.quantize_rows(rows[:, h], fmt, scale)) for h in range(rows.shape[1])], 1)


@pytest.mark.parametrize("kf,vf,D", [("q8_0", "q5_1", 128), ("fp8", "fp8", 256), ("nvfp4", "q4_0", 128)])
def test_prompt_fork_tree_compact_decode(memra, kf, vf, D):
    rng = np.random.default_rng(D)
    Hq, Hkv, N = 8, 2, 6
    lens = [70, 45]
    total = sum(lens)
    scale = D ** -0.5

    def normal(*shape):
        return rng.standard_normal(shape).astype(np.float16)

    # the prompts, packed in one fused buffer
    rows = normal(total, Hq + 2 * Hkv, D)
    fused = dev(rows)
    q, k, v = fused[:, :Hq], fused[:, Hq:Hq + Hkv], fused[:, Hq + Hkv:]
    out = torch.empty(total, Hq, D, dtype=torch.float16, device="cuda")
    memra.prompt_attn(q, k, v, dev(np.array([0, 70, 115], np.int32)), out)
    got = out.cpu().numpy().astype(np.float64)
    for a, b in ((0, 70), (70, 115)):
        want = attention.masked_rows(rows[a:b, :Hq], rows[a:b, Hq:Hq + Hkv], rows[a:b, Hq + Hkv:],
                                     attention.prompt_sees(b - a), scale)
        assert np.abs(got[a:b] - want).max() <= TOL

    # their rows into the cache
    ks, vs = (4.0 / 448 if f == "fp8" else 4.0 / 2688 if f == "nvfp4" else 1.0 for f in (kf, vf))
    pages, cols = 40, 8
    cache = memra.KVCache(kf, vf, pages, Hkv, D, ks, vs)
    free = list(rng.permutation(pages))
    table = np.zeros((3, cols), np.int32)
    for b, n in enumerate(lens):
        for c in range(-(-n // 16)):
            table[b, c] = free.pop()
    slots = np.concatenate([table[b, np.arange(n) // 16] * 16 + np.arange(n) % 16 for b, n in enumerate(lens)])
    memra.kv_append(cache, k.contiguous(), v.contiguous(), dev(slots.astype(np.int32)))
    held_k = [rows[:70, Hq:Hq + Hkv], rows[70:, Hq:Hq + Hkv]]
    held_v = [rows[:70, Hq + Hkv:], rows[70:, Hq + Hkv:]]

    # a fork of the first: full pages shared, the partial one copied
    full = 70 // 16
    table[2, :full] = table[0, :full]
    table[2, full] = free.pop()
    memra.kv_copy_pages(cache, dev(table[0:1, full]), dev(table[2:3, full]))
    held_k.append(held_k[0])
    held_v.append(held_v[0])
    lens = [70, 45, 70]

    # a tree of drafts each
    for b, n in enumerate(lens):
        for c in range(-(-n // 16), -(-(n + N + 1) // 16)):
            table[b, c] = free.pop()
    tk, tv, tq = normal(3, N, Hkv, D), normal(3, N, Hkv, D), normal(3, N, Hq, D)
    pos = np.stack([n + np.arange(N) for n in lens])
    slots = table[np.arange(3)[:, None], pos // 16] * 16 + pos % 16
    memra.kv_append(cache, dev(tk.reshape(-1, Hkv, D)), dev(tv.reshape(-1, Hkv, D)), dev(slots.reshape(-1).astype(np.int32)))
    words = np.array([0b000001, 0b000011, 0b000101, 0b001011, 0b010101, 0b101011], np.int64)     # two branches
    seq = np.array([n + N for n in lens], np.int32)
    longest = int(seq.max())
    ws = torch.empty(max(memra.tree_attn_workspace_bytes(3, N, Hq, D, longest), 16), dtype=torch.uint8, device="cuda")
    tree_out = torch.empty(3, N, Hq, D, dtype=torch.float16, device="cuda")
    memra.tree_attn(cache, dev(tq), dev(table), dev(seq), longest, dev(np.tile(words, (3, 1))), tree_out, ws)
    got = tree_out.cpu().numpy().astype(np.float64)
    for b in range(3):
        kh = dequantized(np.concatenate([held_k[b], tk[b]]), kf, ks)
        vh = dequantized(np.concatenate([held_v[b], tv[b]]), vf, vs)
        want = attention.masked_rows(tq[b], kh, vh, attention.tree_sees(words, lens[b]), scale)
        assert np.abs(got[b] - want).max() <= TOL

    # the accepted branches: nodes 0 1 3 5, 0 2 4, and the root alone
    kept = np.array([[0, 1, 3, 5], [0, 2, 4, 0], [0, 0, 0, 0]], np.int32)
    count = np.array([4, 3, 1], np.int32)
    memra.kv_compact(cache, dev(table), dev(seq), longest, dev(kept), dev(count), N)
    for b in range(3):
        path = kept[b, :count[b]]
        held_k[b] = np.concatenate([held_k[b], tk[b, path]])
        held_v[b] = np.concatenate([held_v[b], tv[b, path]])
    lens = [len(x) for x in held_k]

    # a plain decode step on what was kept
    sk, sv, sq = normal(3, 1, Hkv, D), normal(3, 1, Hkv, D), normal(3, 1, Hq, D)
    seq = np.array([n + 1 for n in lens], np.int32)
    longest = int(seq.max())
    ws = torch.empty(max(memra.decode_attn_workspace_bytes(3, 1, Hq, D, longest), 16), dtype=torch.uint8, device="cuda")
    step_out = torch.empty(3, 1, Hq, D, dtype=torch.float16, device="cuda")
    memra.decode_step(cache, dev(sk), dev(sv), dev(sq), dev(table), dev(seq), longest, step_out, ws)
    assert memra.read_status(cache) == 0
    got = step_out.cpu().numpy().astype(np.float64)
    for b in range(3):
        kh = dequantized(np.concatenate([held_k[b], sk[b]]), kf, ks)
        vh = dequantized(np.concatenate([held_v[b], sv[b]]), vf, vs)
        assert np.abs(got[b] - attention.attention_rows(sq[b], kh, vh, scale)).max() <= TOL


@pytest.mark.parametrize("D", [128, 256])
def test_tensor_memory_kernels_side_by_side(memra, D):
    """Prompt, tree and cascade calls on three streams at once, each with its own workspace: the same bytes as alone.

    All three hold tensor memory; none of their CTAs may wait for another kernel's that waits for it."""
    import workloads as W
    from decode_attention_block_memra_gb300.runner import upload
    g = torch.Generator(device="cuda").manual_seed(D)
    rows = torch.randn(3000, 12, D, device="cuda", generator=g).half()
    cu = torch.tensor([0, 1700, 1750, 3000], dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    w = W.make_workload("tree", batch=6, q_len=7, n_heads=16, n_kv_heads=2, head_dim=D, k_fmt="q8_0", v_fmt="q5_1",
                        seed=1, seq_lens=[900, 2000, 70, 3100, 1500, 400], permute_pages=True)
    c = W.make_workload("cascade", batch=6, q_len=1, n_heads=16, n_kv_heads=2, head_dim=D, k_fmt="q8_0", v_fmt="q5_1",
                        seed=2, seq_lens=[2100, 2300, 2031, 3100, 2025, 2400], shared_prefix=2016)
    dw, dc = upload(w), upload(c)
    for x in (dw, dc):
        memra.kv_append(x.cache, x.step_k, x.step_v, x.step_slots)
    mask = torch.full((6, 7), -1, dtype=torch.int64, device="cuda")

    def calls():
        outs = [torch.empty(3000, 8, D, dtype=torch.float16, device="cuda"), torch.empty_like(dw.q),
                torch.empty_like(dc.q)]
        sizes = (memra.tree_attn_workspace_bytes(6, 7, 16, D, w.max_seq_len),
                 memra.decode_attn_cascade_workspace_bytes(6, 1, 16, D, c.max_seq_len, 2016))
        tws, cws = (torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes)
        return outs, (
            lambda s: memra.prompt_attn(rows[:, :8], rows[:, 8:10], rows[:, 10:], cu, outs[0], status=status, stream=s),
            lambda s: memra.tree_attn(dw.cache, dw.q, dw.page_table, dw.seq_lens, w.max_seq_len, mask, outs[1], tws,
                                      stream=s),
            lambda s: memra.decode_attn_cascade(dc.cache, dc.q, dc.page_table, dc.seq_lens, c.max_seq_len, 2016, outs[2],
                                                cws, stream=s))

    want, alone = calls()
    for call in alone:
        call(None)
        torch.cuda.synchronize()
    got, together = calls()
    streams = [torch.cuda.Stream() for _ in together]
    torch.cuda.synchronize()
    for _ in range(30):
        for call, s in zip(together, streams):
            call(s)
    torch.cuda.synchronize()
    for _ in range(30):                                  # and behind one another on one stream, early launches overlapping
        for call in together:
            call(streams[0])
    torch.cuda.synchronize()
    assert int(status) == 0 and memra.read_status(dw.cache) == 0 and memra.read_status(dc.cache) == 0
    for a, b in zip(got, want):
        assert torch.equal(a, b)
