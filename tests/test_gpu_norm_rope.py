"""Norm, rotation and append of rows on the GPU, against float64.

Tolerance of a value y of a pair (a, b): the rounding to fp16, 2^-11 |y| (2^-25 below the normal range);
and in float32 the norm's factor and weight (sum of squares, root, quotient, two products: under 12 roundings
of 2^-24, a rounding in the sum counted half), the sine and cosine (2 ulps and an angle off by 2^-25 turns, that is 2^-22.3)
and the two products and the sum: under 16 * 2^-24 + 2^-22 + 2^-22.3 < 2^-19 of |a| + |b|.
The stored bytes are compared with those that kv_append makes of the rounded rows: equal.
"""
import numpy as np
import pytest

from oracle import chunked

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

EPS = 1e-6


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


def case(T, Hq, Hkv, D, rotary, seed=0, positions=None):
    rng = np.random.default_rng(seed)
    rows = rng.standard_normal((T, Hq + 2 * Hkv, D)).astype(np.float16)
    pos = rng.integers(0, 262144, T) if positions is None else positions
    freq = (1e6 ** (-np.arange(rotary // 2) / max(1, rotary // 2))).astype(np.float32) if rotary else None
    qw, kw = ((1 + 0.2 * rng.standard_normal(D)).astype(np.float32) for _ in range(2))
    return rows, np.asarray(pos, np.int32), freq, qw, kw


def check(got, x, weight, pos, freq, interleaved):
    want = chunked.norm_rope_rows(x, weight, EPS, pos, freq, interleaved)
    a = np.abs(chunked.norm_rope_rows(x, weight, EPS, None, None, interleaved))
    room = a.copy()
    if freq is not None:
        first, second = chunked.rope_pairs(len(freq), interleaved)
        room[..., first] = room[..., second] = a[..., first] + a[..., second]
    tol = np.abs(want) * 2.0 ** -11 + 2.0 ** -25 + room * 2.0 ** -19
    err = np.abs(got.cpu().numpy().astype(np.float64) - want)
    assert (err <= tol).all(), f"worst {np.max(err / tol)} of the tolerance"


@pytest.mark.parametrize("T,Hq,Hkv", [(1, 1, 1), (1, 32, 4), (3, 5, 3), (33, 8, 2), (700, 12, 4), (2600, 3, 1)])
@pytest.mark.parametrize("D,rotary", [(128, 128), (128, 32), (256, 256), (256, 64), (128, 0), (256, 16)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rows(memra, T, Hq, Hkv, D, rotary, interleaved):
    rows, pos, freq, qw, kw = case(T, Hq, Hkv, D, rotary, seed=T)
    fused = dev(rows)
    q_out = torch.full((T, Hq, D), float("nan"), dtype=torch.float16, device="cuda")
    k_out = torch.full((T, Hkv, D), float("nan"), dtype=torch.float16, device="cuda")
    memra.qk_norm_rope(fused[:, :Hq], fused[:, Hq:Hq + Hkv], dev(pos) if rotary else None, dev(freq) if rotary else None,
                       q_out, k_out, dev(qw), dev(kw), EPS, interleaved)
    check(q_out, rows[:, :Hq], qw, pos, freq, interleaved)
    check(k_out, rows[:, Hq:Hq + Hkv], kw, pos, freq, interleaved)


def test_far_and_negative_positions(memra):
    pos = [0, 1, -1, -262143, 262143, 2 ** 20, -2 ** 20, 1000003]
    rows, pos, freq, qw, kw = case(len(pos), 4, 2, 128, 128, positions=pos)
    fused = dev(rows)
    for interleaved in (False, True):
        q_out = torch.empty(len(pos), 4, 128, dtype=torch.float16, device="cuda")
        memra.qk_norm_rope(fused[:, :4], None, dev(pos), dev(freq), q_out, interleaved=interleaved)
        check(q_out, rows[:, :4], None, pos, freq, interleaved)


def test_position_zero_and_no_norm_copy_the_rows(memra):
    rows, _, freq, _, _ = case(9, 3, 2, 256, 64)
    rows[0, 0, :4] = [0.0, -0.0, 6e-8, 65504.0]
    fused = dev(rows)
    for pos, f in ((dev(np.zeros(9, np.int32)), dev(freq)), (None, None)):
        q_out, k_out = (torch.empty(9, h, 256, dtype=torch.float16, device="cuda") for h in (3, 2))
        memra.qk_norm_rope(fused[:, :3], fused[:, 3:5], pos, f, q_out, k_out)
        assert torch.equal(q_out, fused[:, :3]) and torch.equal(k_out, fused[:, 3:5])


def test_in_place_on_a_fused_buffer(memra):
    T, Hq, Hkv, D = 50, 6, 2, 128
    rows, pos, freq, qw, kw = case(T, Hq, Hkv, D, D)
    fused = dev(rows)
    q, k = fused[:, :Hq], fused[:, Hq:Hq + Hkv]
    memra.qk_norm_rope(q, k, dev(pos), dev(freq), q, k, dev(qw), dev(kw), EPS)
    check(q, rows[:, :Hq], qw, pos, freq, False)
    check(k, rows[:, Hq:Hq + Hkv], kw, pos, freq, False)
    assert np.array_equal(fused[:, Hq + Hkv:].cpu().numpy(), rows[:, Hq + Hkv:])


@pytest.mark.parametrize("weights", [(True, False), (False, True)])
def test_norm_of_one_side(memra, weights):
    rows, pos, freq, qw, kw = case(20, 4, 4, 128, 128)
    fused = dev(rows)
    qw, kw = (w if on else None for w, on in zip((qw, kw), weights))
    q_out, k_out = (torch.empty(20, 4, 128, dtype=torch.float16, device="cuda") for _ in range(2))
    memra.qk_norm_rope(fused[:, :4], fused[:, 4:8], dev(pos), dev(freq), q_out, k_out,
                       None if qw is None else dev(qw), None if kw is None else dev(kw), EPS)
    check(q_out, rows[:, :4], qw, pos, freq, False)
    check(k_out, rows[:, 4:8], kw, pos, freq, False)


def test_large_and_small_rows(memra):
    rows, pos, freq, qw, kw = case(6, 2, 2, 128, 128)
    rows[:2] *= np.float16(6000)
    rows[2:4] *= np.float16(1e-4)
    rows[4] = 0
    fused = dev(rows)
    q_out = torch.empty(6, 2, 128, dtype=torch.float16, device="cuda")
    memra.qk_norm_rope(fused[:, :2], None, dev(pos), dev(freq), q_out, q_weight=dev(qw), eps=EPS)
    check(q_out, rows[:, :2], qw, pos, freq, False)
    assert not q_out[4].any()


@pytest.mark.parametrize("norm,rotary,interleaved", [(False, 128, False), (False, 32, True), (False, 0, False), (True, 128, False),
                                                     (True, 0, True)])
def test_infinite_and_nan_elements_of_keys_as_of_queries(memra, norm, rotary, interleaved):
    rows, pos, freq, qw, _ = case(8, 1, 1, 128, rotary, positions=np.arange(8) * 1000)
    for t, x in enumerate((np.inf, -np.inf, np.nan, 65504.0)):
        rows[t, :, 5] = x
        rows[t + 4, :, [5, 69, 120]] = x
    x, w = dev(rows), dev(qw) if norm else None
    q_out, k_out = (torch.empty(8, 1, 128, dtype=torch.float16, device="cuda") for _ in range(2))
    memra.qk_norm_rope(x[:, :1], x[:, :1], dev(pos), None if freq is None else dev(freq), q_out, k_out, w, w, EPS, interleaved)
    assert torch.equal(q_out.isnan(), k_out.isnan())
    assert torch.equal(q_out.isinf(), k_out.isinf()) and torch.equal(q_out[q_out.isinf()], k_out[q_out.isinf()])
    assert q_out.isnan()[2].any() and not q_out.isnan()[3].any() and (norm or q_out.isinf()[0].any())


PAIRS = [("q8_0", "q5_1"), ("q8_0", "q4_0"), ("fp8", "fp8"), ("nvfp4", "nvfp4"), ("fp8", "q5_1"), ("nvfp4", "q4_0")]


@pytest.mark.parametrize("kf,vf", PAIRS)
@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("T,Hq,Hkv", [(1, 4, 1), (5, 3, 3), (40, 8, 2), (650, 4, 2)])
@pytest.mark.parametrize("with_rows", [False, True])
def test_append_stores_the_bytes_of_kv_append(memra, kf, vf, D, T, Hq, Hkv, with_rows):
    rows, pos, freq, qw, kw = case(T, Hq, Hkv, D, D // 2, seed=T)
    fused = dev(rows)
    q, k, v = fused[:, :Hq], fused[:, Hq:Hq + Hkv], fused[:, Hq + Hkv:]
    rng = np.random.default_rng(1)
    pages = -(-T // 16) + 3
    slots = rng.permutation(pages * 16)[:T].astype(np.int32)
    slots[T // 2:T // 2 + 1] = -3 if T > 1 else slots[0]
    fills = [torch.from_numpy(rng.integers(0, 256, memra.kv_pool_bytes(f, side, pages, Hkv, D), dtype=np.uint8)).cuda()
             for f, side in ((kf, False), (vf, True))]
    ours, theirs = (memra.KVCache(kf, vf, pages, Hkv, D, 0.02, 0.02, k_pool=fills[0].clone(), v_pool=fills[1].clone())
                    for _ in range(2))
    q_out, k_out = (torch.empty(T, h, D, dtype=torch.float16, device="cuda") for h in (Hq, Hkv))
    memra.qk_norm_rope(q, k, dev(pos), dev(freq), q_out, k_out if with_rows else None, dev(qw), dev(kw), EPS, False,
                       cache=ours, v=v, slot_mapping=dev(slots))
    assert memra.read_status(ours) == 0
    check(q_out, rows[:, :Hq], qw, pos, freq, False)
    plain_q, plain_k = torch.empty_like(q_out), torch.empty_like(k_out)
    memra.qk_norm_rope(q, k, dev(pos), dev(freq), plain_q, plain_k, dev(qw), dev(kw), EPS)
    assert torch.equal(plain_q, q_out) and (not with_rows or torch.equal(plain_k, k_out))
    memra.kv_append(theirs, plain_k, v.contiguous(), dev(slots))
    assert torch.equal(ours.k_pool, theirs.k_pool) and torch.equal(ours.v_pool, theirs.v_pool)


def test_slots_past_the_pool_are_skipped_and_flagged(memra):
    rows, pos, freq, _, _ = case(4, 2, 2, 128, 128)
    fused = dev(rows)
    cache = memra.KVCache("q8_0", "q5_1", 3, 2, 128)
    q_out = torch.empty(4, 2, 128, dtype=torch.float16, device="cuda")
    slots = np.array([48, 2 ** 31 - 1, -2 ** 31, 7], np.int32)
    memra.qk_norm_rope(fused[:, :2], fused[:, 2:4], dev(pos), dev(freq), q_out, cache=cache, v=fused[:, 4:],
                       slot_mapping=dev(slots))
    assert memra.read_status(cache) == memra.DEVERR_BAD_SLOT
    check(q_out, rows[:, :2], None, pos, freq, False)
    pool = cache.k_pool.view(3, -1)
    assert pool[0].any() and not pool[1:].any()


def test_refusals_of_the_binding(memra):
    q = torch.zeros(4, 2, 128, dtype=torch.float16, device="cuda")
    freq, pos = torch.ones(64, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda")
    good = dict(q=q, k=q.clone(), positions=pos, inv_freq=freq, q_out=torch.empty_like(q), k_out=torch.empty_like(q))
    memra.qk_norm_rope(**good)
    for bad in (dict(q=q.float()), dict(k=q[:3]), dict(k_out=None), dict(k=None), dict(q_out=q[:, :1]),
                dict(positions=pos.long()), dict(positions=pos[:3]), dict(inv_freq=freq.double()), dict(inv_freq=freq[:60]),
                dict(positions=None), dict(q_weight=torch.ones(64, device="cuda")), dict(v=q), dict(slot_mapping=pos),
                dict(q=q.cpu()), dict(q=q.transpose(0, 2).contiguous().transpose(0, 2)), dict(eps=-1.0), dict(eps=float("nan")),
                dict(cache=memra.KVCache("q8_0", "q5_1", 2, 2, 128)),
                dict(cache=memra.KVCache("q8_0", "q5_1", 2, 3, 128), v=q, slot_mapping=pos)):
        with pytest.raises(memra.MemraError):
            memra.qk_norm_rope(**{**good, **bad})
    none = torch.empty(0, 2, 128, dtype=torch.float16, device="cuda")
    memra.qk_norm_rope(none, none, pos[:0], freq, none, none)


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("stored", [False, True])
def test_keys_are_rounded_once(memra, D, stored):
    """Normalized keys are the fp16 values next to the exact ones: 2 to 4 million of them, of which some 120 to 250 lie so close
    to the middle of two that float32 is the middle.  (numpy rounds float64 to fp16 once; the sums of two floats are off by 2^-45,
    so that one of these keys would differ by chance once in 8,000 runs of other inputs.)"""
    T, rng = 4096, np.random.default_rng(D)
    x = rng.standard_normal((T, 4, D)).astype(np.float16)
    w = (1 + 0.2 * rng.standard_normal(D)).astype(np.float32)
    k_out = torch.empty(T, 4, D, dtype=torch.float16, device="cuda")
    cache = memra.KVCache("fp8", "fp8", T // 16, 4, D, 0.02, 0.02) if stored else None
    memra.qk_norm_rope(dev(x), dev(x), None, None, torch.empty_like(k_out), k_out, None, dev(w), EPS, cache=cache,
                       v=dev(x) if stored else None, slot_mapping=dev(np.arange(T, dtype=np.int32)) if stored else None)
    want = chunked.norm_rope_rows(x, w, EPS, None, None, False).astype(np.float16)
    assert np.array_equal(k_out.cpu().numpy().view(np.uint16), want.view(np.uint16))
    if stored:
        plain = memra.KVCache("fp8", "fp8", T // 16, 4, D, 0.02, 0.02)
        memra.kv_append(plain, dev(want), dev(x), dev(np.arange(T, dtype=np.int32)))
        assert torch.equal(cache.k_pool, plain.k_pool) and torch.equal(cache.v_pool, plain.v_pool)


@pytest.mark.parametrize("D,rotary", [(128, 128), (256, 256), (256, 64)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_turned_keys_fall_to_the_right_side(memra, D, rotary, interleaved):
    """A turned key is the fp16 value next to the exact one, but where the exact one lies within 2^-32 (|a| + |b|) of the middle of two:
    sine and cosine are off by 2^-33, angles below 1,000 turns by 2^-43 turns, the sums of two floats by 2^-45."""
    T, rng = 4096, np.random.default_rng(D + rotary)
    x = rng.standard_normal((T, 4, D)).astype(np.float16)
    w = (1 + 0.2 * rng.standard_normal(D)).astype(np.float32)
    pos = rng.integers(0, 1000, T).astype(np.int32)
    freq = (1e4 ** (-np.arange(rotary // 2) / (rotary // 2))).astype(np.float32)
    k_out = torch.empty(T, 4, D, dtype=torch.float16, device="cuda")
    memra.qk_norm_rope(dev(x), dev(x), dev(pos), dev(freq), torch.empty_like(k_out), k_out, None, dev(w), EPS, interleaved)
    exact = chunked.norm_rope_rows(x, w, EPS, pos, freq, interleaved)
    a = np.abs(chunked.norm_rope_rows(x, w, EPS, None, None, interleaved))
    first, second = chunked.rope_pairs(rotary // 2, interleaved)
    a[..., first] = a[..., second] = a[..., first] + a[..., second]
    want, got = exact.astype(np.float16), k_out.cpu().numpy()
    other = got != want
    assert other.sum() <= 10                 # (by chance one in 2^21)
    near = np.abs(exact[other] - (got[other].astype(np.float64) + want[other].astype(np.float64)) / 2)
    assert (near <= 2.0 ** -32 * a[other]).all()


def test_many_calls_in_a_row_and_side_by_side(memra):
    calls, outs, want = [], [], []
    for i, (T, Hq, Hkv, D) in enumerate(((7, 8, 2, 128), (300, 4, 2, 256), (2600, 3, 1, 128))):
        rows, pos, freq, qw, kw = case(T, Hq, Hkv, D, D // 2, seed=i)
        fused = dev(rows)
        cache = memra.KVCache("fp8", "fp8", T // 16 + 1, Hkv, D, 0.02, 0.02)
        q_out, k_out = (torch.empty(T, h, D, dtype=torch.float16, device="cuda") for h in (Hq, Hkv))
        calls.append(lambda stream, a=(fused[:, :Hq], fused[:, Hq:Hq + Hkv], dev(pos), dev(freq), q_out, k_out, dev(qw), dev(kw)),
                     kw_=dict(cache=cache, v=fused[:, Hq + Hkv:], slot_mapping=dev(np.arange(T, dtype=np.int32))):
                     memra.qk_norm_rope(*a, EPS, False, **kw_, stream=stream))
        calls[-1](None)
        check(q_out, rows[:, :Hq], qw, pos, freq, False)
        assert memra.read_status(cache) == 0
        outs.append((q_out, k_out, cache.k_pool, cache.v_pool))
        want.append([t.clone() for t in outs[-1]])
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for turn in range(600):
        for call, stream in zip(calls, streams):
            call(stream if turn < 300 else None)
        if turn == 299:
            torch.cuda.synchronize()
    assert all(torch.equal(t, u) for a, b in zip(outs, want) for t, u in zip(a, b))
