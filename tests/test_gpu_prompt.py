"""Prompt attention on the GPU against its definition in float64.

Tolerance, per output element, from the arithmetic (u = 2^-11, half a step of
fp16, relative): the output's rounding u |o|; the rounding of each weight to
fp16, u sum p |v| / sum p, or 2^-25 absolute for a weight below fp16's normal
range (the largest weight is at least 1, so l >= 1); the float32 scores, each
K = 16 step of a product off by at most 2^-22 of the absolute products so far,
and 2^-20 for the exponential and the sums: a relative error of twice that on
every weight.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = 2.0 ** -11


@pytest.fixture(scope="module")
def memra():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from decode_attention_block_memra_gb300 import _build
    _build.build()
    import decode_attention_block_memra_gb300 as m
    m.lib()
    return m


def reference(q, k, v, window=0, scale=None):
    """One sequence in float64: q [n, Hq, D], k, v [n, Hkv, D] -> (o, tolerance), both [n, Hq, D]."""
    n, Hq, D = q.shape
    G = Hq // k.shape[1]
    scale = D ** -0.5 if scale is None else scale
    o = torch.empty(n, Hq, D, dtype=torch.float64, device=q.device)
    tol = torch.empty_like(o)
    at = torch.arange(n, device=q.device)
    seen = at[None] <= at[:, None]
    if window:
        seen &= at[None] > at[:, None] - window
    for h in range(Hq):
        qd, kd, vd = q[:, h].double(), k[:, h // G].double(), v[:, h // G].double()
        s = (qd @ kd.T * scale).masked_fill(~seen, -np.inf)
        p = torch.softmax(s, 1)
        mass = (qd.abs() @ kd.abs().T * scale).masked_fill(~seen, 0).amax(1, keepdim=True)
        weight = 2 * ((D // 16 + 2) * 2.0 ** -22 * mass + 2.0 ** -20)
        o[:, h] = p @ vd
        tol[:, h] = U * o[:, h].abs() + (U + weight) * (p @ vd.abs()) + n * 2.0 ** -25 * vd.abs().max()
    return o, tol


def check(memra, lens, Hq, Hkv, D, window=0, fused=False, pad=0, lead=0, seed=0, mult=1.0, scale=None, fill=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    total = lead + sum(lens) + pad
    rows = torch.randn(total, Hq + 2 * Hkv, D, device="cuda", generator=g)
    rows[:, :Hq] *= mult
    rows = rows.half()
    if fill is not None:
        rows[:lead] = fill
        rows[lead + sum(lens):] = fill
    q, k, v = rows[:, :Hq], rows[:, Hq:Hq + Hkv], rows[:, Hq + Hkv:]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    cu = torch.tensor(np.cumsum([lead] + list(lens)), dtype=torch.int32, device="cuda")
    out = torch.full((total, Hq, D), 77.0, dtype=torch.float16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    memra.prompt_attn(q, k, v, cu, out, sm_scale=scale, window=window, status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    begin = lead
    for n in lens:
        if n:
            sl = slice(begin, begin + n)
            want, tol = reference(q[sl], k[sl], v[sl], window, scale)
            err = (out[sl].double() - want).abs()
            assert torch.isfinite(out[sl]).all()
            assert bool((err <= tol).all()), (lens, n, float((err / tol).max()))
        begin += n
    assert bool((out[:lead] == 77).all()) and bool((out[begin:] == 77).all())
    return q, k, v, cu, out


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300, 1000])
def test_lengths(memra, n, D):
    check(memra, [n], 8, 2, D, seed=n)


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("Hq,Hkv", [(4, 4), (1, 1), (2, 1), (6, 2), (10, 2), (7, 1), (32, 4), (40, 1), (128, 1)])
def test_groups_packed(memra, Hq, Hkv, D):
    check(memra, [70, 1, 0, 200, 33], Hq, Hkv, D, seed=Hq)


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("window", [1, 2, 16, 63, 64, 65, 128, 130, 700, 5000])
def test_window(memra, window, D):
    *_, v, _, out = check(memra, [300, 5, 513], 8, 4, D, window=window, seed=window)
    if window == 1:                                  # one visible key: the row is its own v
        assert torch.equal(out, v.repeat_interleave(2, 1))


@pytest.mark.parametrize("D", [128, 256])
def test_fused_rows_and_rows_of_no_sequence(memra, D):
    # what lies before the first and behind the last sequence must not reach any row, not even as 0 * inf
    for fill in (float("nan"), float("inf"), 65504.0):
        check(memra, [130, 1, 67], 16, 4, D, fused=True, lead=9, pad=200, fill=fill)
        check(memra, [130, 1, 67], 16, 4, D, fused=True, lead=9, pad=200, fill=fill, window=40)


@pytest.mark.parametrize("D", [128, 256])
def test_neighbours_do_not_leak(memra, D):
    """Infinities and NaN in one sequence stay in its own rows."""
    q, k, v, cu, out = check(memra, [100, 77, 150], 8, 2, D, seed=3)
    want = out.clone()
    for x in (q, k, v):
        x[100:177] = float("inf")
        x[120:150] = float("nan")
    memra.prompt_attn(q, k, v, cu, out)
    assert torch.equal(out[:100], want[:100]) and torch.equal(out[177:], want[177:])


@pytest.mark.parametrize("D", [128, 256])
def test_peaked_and_flat_scores(memra, D):
    check(memra, [260, 140], 8, 2, D, mult=60.0, seed=4)        # nearly one-hot rows; the maximum moves often
    check(memra, [260, 140], 8, 2, D, scale=1e-6, seed=5)       # means
    check(memra, [900], 4, 4, D, mult=8.0, scale=0.2, seed=6)


def test_rising_maxima(memra):
    """Scores that grow along the keys by more than the lazy threshold a step, so O is rescaled at each."""
    n, D = 700, 128
    k = torch.zeros(n, 1, D, device="cuda").half()
    k[:, 0, 0] = torch.arange(n, device="cuda") * 0.25
    v = torch.randn(n, 1, D, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).half()
    q = torch.zeros(n, 8, D, device="cuda").half()
    q[..., 0] = 1.0
    out = torch.empty_like(q)
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    memra.prompt_attn(q, k, v, cu, out, sm_scale=1.0)
    want, tol = reference(q, k, v, scale=1.0)
    assert bool(((out.double() - want).abs() <= tol).all())


@pytest.mark.parametrize("D", [128, 256])
def test_alone_or_packed_same_bytes(memra, D):
    lens = [400, 33, 257]
    q, k, v, cu, out = check(memra, lens, 16, 4, D, seed=8)
    begin = 0
    for n in lens:
        sl = slice(begin, begin + n)
        alone = torch.empty_like(out[sl])
        memra.prompt_attn(q[sl], k[sl], v[sl], torch.tensor([0, n], dtype=torch.int32, device="cuda"), alone)
        assert torch.equal(alone, out[sl])
        begin += n


@pytest.mark.parametrize("D", [128, 256])
def test_long_means_keep_their_precision(memra, D):
    """Equal scores over up to 524,288 keys: every weight is 1 exactly, every row the mean of the values before it.

    What is left are the output's rounding (half a step, 2^-11 for values in
    [1, 2)) and the float32 sums: at most 512 steps of 16 keys in one sum, each
    off by at most 2^-21 of the sum so far, half of its end on average, so 2^-13
    relative and 2^-12 for values below 2.  A single sum over all the keys would
    be off by thousands of steps' cuts, all towards zero.
    """
    n = 524_288
    g = torch.Generator(device="cuda").manual_seed(14)
    v = (1.9 + 0.09 * torch.rand(n, 1, D, device="cuda", generator=g)).half()
    q, k = torch.zeros_like(v), torch.randn(n, 1, D, device="cuda", generator=g).half()
    out = torch.empty_like(v)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    memra.prompt_attn(q, k, v, torch.tensor([0, n], dtype=torch.int32, device="cuda"), out, status=status)
    assert int(status) == 0
    rows = torch.arange(1, n + 1, device="cuda", dtype=torch.float64)[:, None, None]
    err = (out.double() - v.double().cumsum(0) / rows).abs()      # (the values are multiples of 2^-10: sums are exact)
    assert float(err.max()) <= 2.0 ** -11 + 2.0 ** -12, [float(x.max()) for x in err.split(n // 8)]


def far_rows(memra, n, D, window=0, mult=1.0, drift=0.0, seed=0):
    """(got, want, tolerance) of some rows of one prompt of n tokens: its ends and around each 8,192 keys, two heads."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    Hq, Hkv = 8, 2
    q, k, v = (torch.randn(n, h, D, device="cuda", generator=g) for h in (Hq, Hkv, Hkv))
    q *= mult
    if drift:                                        # scores that rise along the keys
        q[..., 0], k[..., 0] = 1.0, drift * torch.arange(n, device="cuda")[:, None] * D ** 0.5
    q, k, v = q.half(), k.half(), v.half()
    out = torch.empty_like(q)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    memra.prompt_attn(q, k, v, torch.tensor([0, n], dtype=torch.int32, device="cuda"), out, window=window,
                      status=status)
    assert int(status) == 0
    rows = torch.unique(torch.cat([torch.arange(a, a + 40) for a in (0, *range(8192 - 20, n - 40, 8192), n - 40)]))
    rows = rows.cuda()
    at = torch.arange(n, device="cuda")
    seen = at[None] <= rows[:, None]
    if window:
        seen &= at[None] > rows[:, None] - window
    parts = []
    for h in (0, Hq - 1):
        qd, kd, vd = q[rows, h].double(), k[:, h // 4].double(), v[:, h // 4].double()
        p = torch.softmax((qd @ kd.T * D ** -0.5).masked_fill(~seen, -np.inf), 1)
        mass = (qd.abs() @ kd.abs().T * D ** -0.5).masked_fill(~seen, 0).amax(1, keepdim=True)
        weight = 2 * ((D // 16 + 2) * 2.0 ** -22 * mass + 2.0 ** -20)
        want = p @ vd
        # as in reference(), and 2^-13 for 512 steps of the sums of products
        tol = U * want.abs() + (U + weight + 2.0 ** -13) * (p @ vd.abs()) + n * 2.0 ** -25 * vd.abs().max()
        parts.append((out[rows, h].double(), want, tol))
    return [torch.stack(x) for x in zip(*parts)]


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("n,window", [(8192, 0), (8193, 0), (16_640, 0), (40_001, 0), (40_001, 1000), (40_001, 12_345),
                                      (40_001, 30_000)])
def test_long_prompts(memra, n, window, D):
    """Against float64, element by element, and in the 2-norm: there the output's rounding and the weights' are
    at most u each, and the float32 parts of tol add 2^-12."""
    got, want, tol = far_rows(memra, n, D, window, mult=0.5, seed=n + window)
    assert bool(((got - want).abs() <= tol).all())
    assert float((got - want).norm() / want.norm()) <= 2 * U + 2.0 ** -12


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("drift", [-0.002, 0.0005, 0.002, 0.02])
def test_long_prompts_with_drifting_scores(memra, drift, D):
    # scores that rise or fall by 20 to 800 over the keys: what was summed before is scaled down again and again, or rules
    got, want, tol = far_rows(memra, 40_001, D, mult=1.0, drift=drift, seed=15)
    assert bool(((got - want).abs() <= tol).all()), float(((got - want).abs() / tol).max())


@pytest.mark.parametrize("D", [128, 256])
def test_infinite_values_reach_the_rows_that_see_them(memra, D):
    n = 20_000
    g = torch.Generator(device="cuda").manual_seed(16)
    q, k, v = (torch.randn(n, h, D, device="cuda", generator=g).half() for h in (4, 1, 1))
    cu, out, want = torch.tensor([0, n], dtype=torch.int32, device="cuda"), torch.empty_like(q), torch.empty_like(q)
    memra.prompt_attn(q * 0.1, k, v, cu, want)
    v[40, 0, 3], v[40, 0, 7] = float("inf"), float("-inf")
    memra.prompt_attn(q * 0.1, k, v, cu, out)
    assert bool((out[40:, :, 3] == float("inf")).all()) and bool((out[40:, :, 7] == float("-inf")).all())
    keep = [c for c in range(D) if c not in (3, 7)]
    assert torch.equal(out[..., keep], want[..., keep])


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("value", [65504.0, -65504.0, 2.0 ** -14, 3 * 2.0 ** -24])
def test_long_means_at_the_ends_of_the_range(memra, value, D):
    # equal weights and values, over five sums: half a step of fp16 and 2^-13 for the sums
    n = 40_000
    v = torch.full((n, 1, D), value, device="cuda").half()
    q, out = torch.zeros_like(v), torch.empty_like(v)
    memra.prompt_attn(q, q, v, torch.tensor([0, n], dtype=torch.int32, device="cuda"), out)
    err = (out.double() - value).abs()
    assert float(err.max()) <= max(U, 2.0 ** -25 / abs(value)) * abs(value) + 2.0 ** -13 * abs(value)


def test_many_sequences(memra):
    rng = np.random.default_rng(2)
    check(memra, list(rng.integers(0, 40, 101)), 8, 2, 128, seed=9, pad=4)


def test_bad_lengths_are_clamped_and_flagged(memra):
    q, k, v, cu, out = check(memra, [64, 64], 8, 2, 128, seed=10)
    want = out.clone()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for bad in ([0, 64, 1000], [0, 64, 2 ** 31 - 1]):            # past the rows: the second ends at 128
        out.zero_()
        memra.prompt_attn(q, k, v, torch.tensor(bad, dtype=torch.int32, device="cuda"), out, status=status)
        assert int(status) == memra.DEVERR_BAD_SEQ_LEN
        assert torch.equal(out, want)
        status.zero_()
    for bad in ([-5, 64, 128], [64, 0, 64], [0, 128, 64], [200, 300, 400]):
        memra.prompt_attn(q, k, v, torch.tensor(bad, dtype=torch.int32, device="cuda"), out, status=status)
        assert int(status) == memra.DEVERR_BAD_SEQ_LEN
        status.zero_()


def test_rows_past_32_bit_offsets(memra):
    # 70,000 tokens x 128 heads x 256: the last sequences' rows start past 2^31 elements
    n, Hq, D, lens = 70_000, 128, 256, [70] * 1000
    g = torch.Generator(device="cuda").manual_seed(13)
    q = torch.empty(n, Hq, D, dtype=torch.float16, device="cuda")
    q.normal_(generator=g)
    k, v = (torch.randn(n, 1, D, device="cuda", generator=g).half() for _ in range(2))
    out = torch.empty_like(q)
    cu = torch.arange(0, n + 1, 70, dtype=torch.int32, device="cuda")
    memra.prompt_attn(q, k, v, cu, out)
    for b in (0, 500, 999):
        sl = slice(70 * b, 70 * b + 70)
        want, tol = reference(q[sl], k[sl], v[sl])
        assert bool(((out[sl].double() - want).abs() <= tol).all())


def test_captured_call_reads_new_lengths(memra):
    q, k, v, cu, out = check(memra, [90, 38], 8, 2, 128, seed=11)
    first = out.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        memra.prompt_attn(q, k, v, cu, out)
    out.zero_()
    g.replay()
    assert torch.equal(out, first)
    cu.copy_(torch.tensor([0, 20, 128], dtype=torch.int32))
    g.replay()
    for a, b in ((0, 20), (20, 128)):
        want, tol = reference(q[a:b], k[a:b], v[a:b])
        assert bool(((out[a:b].double() - want).abs() <= tol).all())


@pytest.mark.parametrize("D", [128, 256])
def test_many_calls_in_a_row(memra, D):
    """No wait runs out and no byte changes over thousands of calls (a wait that names the wrong phase would)."""
    q, k, v, cu, out = check(memra, [700, 300, 64], 8, 2, D, window=150, seed=12)
    want = out.clone()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    same = torch.ones((), dtype=torch.bool, device="cuda")
    for _ in range(3000):
        out.zero_()
        memra.prompt_attn(q, k, v, cu, out, window=150, status=status)
        same &= (out == want).all()
    assert int(status) == 0 and bool(same)


def test_binding_refuses_other_layouts(memra):
    q = torch.zeros(4, 8, 128, device="cuda").half()
    k = torch.zeros(4, 2, 128, device="cuda").half()
    cu = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    bad = torch.zeros(4, 128, 8, device="cuda").half().transpose(1, 2)
    for args in ((bad, k, k, cu, q), (q, k[:3], k, cu, q), (q, k, k[:, :1], cu, q), (q, k, k, cu, bad),
                 (q.float(), k, k, cu, q), (q, k.cpu(), k, cu, q), (q, k, k, cu.long(), q), (q, k, k, cu.cpu(), q),
                 (q, k, k, cu, q.bfloat16())):
        with pytest.raises(memra.MemraError):
            memra.prompt_attn(*args)
    with pytest.raises(memra.MemraError):
        memra.prompt_attn(q, k, k, cu, q, status=torch.zeros(1, dtype=torch.int32))


def test_binding_refuses_a_nested_list_and_other_status_words(memra):
    """[[0, 4]] would be no sequence at all, and the kernel writes 32 bits of the status word."""
    q = torch.zeros(4, 8, 128, device="cuda").half()
    k = torch.zeros(4, 2, 128, device="cuda").half()
    cu = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    with pytest.raises(memra.MemraError):
        memra.prompt_attn(q, k, k, cu[None], q)
    for dtype, n in ((torch.uint8, 4), (torch.int64, 1), (torch.float32, 1), (torch.int32, 0)):
        with pytest.raises(memra.MemraError):
            memra.prompt_attn(q, k, k, cu, q, status=torch.zeros(n, dtype=dtype, device="cuda"))
