"""Host checks of the operators around the decode step: page copies, tree compaction (CPU only).

Every refusal returns before any CUDA call, so the pointers are made-up numbers."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def memra():
    from decode_attention_block_memra_gb300 import _build
    try:
        _build.build()
    except RuntimeError as e:          # no nvcc on this machine
        pytest.skip(str(e))
    import decode_attention_block_memra_gb300 as m
    m.lib()
    return m


def cache(memra, **kw):
    c = memra.KVCacheStruct(0, 1, 16, 2, 128, 4, 4096, 8192, 1.0, 1.0, 0)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


def test_copy_pages_checks(memra):
    def call(c=None, src=64, dst=128, n=3):
        return memra.lib().memra_kv_copy_pages(ctypes.byref(c or cache(memra)), src, dst, n, None)

    assert memra.lib().memra_kv_copy_pages(None, 64, 128, 1, None) == INVALID
    assert call(n=-1) == INVALID
    assert call(n=0, src=0, dst=0) == 0
    assert call(src=0) == INVALID
    assert call(dst=0) == INVALID
    assert call(src=66) == INVALID
    assert call(c=cache(memra, head_dim=64)) == UNSUPPORTED
    assert call(c=cache(memra, k_fmt=1)) == UNSUPPORTED
    assert call(c=cache(memra, num_pages=0)) == INVALID
    assert call(c=cache(memra, n_kv_heads=2 ** 31 - 1)) == UNSUPPORTED


def test_compact_checks(memra):
    good = dict(pt=64, maxp=4, sl=64, maxlen=64, acc=64, most=4, n=64, B=2, nodes=8)

    def call(c=None, **kw):
        a = {**good, **kw}
        return memra.lib().memra_kv_compact(ctypes.byref(c or cache(memra)), a["pt"], a["maxp"], a["sl"], a["maxlen"],
                                            a["acc"], a["most"], a["n"], a["B"], a["nodes"], None)

    assert call(c=cache(memra, page_size=32)) == UNSUPPORTED
    for name in ("pt", "sl", "acc", "n"):
        assert call(**{name: 0}) == INVALID
        assert call(**{name: 66}) == INVALID
    assert call(B=-1) == INVALID
    assert call(B=65536) == UNSUPPORTED
    assert call(nodes=0) == INVALID
    assert call(nodes=memra.MAX_TREE_NODES + 1) == UNSUPPORTED
    assert call(most=9) == INVALID                 # more kept rows than nodes
    assert call(most=-1) == INVALID
    assert call(maxp=0) == INVALID
    assert call(maxlen=-1) == INVALID
    assert call(B=0) == 0
    assert call(most=0) == 0


def test_prompt_checks(memra):
    good = dict(q=64, qs=1024, k=64, ks=256, v=64, vs=256, cu=64, B=2, T=10, Hq=8, Hkv=2, D=128, scale=0.1, window=0,
                out=64, status=0)

    def call(**kw):
        a = {**good, **kw}
        return memra.lib().memra_prompt_attn(a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["cu"], a["B"], a["T"],
                                             a["Hq"], a["Hkv"], a["D"], a["scale"], a["window"], a["out"], a["status"],
                                             None)

    assert call(B=0) == 0
    assert call(T=0) == 0
    for name in ("q", "k", "v", "out"):
        assert call(**{name: 0}) == INVALID
        assert call(**{name: 72}) == INVALID
    assert call(cu=0) == INVALID
    assert call(cu=66) == INVALID
    assert call(status=66) == INVALID
    assert call(qs=1016) == INVALID                # less than a token's heads
    assert call(ks=248) == INVALID
    assert call(vs=260) == INVALID                 # not a multiple of 8
    assert call(qs=1 << 38) == UNSUPPORTED
    assert call(Hq=7) == INVALID
    assert call(Hkv=0) == INVALID
    assert call(D=64) == UNSUPPORTED
    assert call(Hq=129 * 2, qs=129 * 256) == UNSUPPORTED
    assert call(window=-1) == INVALID
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert call(scale=scale) == INVALID
    assert call(B=65536) == UNSUPPORTED
    assert call(B=-1) == INVALID
    assert call(T=-1) == INVALID


def test_tree_checks(memra):
    good = dict(q=64, pt=64, maxp=4, sl=64, maxlen=64, mask=64, B=2, N=8, Hq=8, Hkv=2, D=128, scale=0.1, ws=64,
                wsb=1 << 20, out=64)

    def call(c=None, **kw):
        a = {**good, **kw}
        return memra.lib().memra_tree_attn(ctypes.byref(c or cache(memra)), a["q"], a["pt"], a["maxp"], a["sl"],
                                           a["maxlen"], a["mask"], a["B"], a["N"], a["Hq"], a["Hkv"], a["D"],
                                           a["scale"], a["ws"], a["wsb"], a["out"], None)

    assert call(B=0) == 0
    for name in ("q", "pt", "sl", "mask", "out"):
        assert call(**{name: 0}) == INVALID
    for name, at in (("q", 72), ("out", 72), ("pt", 66), ("sl", 66), ("mask", 68)):
        assert call(**{name: at}) == INVALID
    assert call(c=cache(memra, k_pool=72)) == INVALID
    assert call(c=cache(memra, v_fmt=0)) == UNSUPPORTED
    assert call(N=0) == INVALID
    assert call(N=memra.MAX_TREE_NODES + 1) == UNSUPPORTED
    assert call(Hq=7) == INVALID
    assert call(Hkv=4) == INVALID                  # not the cache's
    assert call(D=256) == INVALID
    assert call(Hq=2 * 129) == UNSUPPORTED
    assert call(B=-1) == INVALID
    assert call(B=65536) == UNSUPPORTED
    assert call(maxp=0) == INVALID
    assert call(maxlen=-1) == INVALID
    assert call(scale=float("nan")) == INVALID
    need = memra.tree_attn_workspace_bytes(2, 8, 8, 128, 5000)
    assert need == 16 + 2 * 8 * 8 * 20 * 129 * 4   # 79 chunks of 64 keys: 20 splits of 4 chunks at most
    assert call(maxlen=5000, wsb=need - 1) == WORKSPACE
    assert call(maxlen=5000, wsb=need, ws=72) == INVALID
    assert call(maxlen=5000, wsb=need, ws=0) == INVALID
    assert memra.tree_attn_workspace_bytes(2, 8, 8, 128, 256) == 16      # one split: the plan word alone
    assert memra.tree_attn_workspace_bytes(2, 65, 8, 128, 5000) == 0
    assert memra.tree_attn_workspace_bytes(2, 8, 8, 64, 5000) == 0
    # 262,144 tokens: 160 partials a row, whatever the device
    assert memra.tree_attn_workspace_bytes(1, 64, 32, 128, 262144) == 16 + 64 * 32 * 160 * 129 * 4


def test_hooks_of_the_bounded_waits_check_as_the_plain_calls(memra):
    L, c = memra.lib(), cache(memra)
    for heads, batch, want in ((7, 2, INVALID), (8, -1, INVALID), (2 * 129, 2, UNSUPPORTED), (8, 0, 0)):
        assert L.memra_testing_prompt_attn_short_copy(64, 128 * 258, 64, 256, 64, 256, 64, batch, 10, heads, 2, 128, 0.1,
                                                      0, 64, 0, None) == want
        assert L.memra_testing_tree_attn_short_page(ctypes.byref(c), 64, 64, 4, 64, 64, 64, batch, 8, heads, 2, 128, 0.1,
                                                    64, 1 << 20, 64, None) == want
