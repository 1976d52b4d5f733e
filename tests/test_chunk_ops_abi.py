"""Host checks of the operators of a prompt in chunks (CPU only): every refusal returns before any CUDA call."""
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


def test_norm_rope_checks(memra):
    good = dict(q=64, qs=1024, k=64, ks=256, v=64, vs=256, qw=64, kw=64, eps=1e-6, pos=64, freq=64, rot=128, il=0, n=4,
                Hq=8, Hkv=2, D=128, qo=64, qos=1024, ko=64, kos=256, slots=64)

    def call(c=None, no_cache=False, **kw):
        a = {**good, **kw}
        return memra.lib().memra_qk_norm_rope(
            a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["qw"], a["kw"], a["eps"], a["pos"], a["freq"], a["rot"],
            a["il"], a["n"], a["Hq"], a["Hkv"], a["D"], a["qo"], a["qos"], a["ko"], a["kos"],
            None if no_cache else ctypes.byref(c or cache(memra)), a["slots"], None)

    assert call(n=0) == 0
    assert call(n=0, q=0, k=0, v=0, qo=0, ko=0, slots=0) == 0
    for name in ("q", "k", "v", "qo", "slots", "pos", "freq"):
        assert call(**{name: 0}) == INVALID
    for name in ("q", "k", "v", "qo", "ko"):
        assert call(**{name: 72}) == INVALID
    for name in ("qw", "kw", "pos", "freq", "slots"):
        assert call(**{name: 66}) == INVALID
    for name, stride in (("qs", 1016), ("ks", 248), ("vs", 260), ("qos", 1028), ("kos", 0)):
        assert call(**{name: stride}) == INVALID
    for rot in (-16, 8, 120, 144):
        assert call(rot=rot) == INVALID
    for eps in (-1e-6, float("nan"), float("inf")):
        assert call(eps=eps) == INVALID
    assert call(n=-1) == INVALID
    assert call(Hq=0) == INVALID
    assert call(Hkv=0) == INVALID
    assert call(Hkv=3, ks=384, vs=384, kos=384) == INVALID         # not the cache's
    assert call(D=256, rot=128) == INVALID                         # not the cache's
    assert call(D=64, rot=64) == UNSUPPORTED
    assert call(Hq=65536) == UNSUPPORTED
    assert call(c=cache(memra, page_size=32)) == UNSUPPORTED
    # keys, values and slots come exactly with where they go
    assert call(no_cache=True) == INVALID
    assert call(no_cache=True, v=0) == INVALID
    assert call(no_cache=True, slots=0) == INVALID
    assert call(no_cache=True, v=0, slots=0, ko=0) == INVALID
    assert call(no_cache=True, v=0, slots=0, k=0) == INVALID


def test_evict_checks(memra):
    good = dict(pt=64, maxp=4, sl=64, maxlen=64, w=64, ws=64, bud=64, most=32, sink=1, recent=1, dt=64, dp=2, B=2, kept=64,
                nw=128, nws=32, nl=64)

    def call(c=None, **kw):
        a = {**good, **kw}
        return memra.lib().memra_kv_evict(ctypes.byref(c or cache(memra)), a["pt"], a["maxp"], a["sl"], a["maxlen"], a["w"],
                                          a["ws"], a["bud"], a["most"], a["sink"], a["recent"], a["dt"], a["dp"], a["B"],
                                          a["kept"], a["nw"], a["nws"], a["nl"], None)

    assert memra.lib().memra_kv_evict(None, *[64] * 5, 64, *[64] * 3, 1, 1, 64, 8, 2, 64, 128, 64, 64, None) == INVALID
    assert call(B=0) == 0
    assert call(most=0) == 0
    for name in ("pt", "sl", "w", "bud", "dt", "kept"):
        assert call(**{name: 0}) == INVALID
    for name in ("pt", "sl", "w", "bud", "dt", "kept", "nw", "nl"):
        assert call(**{name: 66}) == INVALID
    for name in ("B", "maxlen", "most", "sink", "recent", "dp"):
        assert call(**{name: -1}) == INVALID
    assert call(maxp=0) == INVALID
    assert call(ws=63) == INVALID
    assert call(most=33) == INVALID                # more than dst_table's pages
    assert call(nws=31) == INVALID
    assert call(nw=64) == INVALID                  # the weights themselves
    assert call(B=32768) == UNSUPPORTED
    assert call(c=cache(memra, v_fmt=0)) == UNSUPPORTED


def test_chunk_checks(memra):
    need = memra.chunk_attn_workspace_bytes(128)
    good = dict(q=64, qs=1024, cu=64, pt=64, maxp=4, sl=64, maxlen=64, B=2, T=8, Hq=8, Hkv=2, D=128, scale=0.1, window=0,
                ws=64, wsb=need, out=64, lse=64)

    def call(c=None, f=None, **kw):
        a = {**good, **kw}
        return (f or memra.lib().memra_chunk_attn)(
            ctypes.byref(c or cache(memra)), a["q"], a["qs"], a["cu"], a["pt"], a["maxp"], a["sl"], a["maxlen"], a["B"],
            a["T"], a["Hq"], a["Hkv"], a["D"], a["scale"], a["window"], a["ws"], a["wsb"], a["out"], a["lse"], None)

    assert need > 0 and memra.chunk_attn_workspace_bytes(256) > 0 and memra.chunk_attn_workspace_bytes(64) == 0
    assert call(B=0) == 0
    assert call(T=0) == 0
    for name in ("q", "cu", "pt", "sl", "out", "ws"):
        assert call(**{name: 0}) == INVALID
    for name, at in (("q", 72), ("out", 72), ("ws", 72), ("cu", 66), ("pt", 66), ("sl", 66), ("lse", 66)):
        assert call(**{name: at}) == INVALID
    for name in ("B", "T", "maxlen", "window"):
        assert call(**{name: -1}) == INVALID
    assert call(wsb=need - 1) == WORKSPACE
    assert call(maxp=0) == INVALID
    assert call(qs=1016) == INVALID
    assert call(qs=1028) == INVALID
    assert call(Hq=7) == INVALID
    assert call(Hq=0) == INVALID
    assert call(Hkv=4) == INVALID                  # not the cache's
    assert call(D=256) == INVALID
    assert call(Hq=2 * 129, qs=2 * 129 * 128) == UNSUPPORTED
    assert call(B=65536) == UNSUPPORTED
    assert call(c=cache(memra, v_fmt=0)) == UNSUPPORTED
    assert call(c=cache(memra, k_pool=72)) == INVALID
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert call(scale=scale) == INVALID
    hook = memra.lib().memra_testing_chunk_attn_short_page
    assert call(f=hook, Hq=7) == INVALID and call(f=hook, B=0) == 0


def test_key_weights_checks(memra):
    good = dict(q=64, qs=1024, lse=64, cu=64, pt=64, maxp=4, sl=64, maxlen=64, B=2, T=8, Hq=8, Hkv=2, D=128, scale=0.1,
                keep=1.0, w=64, ws=64)

    def call(c=None, **kw):
        a = {**good, **kw}
        return memra.lib().memra_key_weights(
            ctypes.byref(c or cache(memra)), a["q"], a["qs"], a["lse"], a["cu"], a["pt"], a["maxp"], a["sl"], a["maxlen"],
            a["B"], a["T"], a["Hq"], a["Hkv"], a["D"], a["scale"], a["keep"], a["w"], a["ws"], None)

    assert call(B=0) == 0
    assert call(T=0) == 0
    for name in ("q", "lse", "cu", "pt", "sl", "w"):
        assert call(**{name: 0}) == INVALID
    assert call(q=72) == INVALID
    for name in ("lse", "cu", "pt", "sl", "w"):
        assert call(**{name: 66}) == INVALID
    for name in ("B", "T", "maxlen"):
        assert call(**{name: -1}) == INVALID
    assert call(maxp=0) == INVALID
    assert call(ws=63) == INVALID
    assert call(qs=1016) == INVALID
    assert call(qs=1028) == INVALID
    assert call(qs=1 << 38) == UNSUPPORTED
    assert call(Hq=7) == INVALID
    assert call(Hkv=4) == INVALID                  # not the cache's
    assert call(D=256) == INVALID
    assert call(Hq=2 * 129, qs=2 * 129 * 128) == UNSUPPORTED
    assert call(B=65536) == UNSUPPORTED
    assert call(c=cache(memra, v_fmt=0)) == UNSUPPORTED
    for x in (float("nan"), float("inf")):
        assert call(keep=x) == INVALID and call(scale=x) == INVALID
    assert call(scale=0.0) == INVALID


def test_key_weights_hook_checks(memra):
    c, none = cache(memra), [0.1, 1.0, 64, 64, None]
    hook = memra.lib().memra_testing_key_weights_short_page
    good = [64, 1024, 64, 64, 64, 4, 64, 64, 2, 8, 8, 2, 128]
    for at, value, want in ((8, 0, 0), (9, 0, 0), (0, 0, INVALID), (10, 7, INVALID), (1, 1016, INVALID)):
        assert hook(ctypes.byref(c), *[value if i == at else x for i, x in enumerate(good)], *none) == want


def test_evict_refuses_budgets_at_the_end_of_int32(memra):
    """Row numbers up to a CTA's pages behind the last would pass 2^31."""
    def call(most):
        return memra.lib().memra_kv_evict(ctypes.byref(cache(memra)), 64, 4, 64, 64, 64, 64, 64, most, 1, 1, 64, 1 << 27, 2, 64,
                                          128, 1 << 31, 64, None)

    assert call(2 ** 31 - 1) == UNSUPPORTED
    assert call(2 ** 31 - 65536) == UNSUPPORTED
