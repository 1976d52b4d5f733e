"""Python binding of the memra decode-attention C ABI (include/memra.h).

Argument marshalling only: every step of the hot path (quantize-append,
split-K decode, log-sum-exp combine) runs in the CUDA kernels of
``libmemra.so``.  PyTorch supplies device memory and the current stream; the
functions take torch tensors (or raw integers for pointers) and raise
``MemraError`` on any non-zero status.  There is no CPU fallback: if the
library is missing, every call raises.
"""
from __future__ import annotations

import ctypes
import os

from . import _build

FORMATS = {"q8_0": 0, "q5_1": 1, "q4_0": 2, "fp8": 3, "nvfp4": 4}
PAGE_SIZE = 16
SPLIT_TOKENS = 1280
MAX_TREE_NODES = 64

DEVERR_BAD_PAGE = 1
DEVERR_BAD_SLOT = 2
DEVERR_BAD_SEQ_LEN = 4
DEVERR_TIMEOUT = 8
DEVERR_PREFIX = 16


class MemraError(RuntimeError):
    def __init__(self, status: int, where: str, flags: int = 0):
        self.status = status
        self.flags = flags
        msg = f"{where}: {status_string(status)} (status {status})"
        if flags:
            msg += f", device flags 0x{flags:x}"
        super().__init__(msg)


class KVCacheStruct(ctypes.Structure):
    """Mirror of memra_kv_cache."""
    _fields_ = [
        ("k_fmt", ctypes.c_int32),
        ("v_fmt", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("n_kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("num_pages", ctypes.c_int32),
        ("k_pool", ctypes.c_void_p),
        ("v_pool", ctypes.c_void_p),
        ("k_scale", ctypes.c_float),
        ("v_scale", ctypes.c_float),
        ("status", ctypes.c_void_p),
    ]


_LIB = None

_CHUNK_ARGS = ([ctypes.POINTER(KVCacheStruct), ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p,
                ctypes.c_int32, ctypes.c_void_p] + [ctypes.c_int32] * 6 +
               [ctypes.c_float, ctypes.c_int32, ctypes.c_void_p, ctypes.c_size_t] + [ctypes.c_void_p] * 3)

_WEIGHT_ARGS = ([ctypes.POINTER(KVCacheStruct), ctypes.c_void_p, ctypes.c_int64] + [ctypes.c_void_p] * 3 +
                [ctypes.c_int32, ctypes.c_void_p] + [ctypes.c_int32] * 6 + [ctypes.c_float] * 2 +
                [ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p])

_SIGS = {
    "memra_kv_segment_bytes": (ctypes.c_size_t, [ctypes.c_int32] * 3),
    "memra_kv_pool_bytes": (ctypes.c_size_t, [ctypes.c_int32] * 6),
    "memra_kv_append": (ctypes.c_int, [ctypes.POINTER(KVCacheStruct), ctypes.c_void_p, ctypes.c_void_p,
                                       ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p]),
    "memra_decode_attn_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int32] * 5),
    "memra_decode_attn": (ctypes.c_int, [ctypes.POINTER(KVCacheStruct), ctypes.c_void_p, ctypes.c_void_p,
                                         ctypes.c_int32, ctypes.c_void_p] + [ctypes.c_int32] * 6 +
                          [ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_void_p]),
    "memra_decode_attn_partials": (ctypes.c_int, [ctypes.POINTER(KVCacheStruct), ctypes.c_void_p, ctypes.c_void_p,
                                                  ctypes.c_int32, ctypes.c_void_p] + [ctypes.c_int32] * 6 +
                                   [ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p,
                                    ctypes.c_void_p]),
    "memra_decode_attn_combine": (ctypes.c_int, [ctypes.POINTER(KVCacheStruct), ctypes.c_void_p] +
                                  [ctypes.c_int32] * 6 + [ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p,
                                                          ctypes.c_void_p]),
    "memra_decode_step": (ctypes.c_int, [ctypes.POINTER(KVCacheStruct), ctypes.c_void_p, ctypes.c_void_p,
                                         ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p] +
                          [ctypes.c_int32] * 6 + [ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p,
                                                  ctypes.c_void_p]),
    "memra_decode_attn_window": (ctypes.c_int, [ctypes.POINTER(KVCacheStruct), ctypes.c_void_p, ctypes.c_void_p,
                                                ctypes.c_int32, ctypes.c_void_p] + [ctypes.c_int32] * 6 +
                                 [ctypes.c_float, ctypes.c_int32, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p,
                                  ctypes.c_void_p]),
    "memra_decode_step_window": (ctypes.c_int, [ctypes.POINTER(KVCacheStruct), ctypes.c_void_p, ctypes.c_void_p,
                                                ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p] +
                                 [ctypes.c_int32] * 6 + [ctypes.c_float, ctypes.c_int32, ctypes.c_void_p,
                                                         ctypes.c_size_t, ctypes.c_void_p, ctypes.c_void_p]),
    "memra_decode_attn_cascade_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int32] * 6),
    "memra_decode_attn_cascade": (ctypes.c_int, [ctypes.POINTER(KVCacheStruct), ctypes.c_void_p, ctypes.c_void_p,
                                                 ctypes.c_int32, ctypes.c_void_p] + [ctypes.c_int32] * 7 +
                                  [ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p,
                                   ctypes.c_void_p]),
    "memra_decode_step_cascade": (ctypes.c_int, [ctypes.POINTER(KVCacheStruct), ctypes.c_void_p, ctypes.c_void_p,
                                                 ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p] +
                                  [ctypes.c_int32] * 7 + [ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t,
                                                          ctypes.c_void_p, ctypes.c_void_p]),
    "memra_decode_attn_noalloc": (ctypes.c_int, [ctypes.POINTER(KVCacheStruct), ctypes.c_void_p, ctypes.c_void_p,
                                                 ctypes.c_int32, ctypes.c_void_p] + [ctypes.c_int32] * 6 +
                                  [ctypes.c_float, ctypes.c_void_p, ctypes.c_void_p]),
    "memra_prompt_attn": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64] * 3 + [ctypes.c_void_p] +
                          [ctypes.c_int32] * 5 + [ctypes.c_float, ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p,
                                                  ctypes.c_void_p]),
    "memra_tree_attn_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int32] * 5),
    "memra_tree_attn": (ctypes.c_int, [ctypes.POINTER(KVCacheStruct), ctypes.c_void_p, ctypes.c_void_p,
                                       ctypes.c_int32, ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p] +
                        [ctypes.c_int32] * 5 + [ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p,
                                                ctypes.c_void_p]),
    "memra_kv_copy_pages": (ctypes.c_int, [ctypes.POINTER(KVCacheStruct), ctypes.c_void_p, ctypes.c_void_p,
                                           ctypes.c_int32, ctypes.c_void_p]),
    "memra_kv_compact": (ctypes.c_int, [ctypes.POINTER(KVCacheStruct), ctypes.c_void_p, ctypes.c_int32,
                                        ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p, ctypes.c_int32,
                                        ctypes.c_void_p, ctypes.c_int32, ctypes.c_int32, ctypes.c_void_p]),
    "memra_qk_norm_rope": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64] * 3 + [ctypes.c_void_p] * 2 +
                           [ctypes.c_float] + [ctypes.c_void_p] * 2 + [ctypes.c_int32] * 6 +
                           [ctypes.c_void_p, ctypes.c_int64] * 2 + [ctypes.POINTER(KVCacheStruct), ctypes.c_void_p,
                                                                    ctypes.c_void_p]),
    "memra_chunk_attn_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int32]),
    "memra_chunk_attn": (ctypes.c_int, _CHUNK_ARGS),
    "memra_testing_chunk_attn_short_page": (ctypes.c_int, _CHUNK_ARGS),
    "memra_key_weights": (ctypes.c_int, _WEIGHT_ARGS),
    "memra_testing_key_weights_short_page": (ctypes.c_int, _WEIGHT_ARGS),
    "memra_kv_evict": (ctypes.c_int, [ctypes.POINTER(KVCacheStruct), ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p,
                                      ctypes.c_int32, ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p] +
                       [ctypes.c_int32] * 3 + [ctypes.c_void_p, ctypes.c_int32, ctypes.c_int32, ctypes.c_void_p,
                                               ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p]),
    "memra_testing_decode_attn_short_page": (ctypes.c_int, [ctypes.POINTER(KVCacheStruct), ctypes.c_void_p,
                                                            ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p] +
                                             [ctypes.c_int32] * 6 + [ctypes.c_float, ctypes.c_void_p,
                                                                     ctypes.c_size_t, ctypes.c_void_p,
                                                                     ctypes.c_uint64, ctypes.c_void_p]),
    "memra_testing_prompt_attn_short_copy": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64] * 3 + [ctypes.c_void_p] +
                                             [ctypes.c_int32] * 5 + [ctypes.c_float, ctypes.c_int32, ctypes.c_void_p,
                                                                     ctypes.c_void_p, ctypes.c_void_p]),
    "memra_testing_tree_attn_short_page": (ctypes.c_int, [ctypes.POINTER(KVCacheStruct), ctypes.c_void_p,
                                                          ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p,
                                                          ctypes.c_int32, ctypes.c_void_p] + [ctypes.c_int32] * 5 +
                                           [ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p,
                                            ctypes.c_void_p]),
    "memra_testing_scale_division_mismatches": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p,
                                                                ctypes.c_void_p]),
    "memra_read_status": (ctypes.c_int, [ctypes.POINTER(KVCacheStruct), ctypes.POINTER(ctypes.c_int32),
                                         ctypes.c_void_p]),
    "memra_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "memra_num_splits": (ctypes.c_int32, [ctypes.c_int32]),
}


def library_path() -> str:
    return _build.LIB


def lib() -> ctypes.CDLL:
    """Load libmemra.so (built in-tree by ``_build.build()``); raises if absent."""
    global _LIB
    if _LIB is None:
        path = _build.LIB
        if not os.path.exists(path):
            raise RuntimeError(f"libmemra.so is not built ({path}); run __graft_entry__.build() first")
        h = ctypes.CDLL(path)
        for name, (res, args) in _SIGS.items():
            fn = getattr(h, name)
            fn.restype = res
            fn.argtypes = args
        _LIB = h
    return _LIB


def status_string(status: int) -> str:
    return lib().memra_status_string(int(status)).decode()


def _check(rc: int, where: str):
    if rc != 0:
        raise MemraError(rc, where)


def _ptr(x) -> int:
    if x is None:
        return 0
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _device() -> int:
    import torch
    return torch._C._cuda_getDevice()


def _stream(stream) -> int:
    if stream is None:
        # the current stream's handle without building a Stream object (3 us of a call's 8)
        import torch
        return torch._C._cuda_getCurrentRawStream(_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def fmt_id(fmt) -> int:
    return FORMATS[fmt] if isinstance(fmt, str) else int(fmt)


def kv_segment_bytes(fmt, is_v: bool, head_dim: int) -> int:
    return int(lib().memra_kv_segment_bytes(fmt_id(fmt), int(bool(is_v)), head_dim))


def kv_pool_bytes(fmt, is_v: bool, num_pages: int, n_kv_heads: int, head_dim: int, page_size: int = PAGE_SIZE) -> int:
    return int(lib().memra_kv_pool_bytes(fmt_id(fmt), int(bool(is_v)), num_pages, page_size, n_kv_heads, head_dim))


def num_splits(seq_len: int) -> int:
    return int(lib().memra_num_splits(int(seq_len)))


def decode_attn_workspace_bytes(batch: int, q_len: int, n_heads: int, head_dim: int, max_seq_len: int) -> int:
    return int(lib().memra_decode_attn_workspace_bytes(batch, q_len, n_heads, head_dim, max_seq_len))


class KVCache:
    """A paged KV cache: the two pools and the status word as torch device tensors."""

    def __init__(self, k_fmt, v_fmt, num_pages: int, n_kv_heads: int, head_dim: int, k_scale: float = 1.0,
                 v_scale: float = 1.0, device="cuda", k_pool=None, v_pool=None):
        import torch
        self.k_fmt, self.v_fmt = k_fmt, v_fmt
        self.num_pages, self.n_kv_heads, self.head_dim = num_pages, n_kv_heads, head_dim
        kb = kv_pool_bytes(k_fmt, False, num_pages, n_kv_heads, head_dim)
        vb = kv_pool_bytes(v_fmt, True, num_pages, n_kv_heads, head_dim)
        if kb == 0 or vb == 0:
            raise MemraError(2, "KVCache")
        self.k_pool = k_pool if k_pool is not None else torch.zeros(kb, dtype=torch.uint8, device=device)
        self.v_pool = v_pool if v_pool is not None else torch.zeros(vb, dtype=torch.uint8, device=device)
        assert self.k_pool.numel() == kb and self.v_pool.numel() == vb
        self.status = torch.zeros(4, dtype=torch.int32, device=device)
        on = {t.get_device() for t in (self.k_pool, self.v_pool, self.status)}
        self.device_index = on.pop() if len(on) == 1 else None
        self.struct = KVCacheStruct(fmt_id(k_fmt), fmt_id(v_fmt), PAGE_SIZE, n_kv_heads, head_dim, num_pages,
                                    self.k_pool.data_ptr(), self.v_pool.data_ptr(), float(k_scale), float(v_scale),
                                    self.status.data_ptr())

    @property
    def ref(self):
        return ctypes.byref(self.struct)


def kv_append(cache: KVCache, k, v, slot_mapping, n_tok: int | None = None, stream=None) -> None:
    """memra_kv_append: k, v fp16 [n_tok, Hkv, D]; slot_mapping int32 [n_tok]."""
    n = int(slot_mapping.shape[0]) if n_tok is None else n_tok
    _check(lib().memra_kv_append(cache.ref, _ptr(k), _ptr(v), _ptr(slot_mapping), n, _stream(stream)),
           "memra_kv_append")


def _decode_args(cache, q, page_table, seq_lens, max_seq_len, out, workspace, sm_scale):
    B, Q, Hq, D = q.shape
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    return (cache.ref, _ptr(q), _ptr(page_table), int(page_table.shape[1]), _ptr(seq_lens), int(max_seq_len), B, Q,
            Hq, cache.n_kv_heads, D, float(sm_scale if sm_scale is not None else D ** -0.5), _ptr(workspace),
            ws_bytes, _ptr(out))


def decode_attn(cache: KVCache, q, page_table, seq_lens, max_seq_len: int, out, workspace, sm_scale=None,
                stream=None, window: int = 0) -> None:
    """memra_decode_attn: q fp16 [B, Q, Hq, D] -> out fp16 [B, Q, Hq, D].

    window > 0: memra_decode_attn_window (sliding window; page_table rows are rings).
    """
    a = _decode_args(cache, q, page_table, seq_lens, max_seq_len, out, workspace, sm_scale)
    if window:
        _check(lib().memra_decode_attn_window(*a[:12], int(window), *a[12:], _stream(stream)),
               "memra_decode_attn_window")
        return
    _check(lib().memra_decode_attn(*a, _stream(stream)), "memra_decode_attn")


def decode_attn_partials(cache: KVCache, q, page_table, seq_lens, max_seq_len: int, out, workspace, sm_scale=None,
                         stream=None) -> None:
    _check(lib().memra_decode_attn_partials(*_decode_args(cache, q, page_table, seq_lens, max_seq_len, out, workspace,
                                                          sm_scale), _stream(stream)), "memra_decode_attn_partials")


def decode_attn_combine(cache: KVCache, seq_lens, max_seq_len: int, max_pages_per_seq: int, batch: int, q_len: int,
                        n_heads: int, out, workspace, stream=None) -> None:
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib().memra_decode_attn_combine(cache.ref, _ptr(seq_lens), int(max_seq_len), int(max_pages_per_seq), batch,
                                           q_len, n_heads, cache.head_dim, _ptr(workspace), ws_bytes, _ptr(out),
                                           _stream(stream)), "memra_decode_attn_combine")


def decode_step(cache: KVCache, k_new, v_new, q, page_table, seq_lens, max_seq_len: int, out, workspace,
                sm_scale=None, stream=None, window: int = 0) -> None:
    """memra_decode_step: store the step's rows (k_new, v_new fp16 [B, Q, Hkv, D]) and attend, in one pass.

    seq_lens include the Q new tokens; their rows go to the positions
    seq_lens[b] - Q .. seq_lens[b] - 1 of each sequence's pages.  window > 0:
    memra_decode_step_window (sliding window; page_table rows are rings).
    """
    a = _decode_args(cache, q, page_table, seq_lens, max_seq_len, out, workspace, sm_scale)
    if window:
        _check(lib().memra_decode_step_window(a[0], _ptr(k_new), _ptr(v_new), *a[1:12], int(window), *a[12:],
                                              _stream(stream)), "memra_decode_step_window")
        return
    _check(lib().memra_decode_step(a[0], _ptr(k_new), _ptr(v_new), *a[1:], _stream(stream)), "memra_decode_step")


def decode_attn_cascade_workspace_bytes(batch: int, q_len: int, n_heads: int, head_dim: int, max_seq_len: int,
                                        prefix_len: int) -> int:
    return int(lib().memra_decode_attn_cascade_workspace_bytes(batch, q_len, n_heads, head_dim, max_seq_len,
                                                               prefix_len))


def decode_attn_cascade(cache: KVCache, q, page_table, seq_lens, max_seq_len: int, prefix_len: int, out, workspace,
                        sm_scale=None, stream=None, k_new=None, v_new=None) -> None:
    """memra_decode_attn_cascade (or memra_decode_step_cascade when k_new / v_new are given).

    Keys 0 .. prefix_len - 1 of every sequence are the pages of page_table row
    0's first prefix_len / 16 columns, attended once per KV head for all rows
    on the tcgen05 tensor cores; each sequence's own keys go through the split
    kernel; the workspace is decode_attn_cascade_workspace_bytes(...).
    """
    a = _decode_args(cache, q, page_table, seq_lens, max_seq_len, out, workspace, sm_scale)
    if k_new is not None or v_new is not None:
        _check(lib().memra_decode_step_cascade(a[0], _ptr(k_new), _ptr(v_new), *a[1:6], int(prefix_len), *a[6:],
                                               _stream(stream)), "memra_decode_step_cascade")
        return
    _check(lib().memra_decode_attn_cascade(*a[:6], int(prefix_len), *a[6:], _stream(stream)),
           "memra_decode_attn_cascade")


NOALLOC_SCRATCH_BYTES = 16 << 20


def decode_attn_noalloc(cache: KVCache, q, page_table, seq_lens, max_seq_len: int, out, sm_scale=None,
                        stream=None) -> None:
    """memra_decode_attn_noalloc: decode attention without a workspace, for callers that cannot allocate.

    The split-K partials go to a fixed library-owned device array of
    NOALLOC_SCRATCH_BYTES; calls that may overlap on the GPU race on it.
    """
    B, Q, Hq, D = q.shape
    _check(lib().memra_decode_attn_noalloc(cache.ref, _ptr(q), _ptr(page_table), int(page_table.shape[1]),
                                           _ptr(seq_lens), int(max_seq_len), B, Q, Hq, cache.n_kv_heads, D,
                                           float(sm_scale if sm_scale is not None else D ** -0.5), _ptr(out),
                                           _stream(stream)), "memra_decode_attn_noalloc")


def _need_dense(where: str, *wanted) -> int:
    """Refuse tensors that are not dense, not of the (dtype, shape) wanted, or not on the current device: its index."""
    device = _device()
    for t, dtype, shape in wanted:
        if t.dtype is not dtype or t.shape != shape or t.get_device() != device or not t.is_contiguous():
            raise MemraError(1, where)
    return device


def prompt_attn(q, k, v, cu_seqlens, out, sm_scale=None, window: int = 0, status=None, stream=None) -> None:
    """memra_prompt_attn: causal attention of packed prompts.

    q fp16 [tokens, Hq, D], k and v fp16 [tokens, Hkv, D]: any token stride, a
    token's heads dense (views of one fused QKV buffer will do); cu_seqlens
    int32 [B + 1]; out fp16 [tokens, Hq, D], dense.  status: a device int32
    the kernel ORs DEVERR_* bits into (KVCache.status will do).
    """
    a = _prompt_args(q, k, v, cu_seqlens, out, sm_scale, window, status)
    _check(lib().memra_prompt_attn(*a, _stream(stream)), "memra_prompt_attn")


def _prompt_args(q, k, v, cu_seqlens, out, sm_scale, window, status):
    import torch
    T, Hq, D = q.shape
    Hkv = k.shape[1]
    _need_dense("memra_prompt_attn", (out, torch.float16, q.shape), (cu_seqlens, torch.int32, cu_seqlens.shape))
    if cu_seqlens.dim() != 1 or (status is not None and (status.dtype is not torch.int32 or status.numel() < 1 or
                                                         status.get_device() != out.get_device())):
        raise MemraError(1, "memra_prompt_attn")
    strides = []
    for x in (q, k, v):
        s = x.stride()
        if (x.shape != (T, Hq if x is q else Hkv, D) or s[2] != 1 or (x.shape[1] > 1 and s[1] != D) or
                x.dtype is not torch.float16 or x.get_device() != out.get_device()):
            raise MemraError(1, "memra_prompt_attn")
        strides.append(s[0] if T > 1 else x.shape[1] * D)
    return (_ptr(q), strides[0], _ptr(k), strides[1], _ptr(v), strides[2], _ptr(cu_seqlens),
            int(cu_seqlens.shape[0]) - 1, T, Hq, Hkv, D, float(sm_scale if sm_scale is not None else D ** -0.5),
            int(window), _ptr(out), _ptr(status))


def tree_attn_workspace_bytes(batch: int, n_nodes: int, n_heads: int, head_dim: int, max_seq_len: int) -> int:
    return int(lib().memra_tree_attn_workspace_bytes(batch, n_nodes, n_heads, head_dim, max_seq_len))


def tree_attn(cache: KVCache, q, page_table, seq_lens, max_seq_len: int, tree_mask, out, workspace, sm_scale=None,
              stream=None) -> None:
    """memra_tree_attn: q fp16 [B, N, Hq, D], a tree of N drafted nodes per sequence -> out fp16 [B, N, Hq, D].

    The tree's rows are the last N of each sequence (seq_lens include them).
    tree_mask int64 [B, N]: bit j of word [b, i] shows node j to node i; every
    node sees all keys before the tree.
    """
    a = _tree_args(cache, q, page_table, seq_lens, max_seq_len, tree_mask, out, workspace, sm_scale)
    _check(lib().memra_tree_attn(*a, _stream(stream)), "memra_tree_attn")


def _tree_args(cache, q, page_table, seq_lens, max_seq_len, tree_mask, out, workspace, sm_scale):
    import torch
    B = q.shape[0]
    device = _need_dense("memra_tree_attn", (q, torch.float16, q.shape), (out, torch.float16, q.shape),
                         (page_table, torch.int32, (B, page_table.shape[1])), (seq_lens, torch.int32, (B,)),
                         (tree_mask, torch.int64, q.shape[:2]))
    if cache.device_index != device or (workspace is not None and workspace.get_device() != device):
        raise MemraError(1, "memra_tree_attn")
    a = _decode_args(cache, q, page_table, seq_lens, max_seq_len, out, workspace, sm_scale)
    # (the decode calls' arguments, the mask behind max_seq_len)
    return (*a[:6], _ptr(tree_mask), *a[6:])


def kv_copy_pages(cache: KVCache, src_pages, dst_pages, n: int | None = None, stream=None) -> None:
    """memra_kv_copy_pages: page src_pages[i] -> dst_pages[i] in both pools; int32 [n] on the device, negative skips."""
    import torch
    most = src_pages.shape[0]
    device = _need_dense("memra_kv_copy_pages", (src_pages, torch.int32, (most,)), (dst_pages, torch.int32, (most,)))
    if n is None:
        n = most
    if n > most or cache.device_index != device:
        raise MemraError(1, "memra_kv_copy_pages")
    rc = lib().memra_kv_copy_pages(cache.ref, src_pages.data_ptr(), dst_pages.data_ptr(), int(n), _stream(stream))
    _check(rc, "memra_kv_copy_pages")


def kv_compact(cache: KVCache, page_table, seq_lens, max_seq_len: int, accepted, n_accepted, n_nodes: int,
               stream=None) -> None:
    """memra_kv_compact: the rows of nodes accepted[b, :n_accepted[b]] move to the front of sequence b's tree rows.

    accepted int32 [B, max_accepted], n_accepted int32 [B]; seq_lens include
    the n_nodes rows of the tree.
    """
    import torch
    B, most = accepted.shape
    pages = page_table.shape[-1]
    i32 = torch.int32
    device = _need_dense("memra_kv_compact", (accepted, i32, (B, most)), (n_accepted, i32, (B,)),
                         (page_table, i32, (B, pages)), (seq_lens, i32, (B,)))
    if cache.device_index != device:
        raise MemraError(1, "memra_kv_compact")
    rc = lib().memra_kv_compact(cache.ref, page_table.data_ptr(), pages, seq_lens.data_ptr(), int(max_seq_len),
                                accepted.data_ptr(), most, n_accepted.data_ptr(), B, int(n_nodes), _stream(stream))
    _check(rc, "memra_kv_compact")


def _dense(where: str, t, dtype, shape, device: int) -> int:
    """The address of a dense tensor of the type, shape and device wanted; refuses others."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != device or not t.is_contiguous():
        raise MemraError(1, where)
    return t.data_ptr()


def _rows(where: str, x, dtype, shape, device: int):
    """The address and token stride of rows x [tokens, heads, dim] whose heads lie side by side; refuses others."""
    a, b, c = x.stride() if x.dim() == 3 else (0, 0, 0)
    if x.dtype is not dtype or x.shape != shape or x.get_device() != device or c != 1 or (b != shape[2] and shape[1] > 1):
        raise MemraError(1, where)
    return x.data_ptr(), a if shape[0] > 1 else shape[1] * shape[2]


def qk_norm_rope(q, k, positions, inv_freq, q_out, k_out=None, q_weight=None, k_weight=None, eps: float = 1e-6,
                 interleaved: bool = False, cache: KVCache | None = None, v=None, slot_mapping=None,
                 stream=None) -> None:
    """memra_qk_norm_rope: norm and rotation of query and key rows, and their append, in one pass.

    q fp16 [tokens, Hq, D], k and v fp16 [tokens, Hkv, D], any token stride;
    q_weight, k_weight float32 [D] or None (no norm); positions int32 [tokens]
    and inv_freq float32 [rotary_dim / 2] (None: no rotation).  q_out and k_out
    are rows like q and k (or q and k themselves).  cache, v and slot_mapping
    int32 [tokens] together store the finished rows; k is None if it goes nowhere.
    """
    import torch
    where, f16, f32, i32 = "memra_qk_norm_rope", torch.float16, torch.float32, torch.int32
    T, Hq, D = shape = q.shape
    Hkv = k.shape[1] if k is not None else 1
    kv_shape, device = (T, Hkv, D), _device()
    pq, sq = _rows(where, q, f16, shape, device)
    po, so = _rows(where, q_out, f16, shape, device)
    pk, sk = _rows(where, k, f16, kv_shape, device) if k is not None else (0, 0)
    pv, sv = _rows(where, v, f16, kv_shape, device) if v is not None else (0, 0)
    pko, sko = _rows(where, k_out, f16, kv_shape, device) if k_out is not None else (0, 0)
    half = inv_freq.numel() if inv_freq is not None else 0
    if cache is not None and cache.device_index != device:
        raise MemraError(1, where)
    rc = lib().memra_qk_norm_rope(
        pq, sq, pk, sk, pv, sv, _dense(where, q_weight, f32, (D,), device) if q_weight is not None else 0,
        _dense(where, k_weight, f32, (D,), device) if k_weight is not None else 0, eps,
        _dense(where, positions, i32, (T,), device) if positions is not None else 0,
        _dense(where, inv_freq, f32, (half,), device) if half else 0, 2 * half, 1 if interleaved else 0, T, Hq, Hkv, D,
        po, so, pko, sko, cache.ref if cache is not None else None,
        _dense(where, slot_mapping, i32, (T,), device) if slot_mapping is not None else 0, _stream(stream))
    if rc:
        raise MemraError(rc, where)


def chunk_attn_workspace_bytes(head_dim: int) -> int:
    return int(lib().memra_chunk_attn_workspace_bytes(head_dim))


def chunk_attn(cache: KVCache, q, cu_seqlens, page_table, seq_lens, max_seq_len: int, out, workspace, sm_scale=None,
               window: int = 0, lse=None, stream=None) -> None:
    """memra_chunk_attn: attention of the new tokens of every sequence over the cache that holds them and their context.

    q fp16 [tokens, Hq, D] (any token stride), sequence b's rows cu_seqlens[b] ..
    cu_seqlens[b + 1] - 1 (int32 [B + 1]); seq_lens int32 [B] include them; out
    fp16 [tokens, Hq, D]; lse float32 [tokens, Hq] or None; workspace of
    chunk_attn_workspace_bytes(D) bytes.  window > 0: page_table rows are rings.
    """
    a = _chunk_args(cache, q, cu_seqlens, page_table, seq_lens, max_seq_len, out, workspace, sm_scale, window, lse)
    _check(lib().memra_chunk_attn(*a, _stream(stream)), "memra_chunk_attn")


def _chunk_args(cache, q, cu_seqlens, page_table, seq_lens, max_seq_len, out, workspace, sm_scale, window, lse):
    import torch
    where, f16, i32 = "memra_chunk_attn", torch.float16, torch.int32
    T, Hq, D = shape = q.shape
    B, pages = table = page_table.shape
    device = _device()
    if cache.device_index != device or workspace is None or workspace.get_device() != device:
        raise MemraError(1, where)
    pq, sq = _rows(where, q, f16, shape, device)
    return (cache.ref, pq, sq, _dense(where, cu_seqlens, i32, (B + 1,), device),
            _dense(where, page_table, i32, table, device), pages, _dense(where, seq_lens, i32, (B,), device),
            int(max_seq_len), B, T, Hq, cache.n_kv_heads, D, D ** -0.5 if sm_scale is None else sm_scale, int(window),
            workspace.data_ptr(), workspace.nbytes, _dense(where, out, f16, shape, device),
            _dense(where, lse, torch.float32, (T, Hq), device) if lse is not None else 0)


def key_weights(cache: KVCache, q, lse, cu_seqlens, page_table, seq_lens, max_seq_len: int, weights, keep: float = 1.0,
                sm_scale=None, stream=None) -> None:
    """memra_key_weights: adds to weights what each key collects from the rows of a chunk.

    q, cu_seqlens, page_table, seq_lens as in chunk_attn, lse float32 [tokens,
    Hq] as it writes them; weights float32 [B, Hkv, >= max_seq_len], times keep first
    (so that those of new tokens must be set, to 0 as a rule, unless keep is 0).
    """
    a = _weight_args(cache, q, lse, cu_seqlens, page_table, seq_lens, max_seq_len, weights, keep, sm_scale)
    _check(lib().memra_key_weights(*a, _stream(stream)), "memra_key_weights")


def _weight_args(cache, q, lse, cu_seqlens, page_table, seq_lens, max_seq_len, weights, keep, sm_scale):
    import torch
    where, f32, i32 = "memra_key_weights", torch.float32, torch.int32
    T, Hq, D = shape = q.shape
    B, pages = table = page_table.shape
    device, Hkv, row = _device(), cache.n_kv_heads, weights.shape[-1]
    if cache.device_index != device:
        raise MemraError(1, where)
    pq, sq = _rows(where, q, torch.float16, shape, device)
    return (cache.ref, pq, sq, _dense(where, lse, f32, (T, Hq), device), _dense(where, cu_seqlens, i32, (B + 1,), device),
            _dense(where, page_table, i32, table, device), pages, _dense(where, seq_lens, i32, (B,), device),
            int(max_seq_len), B, T, Hq, Hkv, D, D ** -0.5 if sm_scale is None else sm_scale, keep,
            _dense(where, weights, f32, (B, Hkv, row), device), row)


def kv_evict(cache: KVCache, page_table, seq_lens, max_seq_len: int, weights, budgets, dst_table, kept, sink: int = 0,
             recent: int = 0, new_weights=None, new_lens=None, stream=None) -> None:
    """memra_kv_evict: the budgets[b] rows of largest weight of each KV head move to the pages of dst_table.

    weights float32 [B, Hkv, >= max_seq_len]; budgets int32 [B], at most
    kept.shape[2]; dst_table int32 [B, pages] of pages that nothing else uses;
    kept int32 [B, Hkv, max_budget] receives the kept indices, new_weights
    float32 [B, Hkv, >= max_budget] their weights, new_lens int32 [B] how many
    (seq_lens or budgets themselves will do).
    """
    import torch
    where, f32, i32 = "memra_kv_evict", torch.float32, torch.int32
    B, Hkv, most = shape = kept.shape
    device, pages, to, row = _device(), page_table.shape[-1], dst_table.shape[-1], weights.shape[-1]
    if cache.device_index != device or Hkv != cache.n_kv_heads:
        raise MemraError(1, where)
    new_row = new_weights.shape[-1] if new_weights is not None else 0
    rc = lib().memra_kv_evict(
        cache.ref, _dense(where, page_table, i32, (B, pages), device), pages,
        _dense(where, seq_lens, i32, (B,), device), int(max_seq_len),
        _dense(where, weights, f32, (B, Hkv, row), device), row, _dense(where, budgets, i32, (B,), device), most,
        int(sink), int(recent), _dense(where, dst_table, i32, (B, to), device), to, B,
        _dense(where, kept, i32, shape, device),
        _dense(where, new_weights, f32, (B, Hkv, new_row), device) if new_weights is not None else 0, new_row,
        _dense(where, new_lens, i32, (B,), device) if new_lens is not None else 0, _stream(stream))
    if rc:
        raise MemraError(rc, where)
    if most == 0 and new_lens is not None:             # (the entry point has done nothing)
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream)
        with torch.cuda.stream(stream):
            new_lens.zero_()


def testing_decode_attn_short_page(cache: KVCache, q, page_table, seq_lens, max_seq_len: int, out, workspace,
                                   page_wait_ns: int, sm_scale=None, stream=None) -> None:
    """memra_testing_decode_attn_short_page (memra_testing.h): decode attention whose first CTA's first
    page wait cannot complete and runs out after page_wait_ns; the call then flags DEVERR_TIMEOUT."""
    a = _decode_args(cache, q, page_table, seq_lens, max_seq_len, out, workspace, sm_scale)
    _check(lib().memra_testing_decode_attn_short_page(*a, int(page_wait_ns), _stream(stream)),
           "memra_testing_decode_attn_short_page")


def testing_prompt_attn_short_copy(q, k, v, cu_seqlens, out, sm_scale=None, window: int = 0, status=None,
                                   stream=None) -> None:
    """memra_testing_prompt_attn_short_copy (memra_testing.h): prompt attention whose CTA 0 waits for a copy that
    cannot complete; the waits run out, the CTA's rows become NaN and DEVERR_TIMEOUT is flagged."""
    a = _prompt_args(q, k, v, cu_seqlens, out, sm_scale, window, status)
    _check(lib().memra_testing_prompt_attn_short_copy(*a, _stream(stream)),
           "memra_testing_prompt_attn_short_copy")


def testing_tree_attn_short_page(cache: KVCache, q, page_table, seq_lens, max_seq_len: int, tree_mask, out, workspace,
                                 sm_scale=None, stream=None) -> None:
    """memra_testing_tree_attn_short_page (memra_testing.h): the same for tree attention's first chunk."""
    a = _tree_args(cache, q, page_table, seq_lens, max_seq_len, tree_mask, out, workspace, sm_scale)
    _check(lib().memra_testing_tree_attn_short_page(*a, _stream(stream)),
           "memra_testing_tree_attn_short_page")


def testing_chunk_attn_short_page(cache: KVCache, q, cu_seqlens, page_table, seq_lens, max_seq_len: int, out, workspace,
                                  sm_scale=None, window: int = 0, lse=None, stream=None) -> None:
    """memra_testing_chunk_attn_short_page (memra_testing.h): the same for chunk attention's first chunk of keys."""
    a = _chunk_args(cache, q, cu_seqlens, page_table, seq_lens, max_seq_len, out, workspace, sm_scale, window, lse)
    _check(lib().memra_testing_chunk_attn_short_page(*a, _stream(stream)), "memra_testing_chunk_attn_short_page")


def testing_key_weights_short_page(cache: KVCache, q, lse, cu_seqlens, page_table, seq_lens, max_seq_len: int, weights,
                                   keep: float = 1.0, sm_scale=None, stream=None) -> None:
    """memra_testing_key_weights_short_page (memra_testing.h): the same for the key weights' first chunk of keys."""
    a = _weight_args(cache, q, lse, cu_seqlens, page_table, seq_lens, max_seq_len, weights, keep, sm_scale)
    _check(lib().memra_testing_key_weights_short_page(*a, _stream(stream)), "memra_testing_key_weights_short_page")


def testing_scale_division_mismatches(scales, mismatches, stream=None) -> None:
    """memra_testing_scale_division_mismatches (memra_testing.h): adds to mismatches (one int64 on the device)
    the (fp16 x, scale) pairs whose division-free quotient differs from the IEEE one."""
    _check(lib().memra_testing_scale_division_mismatches(_ptr(scales), int(scales.numel()), _ptr(mismatches),
                                                         _stream(stream)), "memra_testing_scale_division_mismatches")


def read_status(cache: KVCache, stream=None) -> int:
    """memra_read_status: synchronizes, returns and clears the device error bits."""
    flags = ctypes.c_int32(0)
    rc = lib().memra_read_status(cache.ref, ctypes.byref(flags), _stream(stream))
    if rc not in (0, 5):
        raise MemraError(rc, "memra_read_status")
    return int(flags.value)
