"""Caches, chunks and expected rows for the GPU tests of chunk attention, key weights and eviction."""
import numpy as np
import torch

from oracle import chunked, quant

PAIRS = [("q8_0", "q5_1"), ("q8_0", "q4_0"), ("fp8", "fp8"), ("nvfp4", "nvfp4"), ("fp8", "q5_1"), ("nvfp4", "q4_0")]


def dev(a, dtype=None):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=dtype)).cuda()


def dequantized(rows, fmt, scale):
    """[T, D] fp16 rows as the cache holds them, float64."""
    return quant.dequantize_rows(quant.quantize_rows(rows, fmt, scale))


class Chunk:
    """Sequences of past[b] cached and new[b] new tokens in a paged cache, and their queries."""

    def __init__(self, memra, kf, vf, D, Hq, Hkv, new, past, window=0, seed=0, pad=0, extra_columns=0, k_gain=1.0,
                 q_gain=1.0, v_of=None, stride_heads=0, fill=True):
        rng = np.random.default_rng(seed)
        self.memra, self.kf, self.vf, self.D, self.Hq, self.Hkv, self.window = memra, kf, vf, D, Hq, Hkv, window
        self.new, self.past, self.lens = new, past, [n + p for n, p in zip(new, past)]
        B = len(new)
        self.scales = [5.0 / 448 if f == "fp8" else 5.0 / 2688 if f == "nvfp4" else 1.0 for f in (kf, vf)]
        if window:
            cols = [(window + max(max(new), 1) - 2) // 16 + 2 + extra_columns] * B
        else:
            cols = [max(1, -(-T // 16)) for T in self.lens]
        pages = sum(cols) + 3
        order = rng.permutation(pages)
        self.table = np.full((B, max(cols) + (0 if window else extra_columns)), 2 ** 30, np.int32)
        for b, c in enumerate(cols):
            self.table[b, :c] = order[sum(cols[:b]):sum(cols[:b + 1])]
        self.cache = memra.KVCache(kf, vf, pages, Hkv, D, *self.scales)
        if fill:                             # what nobody wrote may hold anything
            g = torch.Generator(device="cuda").manual_seed(seed)
            for pool in (self.cache.k_pool, self.cache.v_pool):
                pool.copy_(torch.randint(0, 256, pool.shape, dtype=torch.uint8, device="cuda", generator=g))
        self.rows = []
        for b, T in enumerate(self.lens):
            first = max(0, T - self.table.shape[1] * 16) if window else 0
            some, heads = min(Hkv, 8), np.arange(Hkv) % 8          # (many heads repeat eight)
            k = (rng.standard_normal((T - first, some, D)) * k_gain).astype(np.float16)[:, heads]
            v = (rng.standard_normal((T - first, some, D)) if v_of is None else
                 v_of(T - first, some, D)).astype(np.float16)[:, heads]
            self.rows.append((first, k, v))
            for lo in range(first, T, 65536):
                pos = np.arange(lo, min(T, lo + 65536))
                slots = self.table[b, pos // 16 % self.table.shape[1]] * 16 + pos % 16
                memra.kv_append(self.cache, dev(k[pos - first]), dev(v[pos - first]), dev(slots.astype(np.int32)))
        total = sum(new) + pad
        buf = (rng.standard_normal((total, Hq + stride_heads, D)) * q_gain).astype(np.float16)
        self.buf, self.q = dev(buf), buf[:, :Hq]
        self.starts = np.concatenate(([0], np.cumsum(new))).astype(np.int32)
        self.out = torch.full((total, Hq, D), -7.0, dtype=torch.float16, device="cuda")
        self.lse = torch.full((total, Hq), -7.0, device="cuda")
        self.ws = torch.full((memra.chunk_attn_workspace_bytes(D),), 255, dtype=torch.uint8, device="cuda")

    def args(self, want_lse=True):
        return dict(q=self.buf[:, :self.Hq], cu_seqlens=dev(self.starts), page_table=dev(self.table),
                    seq_lens=dev(np.array(self.lens, np.int32)), max_seq_len=max(self.lens), out=self.out,
                    workspace=self.ws, window=self.window, lse=self.lse if want_lse else None)

    def call(self, want_lse=True, **kw):
        self.memra.chunk_attn(self.cache, **{**self.args(want_lse), **kw})
        return self.memra.read_status(self.cache)

    def keys(self, b, h):
        """Dequantized K and V of a KV head, and the position of the first."""
        first, k, v = self.rows[b]
        return first, dequantized(k[:, h], self.kf, self.scales[0]), dequantized(v[:, h], self.vf, self.scales[1])

    operand = 0.0

    def expected(self, b, h):
        """Rows of sequence b and KV head h: out [n, G, D], lse [n, G] and how far each may be off.

        To first order, with p the weights and d_u the errors of the scores:
        |out - o| <= sum_u p_u (|d_u| |v_u - o| + (2^-11 + A) |v_u|) + 2^-11 |o|: a weight rounded to fp16, the output's
        rounding, and the accumulator, whose last bit is cut at each of up to 480 steps of a sum (960 with hi and lo parts:
        A = 960 * 2^-23), and 2^-19 for the sums of weights, the exponential and the joins.
        d_u: the accumulator of the score, cut at each of D / 16 steps (twice for pairs).
        The integer formats enter as fp16 pairs of half their value.  Below fp16's normal range a rounding is off by half of
        2^-24, whatever the value: K^ by up to 2^-24 (2^-24 sum |q_j| in the score), V^ likewise.
        `operand`: what K^ and V^ are off by, relative, where an operator rounds them (2^-11: to fp16).
        """
        G, n = self.Hq // self.Hkv, self.new[b]
        first, k, v = self.keys(b, h)
        T = self.lens[b]
        sees = chunked.chunk_sees(n, T, self.window)[:, first:]
        q = self.q[self.starts[b]:self.starts[b + 1], h * G:(h + 1) * G].astype(np.float64)
        scale = self.D ** -0.5
        per_key = 2.0 ** -23 * (self.D / 8) + self.operand
        out, tol = np.zeros((n, G, self.D)), np.zeros((n, G, self.D))
        lse, lse_tol = np.full((n, G), -np.inf), np.zeros((n, G))
        for g in range(G):
            s = np.where(sees, q[:, g] @ k.T * scale, -np.inf)
            top = s.max(1, initial=-np.inf, keepdims=True)
            top[~np.isfinite(top)] = 0.0
            e = np.exp(s - top)
            mass = e.sum(1, keepdims=True)
            p = np.divide(e, mass, out=np.zeros_like(e), where=mass > 0)
            out[:, g] = p @ v
            d = np.abs(q[:, g]) @ np.abs(k).T * scale * per_key
            if self.kf == "q8_0":
                d = d + np.abs(q[:, g]).sum(1, keepdims=True) * scale * 2.0 ** -24
            av = np.abs(v)
            # |v - o| <= |v| + |o|
            tol[:, g] = 1.05 * ((p * d) @ av + (p * d).sum(1, keepdims=True) * np.abs(out[:, g])) + \
                (2.0 ** -11 + 960 * 2.0 ** -23 + 2.0 ** -19 + self.operand) * (p @ av) + 2.0 ** -11 * np.abs(out[:, g]) + 2.0 ** -23
            with np.errstate(divide="ignore"):
                lse[:, g] = np.where(mass[:, 0] > 0, np.log(mass[:, 0]) + top[:, 0], -np.inf)
            lse_tol[:, g] = 1.05 * (p * d).sum(1) + 2.0 ** -19 + 2.0 ** -22 * np.where(np.isfinite(lse[:, g]), np.abs(lse[:, g]), 0)
        return out, tol, lse, lse_tol

    def check(self, lse=True, sequences=None, heads=None):
        G = self.Hq // self.Hkv
        got, got_lse = self.out.cpu().numpy().astype(np.float64), self.lse.cpu().numpy().astype(np.float64)
        worst = 0.0
        for b in range(len(self.new)) if sequences is None else sequences:
            rows = slice(self.starts[b], self.starts[b + 1])
            for h in range(self.Hkv) if heads is None else heads:
                out, tol, want_lse, lse_tol = self.expected(b, h)
                err = np.abs(got[rows, h * G:(h + 1) * G] - out)
                assert (err <= tol).all(), f"sequence {b} head {h}: {np.nanmax(err / tol)} of the tolerance"
                worst = max(worst, float((err / tol).max(initial=0.0)))
                if lse:
                    l = got_lse[rows, h * G:(h + 1) * G]
                    seen = np.isfinite(want_lse)
                    assert np.array_equal(np.isfinite(l), seen)
                    e = np.abs(l[seen] - want_lse[seen]) / lse_tol[seen]
                    assert (e <= 1).all(), f"lse of sequence {b} head {h}: {e.max()} of the tolerance"
        end = self.starts[-1]
        assert (self.out[end:] == -7).all() and (self.lse[end:] == -7).all()
        return worst
