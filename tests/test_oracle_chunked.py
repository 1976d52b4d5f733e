"""Pins of the oracle of the chunk operators: closed forms, brute force, library routines (CPU only)."""
import itertools

import numpy as np
import pytest

from oracle import chunked


def test_rotation_turns_unit_pairs_by_the_angle():
    for interleaved in (False, True):
        first, second = chunked.rope_pairs(8, interleaved)
        x = np.zeros((1, 1, 32))
        x[..., first] = 1.0
        freq = np.linspace(0.1, 0.8, 8)
        y = chunked.norm_rope_rows(x, None, 0.0, [3], freq, interleaved)
        assert np.allclose(y[0, 0, first], np.cos(3 * freq)) and np.allclose(y[0, 0, second], np.sin(3 * freq))
        assert np.array_equal(y[..., 16:], x[..., 16:])


def test_rotation_keeps_lengths_and_relative_angles():
    rng = np.random.default_rng(0)
    q, k, freq = rng.standard_normal((1, 1, 64)), rng.standard_normal((1, 1, 64)), 10000.0 ** (-np.arange(32) / 32)
    turn = lambda x, p: chunked.norm_rope_rows(x, None, 0.0, [p], freq, False)
    assert np.allclose(np.linalg.norm(turn(q, 1000)), np.linalg.norm(q))
    assert np.allclose((turn(q, 1005) * turn(k, 1000)).sum(), (turn(q, 5) * k).sum())
    assert np.allclose(turn(turn(q, 7), -7), q)


def test_norm_makes_the_mean_square_one():
    x = np.random.default_rng(1).standard_normal((3, 2, 128)) * 7
    y = chunked.norm_rope_rows(x, np.full(128, 2.0), 0.0, None, None, False)
    assert np.allclose((y * y).mean(-1), 4.0)
    assert np.allclose(chunked.norm_rope_rows(np.zeros((1, 1, 128)), np.ones(128), 1e-6, None, None, False), 0.0)


def test_chunk_against_a_library_routine():
    torch = pytest.importorskip("torch")
    rng = np.random.default_rng(2)
    for n, T, window in ((1, 1, 0), (1, 9, 0), (5, 9, 0), (9, 9, 0), (5, 9, 3), (4, 9, 1)):
        q, k, v = rng.standard_normal((n, 4, 8)), rng.standard_normal((T, 2, 8)), rng.standard_normal((T, 2, 8))
        out, lse = chunked.chunk_rows(q, k, v, window, 0.3)
        sees = chunked.chunk_sees(n, T, window)
        assert all(sees[i, j] == (j <= T - n + i and (not window or j > T - n + i - window))
                   for i, j in itertools.product(range(n), range(T)))
        t = lambda x: torch.from_numpy(x).transpose(0, 1)
        want = torch.nn.functional.scaled_dot_product_attention(
            t(q), t(k).repeat_interleave(2, 0), t(v).repeat_interleave(2, 0), attn_mask=torch.from_numpy(sees), scale=0.3)
        assert np.allclose(out, want.transpose(0, 1).numpy())
        s = chunked.logits(q, k, sees, 0.3)
        assert np.allclose(lse, torch.logsumexp(torch.from_numpy(s), -1).numpy().T)


def test_key_weights_sum_to_the_rows():
    rng = np.random.default_rng(3)
    q, k = rng.standard_normal((6, 8, 16)), rng.standard_normal((20, 2, 16))
    _, lse = chunked.chunk_rows(q, k, k, 0, 0.25)
    w = chunked.key_weights(q, k, lse, 0.25)
    assert w.shape == (2, 20) and np.allclose(w.sum(1), 6 * 4)
    assert np.allclose(chunked.key_weights(q[:1], k[:1], lse[:1] * 0 + (q[:1].reshape(1, 2, 4, 16) * k[:1, :, None]).sum(-1)
                                           .reshape(1, 8) * 0.25, 0.25), 4.0)


def test_kept_tokens_brute_force():
    rng = np.random.default_rng(4)
    for _ in range(300):
        T = int(rng.integers(1, 9))
        w = rng.integers(0, 4, T).astype(np.float64)
        n, sink, recent = (int(x) for x in rng.integers(0, 6, 3))
        got = chunked.kept_tokens(w, n, sink, recent)
        n = min(n, T)
        r = min(recent, n)
        s = min(sink, n - r)
        forced = set(range(s)) | set(range(T - r, T))
        assert len(got) == n and forced <= set(got) and list(got) == sorted(set(got))
        free = [i for i in range(T) if i not in forced]
        # the best choice: largest sum, and of equal ones the lexicographically first
        best = max(itertools.combinations(free, n - r - s), key=lambda c: (sorted((w[i] for i in c), reverse=True),
                                                                          [-i for i in c]), default=())
        assert forced | set(best) == set(got)


def test_kept_tokens_nan_weighs_least():
    w = np.array([np.nan, -np.inf, 0.0, np.nan, 2.0])
    assert list(chunked.kept_tokens(w, 3, 0, 0)) == [1, 2, 4]
    assert list(chunked.kept_tokens(w, 4, 0, 0)) == [0, 1, 2, 4]
