"""Pins of the oracle's masked attention: explicit loops, causal and window masks, empty rows, a chain of nodes."""
import math

import numpy as np
import pytest

from oracle import attention


def loops(q, k, v, sees, scale):
    R, Hq, D = q.shape
    G = Hq // k.shape[1]
    out = np.zeros(q.shape)
    for r in range(R):
        for h in range(Hq):
            keys = [t for t in range(k.shape[0]) if sees[r, t]]
            if not keys:
                continue
            s = [sum(q[r, h, d] * k[t, h // G, d] for d in range(D)) * scale for t in keys]
            e = [math.exp(x - max(s)) for x in s]
            for d in range(D):
                out[r, h, d] = sum(p * v[t, h // G, d] for p, t in zip(e, keys)) / sum(e)
    return out


@pytest.fixture
def rows():
    rng = np.random.default_rng(0)
    return rng.standard_normal((5, 4, 3)), rng.standard_normal((7, 2, 3)), rng.standard_normal((7, 2, 3))


def test_against_loops(rows):
    q, k, v = rows
    sees = np.random.default_rng(1).random((5, 7)) < 0.5
    sees[3] = False                                   # a row that sees nothing
    got = attention.masked_rows(q, k, v, sees, 0.7)
    assert np.abs(got - loops(q, k, v, sees, 0.7)).max() < 1e-12
    assert (got[3] == 0).all()


def test_prompt_masks():
    full = attention.prompt_sees(4)
    assert full.tolist() == [[j <= i for j in range(4)] for i in range(4)]
    assert attention.prompt_sees(4, 2).tolist() == [[i - 2 < j <= i for j in range(4)] for i in range(4)]
    assert attention.prompt_sees(3, 1).tolist() == np.eye(3, dtype=bool).tolist()


def test_causal_rows_agree_with_the_decode_oracle(rows):
    _, k, v = rows
    q = np.random.default_rng(2).standard_normal((7, 4, 3))
    for window in (0, 3):
        got = attention.masked_rows(q, k, v, attention.prompt_sees(7, window), 0.5)
        assert np.abs(got - attention.attention_rows(q, k, v, 0.5, window=window)).max() < 1e-12


def test_a_chain_of_nodes_is_the_causal_verify(rows):
    q, k, v = rows
    words = [(1 << (i + 1)) - 1 for i in range(5)]
    got = attention.masked_rows(q, k, v, attention.tree_sees(words, 2), 0.5)
    assert np.abs(got - attention.attention_rows(q, k, v, 0.5)).max() < 1e-12
