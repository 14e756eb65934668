"""Pins of the plain 64-bit forms in plain_ops.py: the generator against its authors' known
answers, the gradients against central differences, the conventions of the edge cases."""
import numpy as np
import pytest

import plain_ops as P


def test_philox_known_answers():
    f = 0xFFFFFFFF
    assert P.philox([0] * 4, [0] * 2) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    assert P.philox([f] * 4, [f] * 2) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    assert P.philox([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], [0xA4093822, 0x299F31D0]) == [
        0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]


def test_dropout_bits_follow_the_counter():
    b = P.dropout_bits(3, 11, seed=7, offset=9)            # two counters a row
    w = P.philox([2 * 2 + 1, 0, 9, 0], [7, 0])             # row 2, columns 8..10
    assert list(b[2, 8:]) == [w[0] & 0xFFFF, w[0] >> 16, w[1] & 0xFFFF]
    assert not np.array_equal(b, P.dropout_bits(3, 11, seed=7, offset=10))
    assert np.array_equal(P.dropout(np.ones((2, 3)), 1.0, 1, 2), np.zeros((2, 3)))
    assert np.array_equal(P.dropout(np.ones((2, 3)), 0.0, 1, 2, np.ones((2, 3))), 2 * np.ones((2, 3)))


@pytest.mark.parametrize("scale", [1.0, 0.6, 1.7])
def test_logprob_gradient_against_differences(scale):
    rng = np.random.default_rng(0)
    T, V = 5, 9
    x = rng.standard_normal((T, V)) * 2
    t = np.array([0, 8, -1, 3, 3])
    x[1, 2:5] = -np.inf                                    # masked
    x[4] = -np.inf
    x[4, 3] = 0.5                                          # only the target is left
    gl, gh = rng.standard_normal(T), rng.standard_normal(T)

    def loss(x):
        logp, h, _ = P.token_logprobs(x, t, scale)
        return (gl * logp).sum() + (gh * h).sum()

    d = P.token_logprobs_grad(x, t, scale, gl, gh)
    eps = 1e-5
    for r in range(T):
        for j in range(V):
            if np.isneginf(x[r, j]):
                assert d[r, j] == 0.0
                continue
            a, b = x.copy(), x.copy()
            a[r, j] += eps
            b[r, j] -= eps
            # central differences: eps^2 * third derivative (of order 1) + rounding / eps
            assert abs((loss(a) - loss(b)) / (2 * eps) - d[r, j]) < 1e-8


def test_embedding_gradient_is_the_transpose():
    rng = np.random.default_rng(1)
    ids = np.array([3, -1, 0, 3, 4, 3, -1])
    table, other = rng.standard_normal((2, 5, 6))
    dout = rng.standard_normal((7, 6))
    g, _, cnt = P.embedding_grad(ids, dout, 5, 1.5)
    lin = (dout * (P.embedding(ids, table + other, 1.5) - P.embedding(ids, table, 1.5))).sum()
    assert abs(lin - (g * other).sum()) < 1e-12
    assert list(cnt) == [1, 0, 0, 3, 1]


def test_edges_of_the_log_probabilities():
    low = float(np.finfo(np.float32).min)
    x = np.array([[low] * 4, [-np.inf] * 4, [0.0, -0.0, 1.0, 1.0]])
    logp, h, lp = P.token_logprobs(x, np.array([1, 2, -1]), 1.0)
    assert logp[0] == -np.log(4) and logp[1] == -np.inf and logp[2] == 0.0
    assert abs(h[0] - np.log(4)) < 1e-15 and h[1] == 0.0
    assert P.top_rows(x, 4).tolist() == [[0, 1, 2, 3], [0, 1, 2, 3], [2, 3, 0, 1]]
