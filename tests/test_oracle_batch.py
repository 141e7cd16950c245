"""Pins of the references of the calls of several sequences."""

import math

import numpy as np
import pytest
import torch

from oracle import batch as O


def test_e4m3_is_that_of_the_type():
    codes = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(O.from_e4m3(codes), want)
    rng = np.random.default_rng(0)
    x = np.concatenate((rng.standard_normal(5000) * 100, rng.standard_normal(5000) * 1e-2,
                        (O.e4m3_values()[1:] + O.e4m3_values()[:-1]) / 2, [0.0, -0.0, 448.0, -448.0]))
    x = x[np.abs(x) <= 448].astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(O.to_e4m3(x.astype(np.float64)), want)
    assert list(O.to_e4m3(np.array([np.nan, np.inf, -np.inf])) & 0x7F) == [0x7F] * 3


@pytest.mark.parametrize("most,scale", [(448.0, 1.0), (449.0, 2.0), (224.0, 0.5), (224.5, 1.0), (0.0, 1.0),
                                        (1e-30, 2.0 ** -64), (3.0, 2.0 ** -7)])
def test_block_scale(most, scale):
    x = np.zeros((4, 8))
    x[2, 3] = -most
    x[1, 1] = np.inf
    assert O.block_scale(x) == scale
    assert most / scale <= 448


def test_rotation_keeps_lengths_and_adds_up():
    x = np.random.default_rng(1).standard_normal((3, 64))
    y = O.rotate(x, 1234567, 1e4)
    np.testing.assert_allclose((y ** 2).sum(-1), (x ** 2).sum(-1))
    np.testing.assert_allclose(O.rotate(O.rotate(x, 3, 1e4), 4, 1e4), O.rotate(x, 7, 1e4), atol=1e-12)


def test_head_norm():
    x = np.random.default_rng(2).standard_normal((5, 64)) * 9
    y = O.head_norm(x, np.ones(64), 0.0)
    np.testing.assert_allclose((y ** 2).mean(-1), 1.0)
    assert O.head_norm(x, None, 0.0) is x


def test_seen_rows():
    assert list(O.seen_rows(5)) == [0, 1, 2, 3, 4, 5]
    assert list(O.seen_rows(5, window=2, sinks=1)) == [0, 4, 5]
    assert list(O.seen_rows(5, window=1)) == [5]
    assert list(O.seen_rows(3, window=9, sinks=2)) == [0, 1, 2, 3]


def test_attend_is_a_softmax():
    rng = np.random.default_rng(3)
    q, K, V = rng.standard_normal(8), rng.standard_normal((6, 8)), rng.standard_normal((6, 8))
    rows = np.array([0, 2, 5])
    want = torch.nn.functional.scaled_dot_product_attention(
        *(torch.from_numpy(x)[None, None] for x in (q[None], K[rows], V[rows])))
    np.testing.assert_allclose(O.attend(q, K, V, rows, 1 / math.sqrt(8))[0], want[0, 0, 0].numpy())


def test_verification_keeps_the_targets_distribution():
    # over all of the random numbers, by their intervals: the first token is
    # distributed as p
    rng = np.random.default_rng(4)
    V = 5
    p, q = rng.dirichlet(np.ones(V), 2), rng.dirichlet(np.ones(V), 1)
    law = np.zeros(V)
    n = 400
    for y in range(V):
        for i in range(n):
            u = (i + 0.5) / n
            if u * q[0, y] < p[0, y]:
                law[O.verify(p, q, [y], [u], 0.5)[0]] += q[0, y] / n
                continue
            for k in range(n // 4):
                law[O.verify(p, q, [y], [u], (k + 0.5) / (n // 4))[0]] += q[0, y] / n / (n // 4)
    np.testing.assert_allclose(law, p[0], atol=2.0 / n + 4.0 / n)


def test_verification_by_hand():
    p = np.array([[0.5, 0.5, 0.0], [0.1, 0.2, 0.7]])
    assert O.verify(p, None, [0], [0.4], 0.0) == [0, 0]
    assert O.verify(p, None, [0], [0.4], 0.95) == [0, 2]
    assert O.verify(p, None, [0], [0.6], 0.0) == [1]       # p without token 0
    assert O.verify(p, None, [2], [0.0], 0.99) == [1]      # 0 < 0 does not hold
    assert O.verify(p, None, [7], [0.0], 0.0) == [0]
    q = np.array([[0.5, 0.5, 0.0]])
    assert O.verify(p, q, [2], [0.5], 0.6) == [1]          # nothing left: from p itself
    assert O.verify(p[:1], None, [], [], 0.999999) == [1]
    assert O.verify(p[:1], None, [], [], 1.0) == [1]       # the last entry over 0
    assert O.verify(np.zeros((1, 3)), None, [], [], 0.5) == []
