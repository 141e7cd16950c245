"""Pins of the tree-decoding references of oracle/ops.py."""

import numpy as np

from oracle import ops as O
from oracle.numerics import bf16_round


def _cache(rng, Hkv, S, dh):
    return bf16_round(rng.standard_normal((Hkv, S, dh))), bf16_round(rng.standard_normal((Hkv, S, dh)))


def test_a_chain_is_the_decode_attention():
    H, Hkv, dh, n, T = 4, 2, 64, 9, 5
    rng = np.random.default_rng(1)
    K, V = _cache(rng, Hkv, 32, dh)
    qkv = rng.standard_normal((T, (H + 2 * Hkv) * dh))
    want, K1, V1 = O.attention(qkv, n, K, V, H, Hkv, dh, 1e4)
    parents = [-1, 0, 1, 2, 3]
    q, k, v = O.tree_rows(qkv, parents, n, H, Hkv, dh, 1e4)
    np.testing.assert_array_equal(bf16_round(k).transpose(1, 0, 2), K1[:, n:n + T])
    np.testing.assert_array_equal(bf16_round(v).transpose(1, 0, 2), V1[:, n:n + T])
    out, mass, _ = O.tree_attention(q, parents, n, K1, V1)
    np.testing.assert_allclose(out.reshape(T, -1), want, atol=1e-2, rtol=2 ** -7)
    assert np.isclose(mass.sum(), H * T)


def test_each_branch_is_its_own_chain():
    H, Hkv, dh, n = 2, 1, 64, 6
    rng = np.random.default_rng(2)
    parents = [-1, 0, 0, 1, -2, 2, 4]
    T = len(parents)
    K, V = _cache(rng, Hkv, n + T, dh)
    q = rng.standard_normal((T, H, dh))
    out, _, _ = O.tree_attention(q, parents, n, K, V)
    for t, path in enumerate(O.tree_paths(parents)):
        if path is None:
            assert t in (4, 6) and not out[t].any()
            continue
        rows = list(range(n)) + [n + i for i in path]
        alone, _, _ = O.tree_attention(q[path], list(range(-1, len(path) - 1)), n, K[:, rows], V[:, rows])
        np.testing.assert_allclose(out[t], alone[-1], atol=1e-13)


def test_evict_and_select_by_brute_force():
    w = np.array([[5.0, 1, 3, 3, np.nan, 3, 2, 9, 0, 0]])
    np.testing.assert_array_equal(O.cache_evict(w, 10, 6, 1, 2), [[0, 2, 3, 7, 8, 9]])
    np.testing.assert_array_equal(O.cache_evict(w, 8, 8, 0, 0), [list(range(8))])
    z = [[0.0, 2, 2, -np.inf], [5, 1, 0, np.nan]]
    got = O.beam_select(z, [0.0, 3.0], [0.0, 0.0], None, 1, 9)
    assert [g[:2] for g in got] == [(1, 0), (2, 0), (0, 1), (0, 0), (1, 1), (2, 1)] + [(-1, -1)] * 3
    assert O.beam_select(z, [0.0, 3.0], [0.0, 1.5], [0, 1], 3, 3) == [
        (1, 0, 2.0, 0), (2, 0, 2.0, 0), (3, 1, 1.5, 1)]
