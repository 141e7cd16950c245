"""The tree-decoding calls at the ends of their ranges: scores beyond 32 bits,
infinities in rows that are seen, waits that run out, sizes that are refused."""

import numpy as np
import pytest
import torch

from oracle import ops as O

pytestmark = pytest.mark.gpu

LOWEST = np.finfo(np.float32).min


@pytest.fixture(scope="module")
def ops():
    import __graft_entry__ as g
    g.build()
    import self_speculative_decoding_gb300 as ssd
    return ssd.ops


# --------------------------------------------------------------------------
# selection: sums that leave the 32-bit range


def check_select(ops, z, scores, lse, W, done=None, end_id=-1):
    t = lambda a, dt: None if a is None else torch.from_numpy(np.asarray(a, dt)).cuda()  # noqa: E731
    tok, par, best, dn = (x.cpu().numpy() for x in ops.beam_select(
        t(z, np.float32), t(scores, np.float32), W, lse=t(lse, np.float32), done=t(done, np.int32), end_id=end_id))
    want = O.beam_select(z, lse, scores, done, end_id, W)
    assert list(zip(tok.tolist(), par.tolist())) == [w[:2] for w in want]
    with np.errstate(over="ignore"):
        np.testing.assert_array_equal(best, np.array([w[2] for w in want], np.float64).astype(np.float32))
    assert dn.tolist() == [w[3] for w in want]


# one launch (a cluster) and two
SIZES = [(2, 1024, 4), (2, 1024, 2), (4, 300, 16), (12, 3000, 12), (60, 5000, 60)]


@pytest.mark.parametrize("B,V,W", SIZES)
@pytest.mark.parametrize("score", [0.5, 5.0, 0.0, -1.0])
def test_select_beside_a_beam_masked_as_a_whole(ops, B, V, W, score):
    """z = lse = the type's lowest value: z - lse = 0, and |z| + |lse| is over
    the 32-bit range."""
    rng = np.random.default_rng(B * V)
    z = rng.standard_normal((B, V)).astype(np.float32)
    lse = np.log(np.exp(z.astype(np.float64)).sum(1)).astype(np.float32)
    scores = (8 + lse + 0.01 * np.arange(B)).astype(np.float32)
    masked = np.arange(B) % 2 == 0
    z[masked], lse[masked], scores[masked] = LOWEST, LOWEST, score
    check_select(ops, z, scores, lse, W)
    check_select(ops, z, -scores, lse, W)


@pytest.mark.parametrize("B,V,W", SIZES)
@pytest.mark.parametrize("seed", range(4))
def test_select_where_32_bits_overflow(ops, B, V, W, seed):
    """z - lse leaves the 32-bit range and the score brings the sum back, or the
    sum itself leaves it."""
    rng = np.random.default_rng(seed)
    ends = np.array([LOWEST, -LOWEST, 3e38, -3e38, 1e38, -1e38, 2e30, -1.0, 0.0, 7.0], np.float32)
    z = rng.choice(ends, (B, V))
    z[:, V // 2:] = rng.uniform(-3.4e38, 3.4e38, (B, V - V // 2))
    scores, lse = rng.choice(ends, B), rng.choice(ends, B)
    check_select(ops, z, scores, lse, W)
    lse[::3] = rng.choice([np.inf, -np.inf, np.nan], len(lse[::3]))
    scores[1::3] = rng.choice([np.inf, -np.inf, np.nan], len(scores[1::3]))
    z[rng.random((B, V)) < 0.01] = np.inf
    check_select(ops, z, scores, lse, W)
    check_select(ops, z, scores, lse, W, (np.arange(B) % 4 == 3).astype(np.int32), 1)


@pytest.mark.parametrize("B,V,W", SIZES)
def test_select_where_the_score_brings_the_sum_back(ops, B, V, W):
    z = np.full((B, V), 2.8e38, np.float32)
    lse, scores = np.zeros(B, np.float32), np.zeros(B, np.float32)
    z[0], lse[0], scores[0] = 3e38, -3e38, LOWEST     # 6e38 - 3.4e38 = 2.6e38
    check_select(ops, z, scores, lse, W)
    check_select(ops, -z, -scores, -lse, W)
