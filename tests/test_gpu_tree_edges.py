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


# --------------------------------------------------------------------------
# waits that run out


@pytest.fixture
def give_up(ops):
    """Makes the waits of one CTA give up at once, in this thread's calls."""
    from self_speculative_decoding_gb300 import _abi
    call = _abi.lib().ssd_debug_tree_give_up
    assert call(-2, -1) == 1 and call(-1, -2) == 1
    yield lambda attention=-1, weights=-1: call(attention, weights)
    call(-1, -1)


def tree_inputs(H, Hkv, dh, n, T, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + 7 * n + T)
    qkv = torch.randn(T, (H + 2 * Hkv) * dh, generator=g, device="cuda")
    parents = torch.tensor([-1] + [i - 1 - (5 * i) % min(i, 4) for i in range(1, T)], dtype=torch.int32).cuda()
    k, v = (torch.randn(Hkv, n + T + 3, dh, generator=g, device="cuda").bfloat16() for _ in range(2))
    return qkv, parents, k, v


def tree_call(ops, x, H, Hkv, dh, n, weights=True):
    w = torch.zeros(Hkv, x[2].shape[1], device="cuda") if weights else None
    return ops.tree_attention(*x, n, n, H, Hkv, dh, 1e4, weights_out=w), w


@pytest.mark.parametrize("H,Hkv,dh,n,T,cta,lost", [
    # (K/V head, its first lost row, the one behind its last) of one split:
    (40, 40, 128, 100, 9, 5, [(5, 0, 9)]),                  # a CTA for each head
    (200, 200, 64, 10, 2, 7, [(7, 0, 2), (159, 0, 2)]),     # 152 CTAs for 200
    (8, 4, 64, 60, 200, 3, [(1, 256, 400)]),                # two pairs of 128-row tiles a head
    (8, 4, 128, 60, 200, 2, [(1, 0, 256)])])
@pytest.mark.parametrize("weights", [False, True])
def test_a_wait_that_runs_out_marks_its_rows(ops, give_up, H, Hkv, dh, n, T, cta, lost, weights):
    x = tree_inputs(H, Hkv, dh, n, T)
    want, want_w = tree_call(ops, x, H, Hkv, dh, n, weights)
    assert torch.isfinite(want).all()
    give_up(attention=cta)
    out, w = tree_call(ops, x, H, Hkv, dh, n, weights)
    give_up()
    bad = torch.zeros(Hkv, T * (H // Hkv), dtype=torch.bool, device="cuda")
    for kvh, a, b in lost:
        bad[kvh, a:b] = True
    rows = out.view(T, Hkv, H // Hkv, dh).permute(1, 0, 2, 3).reshape(Hkv, -1, dh)
    want_rows = want.view(T, Hkv, H // Hkv, dh).permute(1, 0, 2, 3).reshape(Hkv, -1, dh)
    assert torch.isnan(rows[bad]).all() and torch.equal(rows[~bad], want_rows[~bad])
    if weights:
        assert torch.isnan(w[:, :n + T]).all() and not w[:, n + T:].any()
    out, w = tree_call(ops, x, H, Hkv, dh, n, weights)
    assert torch.equal(out, want) and (not weights or torch.equal(w, want_w))


@pytest.mark.parametrize("H,Hkv,dh,n,T", [(4, 1, 128, 9000, 5), (16, 2, 64, 5000, 30)])
def test_a_wait_that_runs_out_marks_what_is_joined(ops, give_up, H, Hkv, dh, n, T):
    x = tree_inputs(H, Hkv, dh, n, T)
    want, want_w = tree_call(ops, x, H, Hkv, dh, n)
    give_up(attention=4)
    out, w = tree_call(ops, x, H, Hkv, dh, n)
    give_up()
    assert torch.isnan(out).all() and torch.isnan(w[:, :n + T]).all()
    out, w = tree_call(ops, x, H, Hkv, dh, n)
    assert torch.equal(out, want) and torch.equal(w, want_w)


def test_a_wait_for_the_weights_that_runs_out_marks_its_keys(ops, give_up):
    H, Hkv, dh, n, T = 16, 2, 128, 1500, 40                 # 13 blocks of 128 keys a head, a CTA each
    x = tree_inputs(H, Hkv, dh, n, T)
    want, want_w = tree_call(ops, x, H, Hkv, dh, n)
    give_up(weights=16)
    out, w = tree_call(ops, x, H, Hkv, dh, n)
    bad = torch.zeros_like(w, dtype=torch.bool)
    bad[1, 3 * 128:4 * 128] = True
    assert torch.equal(out, want)
    assert torch.isnan(w[bad]).all() and torch.equal(w[~bad], want_w[~bad])


# --------------------------------------------------------------------------
# NaN and infinities


@pytest.mark.parametrize("T", [6, 10, 16, 40, 150])     # stored scores for few nodes, a second pass of products for more
@pytest.mark.parametrize("where", ["q", "k"])
def test_weights_of_keys_that_a_row_of_nan_does_not_see(ops, T, where):
    H, Hkv, dh, n = 4, 2, 64, 150
    x = tree_inputs(H, Hkv, dh, n, T)
    parents = [-1, 0, 0] + [i - 2 for i in range(3, T)]     # the odd nodes, and the even ones
    x[1].copy_(torch.tensor(parents, dtype=torch.int32))
    _, clean = tree_call(ops, x, H, Hkv, dh, n)
    row = x[0].view(T, H + 2 * Hkv, dh)[T - 1 - T % 2]      # the last odd node: no node follows it
    row[slice(H) if where == "q" else slice(H, H + Hkv), 3] = float("nan")
    _, w = tree_call(ops, x, H, Hkv, dh, n)
    even = [n + t for t in range(2, T, 2)]
    odd = [n + t for t in range(T) if t == 0 or t % 2]
    assert torch.isfinite(clean[:, :n + T]).all()
    assert torch.isnan(w[:, :n]).all() and torch.isnan(w[:, odd]).all()
    assert torch.equal(w[:, even], clean[:, even])


U = 2.0 ** -8      # half a bf16 step, relative


def seen_softmax(q, parents, n, K, V):
    """out [T, H, dh], the weights of each key, the sum of p |v| and the largest
    sum of |q k|, in 64 bits; K may hold infinities (q k summed term by term)."""
    (T, H, dh), (Hkv, S, _) = q.shape, K.shape
    G = H // Hkv
    seen = np.zeros((T, S), bool)
    seen[:, :n] = True
    for t, path in enumerate(O.tree_paths(parents)):
        seen[t, [n + i for i in path]] = True
    out, spread, size = np.zeros((T, H, dh)), np.zeros((T, H, dh)), np.zeros((T, H))
    mass = np.zeros((Hkv, S))
    with np.errstate(invalid="ignore"):
        for t in range(T):
            for h in range(H):
                terms = q[t, h] * K[h // G, seen[t]]
                s = terms.sum(1) / np.sqrt(dh)
                p = np.exp(s - s.max())
                p /= p.sum()
                out[t, h], spread[t, h] = p @ V[h // G, seen[t]], p @ np.abs(V[h // G, seen[t]])
                size[t, h] = np.where(np.isfinite(terms), np.abs(terms), 0).sum(1).max()
                mass[h // G, seen[t]] += p
    return out, mass, spread, size


# tolerances as in test_gpu_tree_ops.py: the output's rounding and the
# probabilities' u each, and 2 d for a score that is off by d
def check_seen(out, w, x, parents, pos0, n, H, Hkv, dh):
    T = len(parents)
    q, _, _ = O.tree_rows(x[0].double().cpu().numpy(), parents, pos0, H, Hkv, dh, 1e4)
    K, V = (t[:, :n + T].double().cpu().numpy() for t in x[2:])
    ref, mass, spread, size = seen_softmax(q, parents, n, K, V)
    d = (2.0 ** -16 + 2 * dh * 2.0 ** -24) * size / np.sqrt(dh) + 1e-6
    got = out.double().cpu().numpy().reshape(T, H, dh)
    nan = np.isnan(ref)
    np.testing.assert_array_equal(np.isnan(got), nan)
    err, tol = np.abs(got - ref), U * np.abs(ref) + (U + 2 * d[..., None]) * spread
    assert np.all(err[~nan] <= tol[~nan])
    got = w[:, :n + T].double().cpu().numpy()
    nan_w = np.isnan(mass)
    np.testing.assert_array_equal(np.isnan(got), nan_w)
    err, tol = np.abs(got - mass), (2 * d.max() + (T * (H // Hkv) + 2) * 2.0 ** -24) * mass + 1e-12
    assert np.all(err[~nan_w] <= tol[~nan_w])
    return nan


# stored scores and a second pass of products, one tile and two, one split and several
SHAPES = [(4, 2, 64, 150, 6), (4, 4, 128, 700, 30), (2, 1, 128, 300, 40), (4, 2, 64, 60, 150), (8, 2, 128, 5000, 12), (8, 2, 128, 5000, 4)]


@pytest.mark.parametrize("H,Hkv,dh,n,T", SHAPES)
@pytest.mark.parametrize("what", [float("inf"), float("-inf")])
def test_infinite_elements_of_k_that_are_seen(ops, H, Hkv, dh, n, T, what):
    """A score of -infinity is no weight, +infinity makes its row NaN."""
    x = tree_inputs(H, Hkv, dh, n, T)
    x[2][:, [3, n // 2, n - 1], dh // 3] = what
    out, w = tree_call(ops, x, H, Hkv, dh, n)
    nan = check_seen(out, w, x, x[1].tolist(), n, n, H, Hkv, dh)
    assert nan.any() and not nan.all()


@pytest.mark.parametrize("H,Hkv,dh,n,T", SHAPES)
def test_scores_of_minus_infinity_leave_the_rest_finite(ops, H, Hkv, dh, n, T):
    """Roots at position 0 (their projections are not turned), q positive in the
    column where some keys are -infinity, its low part zero in half of the rows."""
    x = tree_inputs(H, Hkv, dh, n, T)
    parents = [-1] * T
    x[1].fill_(-1)
    rows = x[0].view(T, H + 2 * Hkv, dh)
    rows[:, :H, 5] = rows[:, :H, 5].abs() + 0.1
    rows[::2, :H] = rows[::2, :H].bfloat16().float()
    x[2][:, 1:n:7, 5] = float("-inf")
    rows[1, H:H + Hkv, 5] = -3.4e38                   # rounded to -inf in the cache
    w = torch.zeros(Hkv, x[2].shape[1], device="cuda")
    out = ops.tree_attention(*x, n, 0, H, Hkv, dh, 1e4, weights_out=w)
    assert torch.isinf(x[2][:, n + 1, 5]).all()
    nan = check_seen(out, w, x, parents, 0, n, H, Hkv, dh)
    assert not nan.any() and not w[:, 1:n:7].any() and not w[:, n + 1].any()


def test_nan_in_k_stays(ops):
    H, Hkv, dh, n, T = 4, 2, 128, 900, 40
    x = tree_inputs(H, Hkv, dh, n, T)
    x[2][0, 500, 7] = float("nan")
    x[2][0, 600, 9] = float("-inf")
    out, w = tree_call(ops, x, H, Hkv, dh, n)
    out = out.view(T, H, dh)
    assert torch.isnan(out[:, :2]).all() and torch.isfinite(out[:, 2:]).all()
    assert torch.isnan(w[0, :n + T]).all() and torch.isfinite(w[1]).all()


# --------------------------------------------------------------------------
# refusals


def test_rows_that_a_cache_does_not_have_allocate_nothing(ops):
    from self_speculative_decoding_gb300 import SSDError
    H, Hkv, dh = 64, 8, 128
    x = tree_inputs(H, Hkv, dh, 60, 1)
    S = x[2].shape[1]
    w = torch.zeros(Hkv, S, device="cuda")
    k2, v2 = x[2][:, :20].clone(), x[3][:, :20].clone()
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    now = torch.cuda.max_memory_allocated()
    for n in (S, 10 ** 7, 2 ** 31 - 1, -1):
        with pytest.raises(SSDError):
            ops.tree_attention(*x, n, 60, H, Hkv, dh, 1e4)
    for n, keep in ((10 ** 8, 10 ** 8), (10 ** 8, 20), (S, 21), (2 ** 31 - 1, 2 ** 31 - 1)):
        with pytest.raises(SSDError):
            ops.cache_evict(x[2], x[3], w, n, keep, k2, v2)
    assert torch.cuda.max_memory_allocated() - now < 1 << 16


# --------------------------------------------------------------------------
# the largest sizes


def test_select_over_the_largest_vocabulary(ops):
    V = 2 ** 31 - 1
    z = torch.full((1, V), -3.0, device="cuda")
    at = [V - 1, 5, V // 2, 22528, V - 22528]
    for i, v in enumerate(at):
        z[0, v] = 10.0 - i
    tok, par, best, done = ops.beam_select(z, torch.tensor([-1.0], device="cuda"), 8, end_id=V - 1)
    assert tok.tolist() == at + [0, 1, 2] and par.tolist() == [0] * 8
    assert best.tolist() == [9.0, 8.0, 7.0, 6.0, 5.0, -4.0, -4.0, -4.0] and done.tolist() == [1] + [0] * 7


@pytest.mark.parametrize("T", [1, 40])              # stored scores, and a second pass of products
def test_rows_far_along_a_cache_are_the_right_ones(ops, T):
    """1.2 million rows of 8 heads, the last head's beyond 2^31 elements: in each
    head one key outweighs the rest, and every key's weight is checked."""
    H = Hkv = 8
    dh, n, S = 128, 1_200_000, 2_400_000
    g = torch.Generator(device="cuda").manual_seed(T)
    qkv = torch.randn(1, 3 * H * dh, generator=g, device="cuda").repeat(T, 1)
    parents = torch.full((T,), -1, dtype=torch.int32, device="cuda")   # roots at 0: nothing is turned
    k = torch.zeros(Hkv, S, dh, dtype=torch.bfloat16, device="cuda")
    v = torch.empty(Hkv, S, dh, dtype=torch.bfloat16, device="cuda")
    v.copy_(torch.arange(1, Hkv + 1, device="cuda")[:, None, None].expand(v.shape))
    q, own_k, own_v = (x.double() for x in qkv[0].view(3, H, dh))
    own = (q * own_k.bfloat16().double()).sum(1) / dh ** 0.5
    heads = torch.arange(H, device="cuda")
    for rows in (None, [n - 1] * H, [0, 1, 127, 2 ** 20, 2 ** 20 + 1, n - 2, n - 128, 777_777]):
        k[:, :n] = 0
        score = torch.zeros(H, n, dtype=torch.float64, device="cuda")
        if rows is not None:
            at = torch.tensor(rows, device="cuda")
            k[heads, at] = (3 * q).bfloat16()
            v[heads, at] = (100.0 + heads)[:, None].bfloat16()
            score[heads, at] = (q * k[heads, at].double()).sum(1) / dh ** 0.5
        w = torch.zeros(Hkv, S, device="cuda")
        out = ops.tree_attention(qkv, parents, k, v, n, 0, H, Hkv, dh, 1e4, weights_out=w).double().view(T, H, dh)
        p = torch.softmax(torch.cat((score, own[:, None]), 1), 1)
        ref = torch.einsum("hn,hnd->hd", p[:, :n], v[:, :n, :1].double()) + p[:, n:] * own_v.bfloat16().double()
        spread = torch.einsum("hn,hnd->hd", p[:, :n], v[:, :n, :1].double()) + p[:, n:] * own_v.abs()
        # scores up to 3 |q|^2 / sqrt(dh), off by 2^-16 of that and the fp32 sums
        d = (2.0 ** -16 + 2 * dh * 2.0 ** -24) * 3.1 * (q * q).sum(1).max().item() / dh ** 0.5 + 1e-6
        assert ((out - ref).abs() <= U * ref.abs() + (U + 2 * d) * spread).all()
        mass = T * p[:, :n]
        assert ((w[:, :n].double() - mass).abs() <= (2 * d + (T + 2) * 2.0 ** -24) * mass + 1e-30).all()
        assert ((w[:, n:n + T].double() - p[:, n:]).abs() <= 3 * d * p[:, n:] + 1e-30).all() and not w[:, n + T:].any()
        if rows is not None:
            assert (out[0] - (100.0 + heads)[:, None]).abs().max().item() < 0.5 and (w[heads, at] > 0.99 * T).all()
            v[heads, at] = (1.0 + heads)[:, None].bfloat16()


# --------------------------------------------------------------------------
# calls in other forms


def test_a_given_output_is_written_and_returned(ops):
    from self_speculative_decoding_gb300 import SSDError
    H, Hkv, dh, n, T = 8, 2, 64, 400, 9
    x = tree_inputs(H, Hkv, dh, n, T)
    want, _ = tree_call(ops, x, H, Hkv, dh, n, False)
    out = torch.full((T, H * dh), 7.0, device="cuda").bfloat16()
    assert ops.tree_attention(*x, n, n, H, Hkv, dh, 1e4, out=out).data_ptr() == out.data_ptr()
    assert torch.equal(out, want)
    with pytest.raises(SSDError):
        ops.tree_attention(*x, n + 4, n, H, Hkv, dh, 1e4, out=out.fill_(7.0))
    for bad in (out.float(), out[:, :-8].contiguous(), out.t(), out.cpu()):
        with pytest.raises(ValueError, match="out"):
            ops.tree_attention(*x, n, n, H, Hkv, dh, 1e4, out=bad)
    w = torch.zeros(Hkv, x[2].shape[1], device="cuda")
    with pytest.raises(SSDError):
        ops.tree_attention(*x, n, n, H, Hkv, dh, 1e4, weights=w, out=out)
    assert (out == 7).all()


@pytest.mark.parametrize("H,Hkv,dh,n,T", [(8, 2, 64, 700, 4), (8, 2, 128, 700, 20), (16, 2, 128, 3000, 40)])
def test_a_replayed_graph_takes_new_trees(ops, H, Hkv, dh, n, T):
    """Other nodes, parents (absent ones among them) and weights of one captured call."""
    x, y = (tree_inputs(H, Hkv, dh, n, T, seed) for seed in (0, 1))
    y[1].copy_(torch.tensor([-1] + [(3 * i) % i if i % 5 else -2 for i in range(1, T)], dtype=torch.int32))
    w = torch.rand(Hkv, n + T + 3, device="cuda")
    held, held_w = [t.clone() for t in x], w.clone()
    ops.tree_attention(*held, n, n, H, Hkv, dh, 1e4, weights=held_w, weights_out=held_w)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = ops.tree_attention(*held, n, n, H, Hkv, dh, 1e4, weights=held_w, weights_out=held_w)
    for inputs in (x, y, x):
        for a, b in zip(held, inputs):
            a.copy_(b)
        held_w.copy_(w)
        graph.replay()
        mine, mine_w = [t.clone() for t in inputs], w.clone()
        want = ops.tree_attention(*mine, n, n, H, Hkv, dh, 1e4, weights=mine_w, weights_out=mine_w)
        assert torch.equal(out, want) and torch.equal(held_w, mine_w)
        assert all(torch.equal(a, b) for a, b in zip(held, mine))
