"""Tree decoding on the GPU: attention of a tree of drafts over a cache,
eviction by accumulated weight, beam selection and beam reordering, against
the fp64 references of oracle/ops.py.

Tolerances of the tree attention, from the roundings that the call documents
(u = 2^-8, half a bf16 step relative to the value):
* cached K row: the rotation's angle is exact to 2^-24 of half a turn and the
  products to a few 2^-24, so |x| + |y| of the pair times 1e-6, then u |k|;
* out: the output's own rounding u |o|, and the probabilities' u p_j each:
  u sum_j p_j |v_j|.  q = hi + lo to 2^-16 |q_i|, so a score is off by
  d = (2^-16 + 2 dh 2^-24) sum_i |q_i k_i| / sqrt(dh) + 1e-6 at most and a
  probability by the factor e^(2 d): 2 d sum_j p_j |v_j|.  The reference reads
  the K/V rows that the call stored, so their rounding is no error here.
* weights: the factor e^(2 d) on each probability, and the sum's own rounding.
"""

import numpy as np
import pytest
import torch

from oracle import ops as O

pytestmark = pytest.mark.gpu

U = 2.0 ** -8


@pytest.fixture(scope="module")
def ops():
    import __graft_entry__ as g
    g.build()
    import self_speculative_decoding_gb300 as ssd
    return ssd.ops


def make_tree(kind, T, rng):
    if kind == "chain":
        return list(range(-1, T - 1))
    if kind == "roots":
        return [-1] * T
    if kind == "none":
        return [-2] * T
    if kind == "broken":  # a chain with an end that is none
        return [i - 1 if i != T // 3 else T for i in range(T)]
    if kind == "comb":  # a long spine, each node with a leaf
        return [i - 1 if i % 2 else max(i - 2, -1) for i in range(T)]
    if kind == "bad":  # values out of range, self-loops, forward edges
        p = [-1] + [int(rng.integers(0, i)) for i in range(1, T)]
        for i, bad in ((1, 1), (2, 5000), (T // 2, T // 2 + 1), (T - 1, -7), (T // 3, 2 ** 31 - 1)):
            p[i] = bad
        return p
    wide = {"tree": 4, "bushy": 64}.get(kind.split("-")[0], 4)
    p = [-1] + [i - 1 - int(rng.integers(0, min(i, wide))) for i in range(1, T)]
    if kind.endswith("-padded"):
        live = max(1, T - max(1, T // 4))
        p[live:] = [-2] * (T - live)
    return p


class Case:
    """Seeded inputs of one tree attention call, rows behind it marked."""

    def __init__(self, H, Hkv, dh, n, T, kind="tree", spare=7, pos0=None, seed=0, std=1.0):
        rng = np.random.default_rng(seed + 7 * n + T)
        self.H, self.Hkv, self.dh, self.n, self.T = H, Hkv, dh, n, T
        self.pos0 = n if pos0 is None else pos0
        self.S = n + T + spare
        self.parents = make_tree(kind, T, rng)
        f = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32))  # noqa: E731
        self.qkv = (f(T, (H + 2 * Hkv) * dh) * std).cuda()
        self.k0, self.v0 = f(Hkv, self.S, dh).bfloat16().cuda(), f(Hkv, self.S, dh).bfloat16().cuda()
        # rows behind the tree: never read
        self.k0[:, n + T:] = float("nan")
        self.v0[:, n + T:] = float("inf")
        self.par = torch.tensor(self.parents, dtype=torch.int32).cuda()
        self.w0 = torch.from_numpy(rng.exponential(size=(Hkv, self.S)).astype(np.float32)).cuda()

    def call(self, ops, weights=True, **kw):
        self.k, self.v = self.k0.clone(), self.v0.clone()
        self.w = torch.full_like(self.w0, -3.0) if weights else None
        return ops.tree_attention(self.qkv, self.par, self.k, self.v, self.n, self.pos0, self.H,
                                  self.Hkv, self.dh, 1e4, weights=self.w0 if weights else None,
                                  weights_out=self.w, **kw)

    def check(self, out):
        H, Hkv, dh, n, T = self.H, self.Hkv, self.dh, self.n, self.T
        qkv = self.qkv.double().cpu().numpy()
        q, k, v = O.tree_rows(qkv, self.parents, self.pos0, H, Hkv, dh, 1e4)
        K, V = self.k.double().cpu().numpy(), self.v.double().cpu().numpy()
        bits = lambda t: t.view(torch.int16)  # noqa: E731
        for now, was in ((self.k, self.k0), (self.v, self.v0)):
            assert torch.equal(bits(now[:, :n]), bits(was[:, :n]))
            assert torch.equal(bits(now[:, n + T:]), bits(was[:, n + T:]))
        x = np.abs(qkv.reshape(T, H + 2 * Hkv, dh)[:, H:H + Hkv])
        pair = np.concatenate((x[..., :dh // 2] + x[..., dh // 2:],) * 2, -1)
        assert np.all(np.abs(K[:, n:n + T].transpose(1, 0, 2) - k) <= U * np.abs(k) + 1e-6 * pair)
        vt = torch.from_numpy(v).float().bfloat16().double().numpy()
        np.testing.assert_array_equal(V[:, n:n + T].transpose(1, 0, 2), vt)
        ref, mass, spread = O.tree_attention(q, self.parents, n, K, V)
        G = H // Hkv
        size = np.array([[np.max(np.abs(q[t, h]) @ np.abs(K[h // G, :n + T]).T) for h in range(H)]
                         for t in range(T)])
        d = (2.0 ** -16 + 2 * dh * 2.0 ** -24) * size / np.sqrt(dh) + 1e-6
        got = out.double().cpu().numpy().reshape(T, H, dh)
        tol = U * np.abs(ref) + (U + 2 * d[..., None]) * spread + 1e-30
        assert np.all(np.abs(got - ref) <= tol), np.max(np.abs(got - ref) / tol)
        if self.w is not None:
            w, w0 = self.w.double().cpu().numpy(), self.w0.double().cpu().numpy()
            want = mass.copy()
            want[:, :n] += w0[:, :n]
            tol = 2 * d.max() * mass + (T * G + 2) * 2.0 ** -24 * want + 1e-12
            assert np.all(np.abs(w[:, :n + T] - want) <= tol), np.max(np.abs(w[:, :n + T] - want) / tol)
            assert np.all(w[:, n + T:] == -3.0)


HEADS = [(4, 4, 64), (8, 2, 64), (6, 2, 128), (8, 1, 128), (3, 3, 128)]


@pytest.mark.parametrize("H,Hkv,dh", HEADS)
@pytest.mark.parametrize("n,T,kind", [
    (0, 1, "tree"), (1, 1, "tree"), (0, 5, "tree"), (63, 2, "chain"), (127, 1, "tree"),
    (128, 3, "roots"), (129, 17, "tree"), (300, 33, "tree-padded"), (5, 64, "none"),
    (1000, 16, "chain"), (640, 100, "bushy"), (257, 20, "bad")])
def test_tree_attention(ops, H, Hkv, dh, n, T, kind):
    c = Case(H, Hkv, dh, n, T, kind)
    c.check(c.call(ops))


@pytest.mark.parametrize("H,Hkv,dh,n,T,kind", [
    (2, 2, 128, 200, 127, "tree"), (2, 2, 128, 200, 128, "tree"), (2, 2, 64, 200, 129, "bushy"),
    (4, 2, 128, 70, 255, "tree-padded"), (2, 1, 64, 0, 513, "tree"), (2, 1, 128, 300, 1024, "chain"),
    (16, 1, 128, 1500, 40, "tree"), (1, 1, 64, 4100, 9, "tree"), (40, 40, 128, 700, 3, "tree"),
    (64, 8, 128, 2500, 1, "tree"), (33, 11, 64, 129, 2, "chain"), (2, 1, 64, 90, 34, "chain"),
    (2, 1, 64, 90, 300, "broken"), (2, 2, 64, 140, 701, "comb"), (1, 1, 128, 3, 1024, "broken")])
def test_tree_attention_sizes(ops, H, Hkv, dh, n, T, kind):
    c = Case(H, Hkv, dh, n, T, kind, spare=0)
    c.check(c.call(ops))


def test_large_scores_and_far_positions(ops):
    # one key takes nearly all, then the maximum moves late in the cache
    c = Case(4, 2, 128, 900, 9, std=8.0, pos0=1_000_000)
    c.k0[:, 700] *= 12.0
    c.k0[:, 850] *= 30.0
    c.check(c.call(ops))


def test_weights_in_place_and_without(ops):
    c = Case(8, 2, 128, 333, 21)
    a = c.call(ops)
    w = c.w0.clone()
    b = ops.tree_attention(c.qkv, c.par, c.k, c.v, c.n, c.pos0, 8, 2, 128, 1e4, weights=w, weights_out=w)
    n = c.n + c.T
    assert torch.equal(a, b) and torch.equal(w[:, :n], c.w[:, :n])
    assert torch.equal(w[:, n:], c.w0[:, n:])
    assert torch.equal(c.call(ops, weights=False), a)
    z = torch.zeros_like(w)
    ops.tree_attention(c.qkv, c.par, c.k, c.v, c.n, c.pos0, 8, 2, 128, 1e4, weights_out=z)
    mass = (c.w0 * 0).double()
    ref = O.tree_attention(*[x for x in (O.tree_rows(c.qkv.double().cpu().numpy(), c.parents, c.pos0, 8, 2, 128, 1e4)[0],)],
                           c.parents, c.n, c.k.double().cpu().numpy(), c.v.double().cpu().numpy())[1]
    mass[:, :n] = torch.from_numpy(ref).cuda()
    assert (z.double() - mass).abs().max().item() <= 1e-3 * ref.max()


@pytest.mark.parametrize("what", [float("inf"), float("-inf"), float("nan")])
def test_masked_rows_may_hold_anything(ops, what):
    # the left half of the tree holds inf or NaN in its projections; the right
    # half sees none of it and gets the bits that it gets without
    H, Hkv, dh, n, T = 4, 2, 128, 150, 40
    c = Case(H, Hkv, dh, n, T)
    c.parents = [-1, 0, 0] + [i - 2 for i in range(3, T)]
    c.par = torch.tensor(c.parents, dtype=torch.int32).cuda()
    clean = c.call(ops)
    w = c.w.clone()
    x = c.qkv.view(T, H + 2 * Hkv, dh)
    x[5, H + Hkv:, 3] = what           # V of node 5
    x[7, H:H + Hkv, 9] = what          # K of node 7
    x[9, :H, 1] = what                 # q of node 9
    out = c.call(ops)
    paths = O.tree_paths(c.parents)
    apart = [t for t in range(T) if not {5, 7, 9} & set(paths[t])]
    assert len(apart) > T // 2 - 3
    assert torch.equal(out[apart], clean[apart])
    assert not torch.isfinite(out[5].view(H, dh)[:, 3]).any()
    cols = [i for i in range(dh) if i != 3]
    assert torch.equal(out[5].view(H, dh)[:, cols], clean[5].view(H, dh)[:, cols])
    # node 9's query meets 150 keys of either sign: +inf or NaN among its scores,
    # so NaN all over.  Node 7's key gives its own row one score per head, NaN
    # or +inf (NaN all over that head) or -inf (no weight: the head stays finite)
    assert torch.isnan(out[9]).all()
    nans = torch.isnan(out[7].view(H, dh))
    assert (nans.all(1) | ~nans.any(1)).all() and (nans.all() or what == what)
    # a descendant's own inf or NaN reaches it through V, K or both
    below5 = [t for t in range(6, T) if 5 in paths[t] and 7 not in paths[t]]
    for t in below5:
        assert not torch.isfinite(out[t].view(H, dh)[:, 3]).any()
    # weights: the right half's keys (even nodes), which no marked row sees
    same = [n + t for t in range(2, T, 2)]
    assert torch.equal(c.w[:, same], w[:, same])


def test_non_finite_context_is_seen_by_all(ops):
    c = Case(4, 2, 64, 100, 6)
    c.v0[:, 37, 5] = float("nan")
    out = c.call(ops).view(6, 4, 64)
    assert torch.isnan(out[:, :, 5]).all() and torch.isfinite(out[:, :, :5]).all()


def test_calls_repeat_their_bits_and_ignore_the_workspace(ops):
    import self_speculative_decoding_gb300 as ssd
    from self_speculative_decoding_gb300 import _abi
    lib = _abi.lib()
    c = Case(8, 2, 128, 777, 50)
    a, w = c.call(ops), c.w.clone()
    need = lib.ssd_op_tree_attention_workspace(c.T, c.n, 8, 2, 128)
    for fill in (0, 0xFF):
        ws = torch.full((need + 256,), fill, dtype=torch.uint8, device="cuda")
        out = torch.empty_like(a)
        k, v, w2 = c.k0.clone(), c.v0.clone(), torch.full_like(w, -3.0)
        st = lib.ssd_op_tree_attention(c.qkv.data_ptr(), c.par.data_ptr(), c.T, c.n, c.pos0,
                                       k.data_ptr(), v.data_ptr(), c.S, 8, 2, 128, 1e4,
                                       c.w0.data_ptr(), w2.data_ptr(), out.data_ptr(),
                                       ws.data_ptr(), need, ssd.stream_handle())
        assert st == 0
        assert torch.equal(out, a) and torch.equal(w2, w)
        assert bool((ws[need:] == fill).all())


def test_offsets_beyond_32_bits(ops):
    # the last head's rows start beyond 2^31 elements
    H, Hkv, dh, n, T = 8, 8, 128, 70, 3
    S = 2_400_000
    c = Case(H, Hkv, dh, n, T)
    k = torch.empty(Hkv, S, dh, dtype=torch.bfloat16, device="cuda")
    v = torch.empty(Hkv, S, dh, dtype=torch.bfloat16, device="cuda")
    k[:, :n], v[:, :n] = c.k0[:, :n], c.v0[:, :n]
    out = ops.tree_attention(c.qkv, c.par, k, v, n, c.pos0, H, Hkv, dh, 1e4)
    assert torch.equal(out, c.call(ops, weights=False))
    assert torch.equal(k[:, n:n + T], c.k[:, n:n + T]) and torch.equal(v[:, n:n + T], c.v[:, n:n + T])
    # and rows far along one head's cache
    big_n = 1_200_000
    k[:, :big_n] = 0
    v[:, :big_n] = 1
    out = ops.tree_attention(c.qkv, c.par, k, v, big_n, big_n, H, Hkv, dh, 1e4)
    assert torch.isfinite(out).all()
    # zero keys: every row of the context weighs e^0, the tree's rows next to nothing
    assert (out.float() - 1).abs().max().item() < 0.02


@pytest.mark.parametrize("H,Hkv,dh,n,T", [(8, 1, 64, 700_001, 70), (16, 2, 128, 300_000, 40),
                                          (4, 4, 128, 60_000, 7)])
def test_long_contexts(ops, H, Hkv, dh, n, T):
    # long enough that a CTA has several runs of keys and passes over them;
    # the reference is the same formula as torch operations in 64 bits
    g = torch.Generator(device="cuda").manual_seed(n)
    G, S = H // Hkv, n + T
    parents = [-1] + [i - 1 - (5 * i) % min(i, 4) for i in range(1, T)]
    qkv = torch.randn(T, (H + 2 * Hkv) * dh, generator=g, device="cuda")
    k = torch.randn(Hkv, S, dh, generator=g, device="cuda").bfloat16()
    v = torch.randn(Hkv, S, dh, generator=g, device="cuda").bfloat16()
    w = torch.zeros(Hkv, S, device="cuda")
    out = ops.tree_attention(qkv, torch.tensor(parents, dtype=torch.int32).cuda(), k, v, n, n, H,
                             Hkv, dh, 1e4, weights_out=w).double().view(T, H, dh)
    q, _, _ = O.tree_rows(qkv.double().cpu().numpy(), parents, n, H, Hkv, dh, 1e4)
    q = torch.from_numpy(q).cuda()
    seen = torch.ones(T, S, dtype=torch.bool, device="cuda")
    for t, path in enumerate(O.tree_paths(parents)):
        seen[t, n:] = False
        seen[t, [n + i for i in path]] = True
    for kvh in range(Hkv):
        rows = q[:, kvh * G:(kvh + 1) * G].reshape(T * G, dh)
        K, V = k[kvh].double(), v[kvh].double()
        size = (rows.abs() @ K.abs().T).amax().item()
        d = (2.0 ** -16 + 2 * dh * 2.0 ** -24) * size / np.sqrt(dh) + 1e-6
        s = (rows @ K.T / np.sqrt(dh)).masked_fill_(~seen.repeat_interleave(G, 0), float("-inf"))
        p = torch.softmax(s, dim=1)
        ref = (p @ V).view(T, G, dh)
        spread = (p @ V.abs()).view(T, G, dh)
        err = (out[:, kvh * G:(kvh + 1) * G] - ref).abs()
        assert (err <= U * ref.abs() + (U + 2 * d) * spread).all()
        mass = p.sum(0)
        err = (w[kvh].double() - mass).abs()
        assert (err <= 2 * d * mass + (T * G + 2) * 2.0 ** -24 * mass + 1e-12).all()


def test_graphs_and_streams(ops):
    c, d = Case(8, 2, 128, 500, 30), Case(8, 2, 128, 900, 12, seed=3)
    want_c, want_d = c.call(ops), d.call(ops)
    wc, wd = c.w.clone(), d.w.clone()
    side, outs, graphs = torch.cuda.Stream(), [], []
    for x in (c, d):
        x.k, x.v, x.w = x.k0.clone(), x.v0.clone(), torch.full_like(x.w0, -3.0)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            outs.append(ops.tree_attention(x.qkv, x.par, x.k, x.v, x.n, x.pos0, 8, 2, 128, 1e4,
                                           weights=x.w0, weights_out=x.w))
        graphs.append(g)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(s1):
            graphs[0].replay()
        with torch.cuda.stream(s2):
            graphs[1].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want_c) and torch.equal(outs[1], want_d)
        assert torch.equal(c.w, wc) and torch.equal(d.w, wd)


# --------------------------------------------------------------------------
# eviction


def run_evict(ops, w, n, keep, sinks, recent, dh=64, dtype=torch.bfloat16, spare=3):
    Hkv, S = w.shape
    g = torch.Generator(device="cuda").manual_seed(n)
    k = torch.randn(Hkv, S, dh, generator=g, device="cuda").to(dtype)
    v = torch.randn(Hkv, S, dh, generator=g, device="cuda").to(dtype)
    ko = torch.full((Hkv, keep + spare, dh), 7.0, dtype=dtype, device="cuda")
    vo, wo = ko.clone(), torch.full((Hkv, keep + spare), 7.0, device="cuda")
    kept = ops.cache_evict(k, v, w, n, keep, ko, vo, wo, sinks=sinks, recent=recent)
    idx = kept.long()
    rows = idx[:, :, None].expand(Hkv, keep, dh)
    assert torch.equal(ko[:, :keep], k.gather(1, rows)) and torch.equal(vo[:, :keep], v.gather(1, rows))
    assert torch.equal(wo[:, :keep].view(torch.int32), w.gather(1, idx).view(torch.int32))
    assert (ko[:, keep:] == 7).all() and (vo[:, keep:] == 7).all() and (wo[:, keep:] == 7).all()
    return kept.cpu().numpy()


@pytest.mark.parametrize("Hkv,n,keep,sinks,recent", [
    (2, 1, 1, 0, 0), (2, 1, 1, 1, 0), (3, 2, 1, 0, 0), (2, 33, 32, 0, 0), (4, 121, 64, 4, 16),
    (2, 1024, 1024, 0, 0), (2, 1025, 1, 0, 0), (2, 1500, 700, 700, 0), (2, 1500, 700, 0, 700),
    (1, 1500, 700, 300, 400), (5, 4095, 2048, 4, 256), (2, 20000, 777, 3, 100), (8, 70001, 9000, 4, 64)])
@pytest.mark.parametrize("dtype,dh", [(torch.bfloat16, 128), (torch.float32, 4), (torch.bfloat16, 8)])
def test_evict(ops, Hkv, n, keep, sinks, recent, dtype, dh):
    rng = np.random.default_rng(n)
    w = torch.from_numpy(rng.exponential(size=(Hkv, n + 5)).astype(np.float32) ** 3)
    w[:, n:] = 1e9
    got = run_evict(ops, w.cuda(), n, keep, sinks, recent, dh, dtype)
    np.testing.assert_array_equal(got, O.cache_evict(w.numpy(), n, keep, sinks, recent))


def test_evict_ties_and_specials(ops):
    rng = np.random.default_rng(4)
    n = 5000
    w = np.zeros((6, n), np.float32)
    w[1] = rng.integers(0, 3, n)
    w[2] = np.where(rng.random(n) < 0.5, -0.0, 0.0)
    w[3] = rng.choice([np.nan, np.inf, -np.inf, 0.0, 1e-42, -1.0], n)
    w[4] = rng.standard_normal(n) * 1e-40
    w[5] = np.nan
    for keep in (1, 100, 2500, 4999, 5000):
        got = run_evict(ops, torch.from_numpy(w).cuda(), n, keep, 0, min(keep, 7))
        np.testing.assert_array_equal(got, O.cache_evict(w, n, keep, 0, min(keep, 7)))


# weights a few steps of fp32 apart: few, some or many rows share all but their
# last ten bits
@pytest.mark.parametrize("n", [700, 6000, 8999, 20000, 150001])
@pytest.mark.parametrize("steps", [2 ** 21, 2 ** 18, 2 ** 15, 2 ** 11])
def test_evict_weights_that_differ_late(ops, n, steps):
    rng = np.random.default_rng(n)
    w = (1 + rng.integers(0, steps, (3, n)) * 2.0 ** -23).astype(np.float32)
    for keep in (n // 3, n - 40):
        got = run_evict(ops, torch.from_numpy(w).cuda(), n, keep, 3, 20, 8)
        np.testing.assert_array_equal(got, O.cache_evict(w, n, keep, 3, 20))


# as many clusters of one to eight CTAs as these heads get
@pytest.mark.parametrize("Hkv,n,keep", [(160, 20000, 3000), (80, 5000, 700), (100, 17000, 16000), (30, 4200, 4000)])
def test_evict_many_heads(ops, Hkv, n, keep):
    w = torch.rand(Hkv, n, generator=torch.Generator(device="cuda").manual_seed(n), device="cuda") ** 4
    got = run_evict(ops, w, n, keep, 2, 30, 8)
    middle = torch.sort(w[:, 2:n - 30], dim=1, descending=True, stable=True).indices[:, :keep - 32] + 2
    first, last = torch.arange(2).expand(Hkv, 2), torch.arange(n - 30, n).expand(Hkv, 30)
    want = torch.cat([first, torch.sort(middle, dim=1).values.cpu(), last], 1)
    np.testing.assert_array_equal(got, want.numpy())


def test_evict_long_row(ops):
    rng = np.random.default_rng(5)
    n, keep = 1_000_003, 100_000
    w = rng.exponential(size=(2, n)).astype(np.float32)
    w[1] = np.round(w[1] * 4)                 # thousands of ties at the cut
    got = run_evict(ops, torch.from_numpy(w).cuda(), n, keep, 4, 1000, dh=8)
    for h in range(2):
        mid = np.arange(4, n - 1000)
        order = np.lexsort((mid, -w[h, mid]))[:keep - 1004]
        want = np.concatenate((np.arange(4), np.sort(mid[order]), np.arange(n - 1000, n)))
        np.testing.assert_array_equal(got[h], want)


# --------------------------------------------------------------------------
# beam selection


def check_select(ops, z, scores, W, lse=None, done=None, end_id=-1):
    B = z.shape[0]
    t = lambda a, dt: None if a is None else torch.from_numpy(np.asarray(a, dt)).cuda()  # noqa: E731
    got = ops.beam_select(t(z, np.float32), t(scores, np.float32), W, lse=t(lse, np.float32),
                          done=t(done, np.int32), end_id=end_id)
    want = O.beam_select(z, np.zeros(B) if lse is None else lse, scores, done, end_id, W)
    tok, par, sc, dn = (x.cpu().numpy() for x in got)
    assert tok.tolist() == [w[0] for w in want]
    assert par.tolist() == [w[1] for w in want]
    np.testing.assert_array_equal(sc, np.array([w[2] for w in want], dtype=np.float64).astype(np.float32))
    assert dn.tolist() == [w[3] for w in want]


@pytest.mark.parametrize("B,V,W", [(1, 1, 1), (1, 5, 9), (3, 2, 4), (4, 1024, 4), (2, 4096, 16),
                                   (2, 4097, 256), (7, 32000, 7), (16, 50001, 48), (256, 300, 256),
                                   (1, 131075, 64), (48, 9999, 1)])
@pytest.mark.parametrize("ended", [False, True])
def test_select(ops, B, V, W, ended):
    rng = np.random.default_rng(B * V)
    z = (rng.standard_normal((B, V)) * 2).astype(np.float32)
    lse = np.log(np.exp(z.astype(np.float64)).sum(1)).astype(np.float32)
    done = (rng.random(B) < 0.4).astype(np.int32) if ended else None
    check_select(ops, z, (-rng.exponential(size=B)).astype(np.float32), W, lse, done, V - 1 if ended else -1)


@pytest.mark.parametrize("B,V,W", [(128, 5000, 128), (200, 1500, 256), (64, 9000, 64), (3, 30000, 200),
                                   (16, 2500, 256), (2, 900, 256)])
@pytest.mark.parametrize("kind", ["spread", "first", "offset", "one"])
def test_select_uneven_beams(ops, B, V, W, kind):
    """A few beams hold most of the best: spread scores, a first step (one beam
    far above the others, or alone), scores far from zero."""
    rng = np.random.default_rng(B + W)
    z = rng.standard_normal((B, V)).astype(np.float32) * 2
    scores = {"spread": -3 * rng.random(B), "first": np.where(np.arange(B) == B // 2, 0, -1e9),
              "offset": -1000 - rng.random(B) * 1e-3, "one": np.where(np.arange(B) == 0, 0, -np.inf)}[kind]
    check_select(ops, z, scores.astype(np.float32), W)


@pytest.mark.parametrize("B,V,W", [(2, 1500, 7), (5, 30000, 48), (60, 5000, 60), (150, 4500, 256), (3, 25000, 130)])
@pytest.mark.parametrize("kind", ["lowest", "equal", "coarse", "zeros", "infinite"])
def test_select_with_few_different_logits(ops, B, V, W, kind):
    """A vocabulary masked by the type's lowest value, equal logits: more
    candidates share a score than are ranked at once."""
    rng = np.random.default_rng(V + W)
    z = {"lowest": np.full((B, V), np.finfo(np.float32).min), "equal": np.full((B, V), -2.5),
         "coarse": rng.integers(0, 3, (B, V)) * 0.5, "zeros": np.where(rng.random((B, V)) < 0.5, 0.0, -0.0),
         "infinite": np.where(rng.random((B, V)) < 0.001, 1.0, -np.inf)}[kind].astype(np.float32)
    if kind == "lowest":
        z[:, rng.integers(0, V, 3)] = 1.5
        z[0, V - 1] = 2.0
    check_select(ops, z, np.where(np.arange(B) % 3 == 1, -1.0, 0.0).astype(np.float32), W)


def test_select_equal_logits_of_many_beams(ops):
    B, V, W = 256, 100000, 200                     # more lists than a block has threads
    z = torch.zeros(B, V, device="cuda")
    z[200, 5] = 1.0
    sc = -(torch.arange(B, device="cuda") % 7).float()
    tok, par, best, _ = ops.beam_select(z, sc - torch.where(torch.arange(B, device="cuda") == 0, 0.5, 0.0), W)
    # beam 7 is the first of those at 0; beam 200 is at -4, its token 5 at -3
    assert tok.tolist() == list(range(W)) and par.tolist() == [7] * W and (best == 0).all()
    z[7, 100:] = -9.0                              # a hundred of beam 7, then of beam 14
    tok, par, best, _ = ops.beam_select(z, sc - torch.where(torch.arange(B, device="cuda") == 0, 0.5, 0.0), W)
    assert tok.tolist() == list(range(100)) * 2 and par.tolist() == [7] * 100 + [14] * 100 and (best == 0).all()


def test_select_ties_specials_and_sorted_rows(ops):
    rng = np.random.default_rng(8)
    B, V, W = 6, 9001, 40
    z = np.zeros((B, V), np.float32)
    z[1] = rng.integers(-2, 3, V)
    z[2] = -np.inf
    z[2, 77] = 1.0
    z[3] = np.nan
    z[3, 5000:5003] = [np.inf, 0.5, np.inf]
    z[4] = np.arange(V) / 1000                  # ascending: every piece's last entries
    z[5] = -np.arange(V) / 1000
    zero = np.zeros(B, np.float32)
    check_select(ops, z, zero, W)
    check_select(ops, z[[0, 0, 0]], zero[:3], W)                 # equal beams
    check_select(ops, z[[2, 3]], zero[:2], W)                    # fewer candidates than W
    check_select(ops, z, np.array([-np.inf, -np.inf, np.nan, 0, -1, 2], np.float32), W)
    check_select(ops, z, zero, W, np.array([0, np.inf, -np.inf, np.nan, 3, 4], np.float32))
    check_select(ops, z, np.full(B, -np.inf, np.float32), W, None, np.ones(B, np.int32), 3)
    check_select(ops, z, np.array([-1, -1, -5, 0, 2, 2], np.float32), W, None, np.ones(B, np.int32), 3)
    # thousands of equal scores: ties go to the lower beam, then the lower token
    flat = np.zeros((40, 9001), np.float32)
    check_select(ops, flat, np.zeros(40, np.float32), 40)
    check_select(ops, flat, (np.arange(40) // 2).astype(np.float32), 256)
    check_select(ops, flat[:, :3], np.zeros(40, np.float32), 200)


def test_select_reads_odd_rows_and_strided_lse(ops):
    import self_speculative_decoding_gb300 as ssd
    rng = np.random.default_rng(9)
    B, V, W = 3, 1003, 8
    flat = torch.from_numpy(rng.standard_normal(B * V + 1).astype(np.float32)).cuda()
    z = flat[1:].view(B, V)                                      # 4-byte aligned only
    stats = torch.zeros(B, 12, dtype=torch.int32, device="cuda")
    lse = torch.logsumexp(z.double(), 1).float()
    stats.view(torch.float32)[:, 6] = lse
    scores = torch.tensor([-1.0, -2.0, -1.5], device="cuda")
    want = O.beam_select(z.cpu().numpy(), lse.cpu().numpy(), scores.cpu().numpy(), None, -1, W)
    for given in (stats, lse, lse[:, None].expand(B, 3)[:, 1], torch.stack((lse, lse), 1)[:, 0]):
        tok, par, _, _ = ssd.ops.beam_select(z, scores, W, lse=given)
        assert list(zip(tok.tolist(), par.tolist())) == [w[:2] for w in want]


def test_select_with_the_lm_heads_records(ops):
    import self_speculative_decoding_gb300 as ssd
    from tests.gpu_util import rand_bf16, rand_f32
    W, _ = rand_bf16((1024, 256), seed=1, std=0.2)
    x, _ = rand_f32((4, 256), seed=2)
    gain = torch.ones(256, device="cuda")
    logits, stats = ops.lm_head(ssd.pack_weight(W), x, gain, 1e-5)
    scores = torch.tensor([0.0, -0.5, -1.0, -9.0], device="cuda")
    tok, par, sc, _ = ops.beam_select(logits, scores, 6, lse=stats)
    lse = stats.view(torch.float32)[:, 6].cpu().numpy()
    want = O.beam_select(logits.cpu().numpy(), lse, scores.cpu().numpy(), None, -1, 6)
    assert list(zip(tok.tolist(), par.tolist())) == [w[:2] for w in want]


# --------------------------------------------------------------------------
# beam reordering


@pytest.mark.parametrize("B,W,groups,S,dh,dtype,start,stop", [
    (1, 1, (1,), 1, 8, torch.bfloat16, 0, 1), (4, 4, (3, 2), 40, 64, torch.float32, 5, 6),
    (4, 6, (2,), 129, 128, torch.bfloat16, 0, 129), (3, 2, (5,), 77, 24, torch.bfloat16, 3, 70),
    (8, 8, (4, 8), 500, 128, torch.bfloat16, 100, 411), (2, 3, (2,), 9, 64, torch.bfloat16, 4, 4)])
@pytest.mark.parametrize("only_k", [False, True])
def test_reorder(ops, B, W, groups, S, dh, dtype, start, stop, only_k):
    g = torch.Generator(device="cuda").manual_seed(S)
    k = torch.randn(B, *groups, S, dh, generator=g, device="cuda").to(dtype)
    v = None if only_k else torch.randn(B, *groups, S, dh, generator=g, device="cuda").to(dtype)
    parents = [(5 * i + 1) % B for i in range(W)]
    if W > 2:
        parents[1], parents[2] = -1, B
    ko = torch.full((W, *groups, S, dh), 9.0, dtype=dtype, device="cuda")
    vo = None if only_k else ko.clone()
    wk, wv = ko.clone(), None if only_k else ko.clone()
    for w, p in enumerate(parents):
        if 0 <= p < B:
            wk[w, ..., start:stop, :] = k[p, ..., start:stop, :]
            if not only_k:
                wv[w, ..., start:stop, :] = v[p, ..., start:stop, :]
    ops.beam_reorder(k, v, torch.tensor(parents, dtype=torch.int32).cuda(), start, stop, ko, vo)
    assert torch.equal(ko, wk) and (only_k or torch.equal(vo, wv))


def test_reorder_beyond_32_bits(ops):
    S = 1_100_000
    k = torch.empty(4, 8, S, 128, dtype=torch.bfloat16, device="cuda")
    ko = torch.empty(2, 8, S, 128, dtype=torch.bfloat16, device="cuda")
    k[:, :, S - 3:] = torch.arange(4, device="cuda", dtype=torch.bfloat16)[:, None, None, None]
    ko[:, :, S - 4:] = 50
    ops.beam_reorder(k, None, torch.tensor([3, 1], dtype=torch.int32).cuda(), S - 3, S, ko, None)
    assert (ko[0, :, S - 3:] == 3).all() and (ko[1, :, S - 3:] == 1).all() and (ko[:, :, S - 4] == 50).all()


def test_eviction_selection_and_reordering_in_a_graph(ops):
    g = torch.Generator(device="cuda").manual_seed(3)
    k, v = (torch.randn(4, 9000, 64, generator=g, device="cuda").bfloat16() for _ in range(2))
    w = torch.rand(4, 9000, generator=g, device="cuda")
    ko, vo, wo = torch.zeros(4, 700, 64, device="cuda").bfloat16(), torch.zeros(4, 700, 64, device="cuda").bfloat16(), torch.zeros(4, 700, device="cuda")
    z, sc = torch.randn(12, 40000, generator=g, device="cuda"), torch.zeros(12, device="cuda")
    bk = torch.randn(12, 3, 50, 64, generator=g, device="cuda")
    bo = torch.zeros(5, 3, 50, 64, device="cuda")

    def step():
        kept = ops.cache_evict(k, v, w, 8999, 700, ko, vo, wo, sinks=3, recent=50)
        tok, par, best, _ = ops.beam_select(z, sc, 5)
        ops.beam_reorder(bk, None, par, 7, 43, bo, None)
        return kept, tok, par, best

    want = [t.clone() for t in step()] + [t.clone() for t in (ko, vo, wo, bo)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(3):
        for t in (*got, ko, vo, wo, bo):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((*got, ko, vo, wo, bo), want))
    w.mul_(-1)                                     # other inputs of the same graph
    graph.replay()
    torch.cuda.synchronize()
    np.testing.assert_array_equal(got[0].cpu().numpy(), O.cache_evict(w.cpu().numpy(), 8999, 700, 3, 50))


# --------------------------------------------------------------------------
# together


def test_a_round_of_tree_decoding(ops):
    """Draft a tree level by level with beam_select, verify it with
    tree_attention, keep the accepted path, evict, and verify the next tree
    over the evicted cache: every step against the references."""
    H, Hkv, dh, V, n0 = 8, 2, 64, 500, 200
    rng = np.random.default_rng(11)
    table = rng.standard_normal((V, (H + 2 * Hkv) * dh)).astype(np.float32)   # a token's projections
    logit_table = (rng.standard_normal((V, V)) * 2).astype(np.float32)        # a token's draft logits
    S = 300
    k = torch.from_numpy(rng.standard_normal((Hkv, S, dh)).astype(np.float32)).bfloat16().cuda()
    v = torch.from_numpy(rng.standard_normal((Hkv, S, dh)).astype(np.float32)).bfloat16().cuda()
    w = torch.from_numpy(rng.exponential(size=(Hkv, S)).astype(np.float32)).cuda()
    n, pos, token = n0, n0, 17
    dev_table, dev_logits = torch.from_numpy(table).cuda(), torch.from_numpy(logit_table).cuda()
    for rnd in range(3):
        # ---- a tree of 1 + 3 levels of 4 nodes
        tokens, parents = [token], [-1]
        front, scores = [0], torch.zeros(1, device="cuda")
        for _ in range(3):
            at = torch.tensor([tokens[i] for i in front]).cuda()
            z = dev_logits[at].contiguous()
            lse = torch.logsumexp(z.double(), 1).float()
            tok, par, nxt, _ = ops.beam_select(z, scores, 4, lse=lse)
            want = O.beam_select(z.cpu().numpy(), lse.cpu().numpy(), scores.cpu().numpy(), None, -1, 4)
            assert list(zip(tok.tolist(), par.tolist())) == [x[:2] for x in want]
            new = list(range(len(tokens), len(tokens) + 4))
            parents += [front[p] for p in par.tolist()]
            tokens += tok.tolist()
            front, scores = new, nxt.clone()
        T = len(tokens)
        qkv = dev_table[torch.tensor(tokens).cuda()].contiguous()
        k0, v0, w0 = k.clone(), v.clone(), w.clone()
        out = ops.tree_attention(qkv, torch.tensor(parents, dtype=torch.int32).cuda(), k, v, n, pos,
                                 H, Hkv, dh, 1e4, weights=w, weights_out=w)
        c = Case.__new__(Case)
        c.H, c.Hkv, c.dh, c.n, c.T, c.pos0, c.S, c.parents = H, Hkv, dh, n, T, pos, S, parents
        c.qkv, c.k0, c.v0, c.k, c.v, c.w0 = qkv, k0, v0, k, v, w0
        c.w = w.clone()
        c.w[:, n + T:] = -3.0
        c.check(out)
        # ---- the path to the last node is taken: its rows close up behind the context
        path = O.tree_paths(parents)[-1]
        rows = torch.tensor([n + i for i in path]).cuda()
        for t in (k, v, w):
            t[:, n:n + len(path)] = t[:, rows].clone()
        n += len(path)
        pos += len(path)
        token = tokens[path[-1]]
        # ---- evict down to 180 rows
        keep = 180
        ko, vo, wo = torch.zeros_like(k), torch.zeros_like(v), torch.zeros_like(w)
        kept = ops.cache_evict(k, v, w, n, keep, ko, vo, wo, sinks=4, recent=len(path))
        np.testing.assert_array_equal(kept.cpu().numpy(), O.cache_evict(w.cpu().numpy(), n, keep, 4, len(path)))
        k, v, w, n = ko, vo, wo, keep


# --------------------------------------------------------------------------
# the binding


def test_refused_sizes_allocate_nothing(ops):
    from self_speculative_decoding_gb300 import SSDError
    z, sc = torch.zeros(4, 100, device="cuda"), torch.zeros(4, device="cuda")
    k = torch.zeros(2, 64, 64, device="cuda").bfloat16()
    w = torch.zeros(2, 64, device="cuda")
    par = torch.full((3,), -1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    now = torch.cuda.max_memory_allocated()
    for width in (0, -1, 257, 2 ** 31 - 1):
        with pytest.raises(SSDError):
            ops.beam_select(z, sc, width)
    for keep in (0, -5, 64, 2 ** 31 - 1):
        with pytest.raises(SSDError):
            ops.cache_evict(k, k, w, 63, keep, k.clone(), k.clone())
    none = torch.zeros(0, 64, 64, device="cuda").bfloat16()
    with pytest.raises(SSDError):
        ops.tree_attention(torch.zeros(3, 384, device="cuda"), par, none, none, 10, 10, 6, 0, 64, 1e4)
    assert torch.cuda.max_memory_allocated() - now < 1 << 20


def test_two_threads_at_once(ops):
    """Calls from two threads, each on its stream with tensors of its own."""
    import threading
    H, Hkv, dh, n, T = 8, 2, 64, 700, 9
    def inputs(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        qkv = torch.randn(T, (H + 2 * Hkv) * dh, generator=g, device="cuda")
        k, v = (torch.randn(Hkv, n + T, dh, generator=g, device="cuda").bfloat16() for _ in range(2))
        return qkv, torch.tensor([-1, 0, 0, 1, 1, 2, -1, 6, 7], dtype=torch.int32, device="cuda"), k, v
    def step(x):
        w = torch.zeros(Hkv, n + T, device="cuda")
        out = ops.tree_attention(*x, n, n, H, Hkv, dh, 1e4, weights=w, weights_out=w)
        ko, vo = torch.zeros_like(x[2]), torch.zeros_like(x[3])
        kept = ops.cache_evict(x[2], x[3], w, n + T, 300, ko, vo, sinks=2, recent=9)
        return out, w, kept, ko[:, :300], vo[:, :300]
    data = [inputs(s) for s in (1, 2)]
    want = [step(x) for x in data]
    torch.cuda.synchronize()
    bad, streams = [], [torch.cuda.Stream() for _ in data]
    def work(i):
        try:
            with torch.cuda.stream(streams[i]):
                for _ in range(50):
                    got = step(data[i])
                    streams[i].synchronize()
                    if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                        bad.append(i)
        except Exception as e:
            bad.append(e)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad
