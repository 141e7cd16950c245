"""The calls of several sequences on the GPU (head norms with rotation and
append, 8-bit rows, attention over them, verification of drafts) against the
fp64 references of oracle/batch.py.

Tolerances, from the roundings that the calls document (U = 2^-8, half a bf16
step relative to the value):
* rotated heads: the norm's sum, root and products are good to a few 2^-24 of
  the value, the angle to 2^-24 of half a turn, the products to 2^-24 each: |x| +
  |y| of the pair times 2e-6, then U of the result.  v is rounded once, exactly.
* 8-bit rows and their scales: exact.
* attention: the output's own rounding U |o|; probabilities times the value's
  scale, U each: U sum p |v|.  A score is off by
    d = scale (2^-17 max|q| sum |k| + 2 dh 2^-24 sum |q k|) + 1e-6,
  a probability by the factor e^(2 d): 2 d sum p |v|.
* verification: the tokens themselves.
"""

import numpy as np
import pytest
import torch

from oracle import batch as O

pytestmark = pytest.mark.gpu

U = 2.0 ** -8
NAN = float("nan")


@pytest.fixture(scope="module")
def ops():
    import __graft_entry__ as g
    g.build()
    import self_speculative_decoding_gb300 as ssd
    return ssd.ops


def whole(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def normal(rng, *shape):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32))


def bits(t):
    return t.contiguous().view(torch.uint8)


# --------------------------------------------------------------------------
# norms, rotation, append


def run_rope(ops, lengths, T, H, Hkv, dh, rows, norms="qk", counts=None, positions=None, seed=0, theta=1e4,
             eps=1e-5, layers=None, std=1.0):
    rng = np.random.default_rng(seed + T)
    B = len(lengths)
    qkv = normal(rng, B, T, (H + 2 * Hkv) * dh) * std
    shape = (B, Hkv, rows, dh) if layers is None else (B, layers, Hkv, rows, dh)
    k0, v0 = normal(rng, *shape).bfloat16().cuda(), normal(rng, *shape).bfloat16().cuda()
    k, v = k0.clone(), v0.clone()
    pick = (lambda t: t) if layers is None else (lambda t: t[:, layers // 2])
    gq = (1 + 0.3 * normal(rng, dh)) if "q" in norms else None
    gk = (1 + 0.3 * normal(rng, dh)) if "k" in norms else None
    on = lambda t: None if t is None else t.cuda()  # noqa: E731
    q = ops.rope_append(qkv.cuda(), whole(lengths), pick(k), pick(v), H, Hkv, dh, theta, q_gain=on(gq),
                        k_gain=on(gk), eps=eps, counts=None if counts is None else whole(counts),
                        positions=None if positions is None else whole(positions))
    if layers is not None:              # the other layers stay
        for now, was in ((k, k0), (v, v0)):
            rest = [i for i in range(layers) if i != layers // 2]
            assert torch.equal(bits(now[:, rest]), bits(was[:, rest]))
    got = q.double().cpu().numpy()
    K, V = pick(k).double().cpu().numpy(), pick(v).double().cpu().numpy()
    x = qkv.double().numpy().reshape(B, T, H + 2 * Hkv, dh)
    np_ = lambda t: None if t is None else t.double().numpy()  # noqa: E731
    written = np.zeros((B, rows), bool)
    for b, n in enumerate(lengths):
        c = T if counts is None else min(max(counts[b], 0), T)
        if n < 0 or n > 2 ** 31 - 1 - T:
            c = 0
        assert not got[b, c:].any()
        for t in range(c):
            p = (n if positions is None else positions[b]) + t
            slot = (n + t) % rows
            written[b, slot] = True
            for part, lo, hi, gain, res in (("q", 0, H, np_(gq), got[b, t]), ("k", H, H + Hkv, np_(gk), K[b, :, slot])):
                y = O.head_norm(x[b, t, lo:hi], gain, eps)
                want = O.rotate(y, p, theta)
                pair = np.abs(y[:, :dh // 2]) + np.abs(y[:, dh // 2:])
                tol = U * np.abs(want) + 2e-6 * np.concatenate((pair, pair), -1)
                assert np.all(np.abs(res - want) <= tol), (part, b, t, np.max(np.abs(res - want) / tol))
            want = torch.from_numpy(x[b, t, H + Hkv:]).float().bfloat16().double().numpy()
            np.testing.assert_array_equal(V[b, :, slot], want)
    keep = torch.from_numpy(~written).cuda()
    for now, was in ((pick(k), pick(k0)), (pick(v), pick(v0))):
        assert torch.equal(now.transpose(1, 2)[keep], was.transpose(1, 2)[keep])
    return q, k, v


@pytest.mark.parametrize("H,Hkv,dh", [(4, 4, 64), (8, 2, 64), (6, 2, 128), (1, 1, 128), (5, 1, 64), (64, 8, 128)])
@pytest.mark.parametrize("lengths,T,rows", [([0], 1, 1), ([7, 0, 130], 5, 200), ([1000, 255], 16, 128),
                                            ([131071], 3, 256)])
def test_rope_append(ops, H, Hkv, dh, lengths, T, rows):
    run_rope(ops, lengths, T, H, Hkv, dh, rows)


@pytest.mark.parametrize("norms", ["", "q", "k", "qk"])
def test_rope_append_norms(ops, norms):
    run_rope(ops, [5, 40], 7, 4, 2, 128, 64, norms)
    run_rope(ops, [5, 40], 7, 4, 2, 64, 64, norms, std=1e-4, eps=1e-12)


def test_rope_append_counts_positions_and_layers(ops):
    run_rope(ops, [3, 90, 17, 0, -5, 2 ** 31 - 4], 6, 4, 2, 64, 99, counts=[6, 0, 2, 9, 4, 6])
    run_rope(ops, [3, 90, 17], 6, 4, 2, 128, 99, counts=[-3, 6, 1], positions=[1_000_000, 0, -40])
    run_rope(ops, [3, 90, 17], 6, 4, 2, 128, 99, positions=[2 ** 31 - 1, 2 ** 30, 77], layers=3)
    run_rope(ops, [2 ** 31 - 1 - 6, 1], 6, 2, 1, 64, 7)
    run_rope(ops, [3], 300, 6, 3, 64, 301, theta=5e5)
    run_rope(ops, [3, 4], 5, 6, 3, 64, 301, theta=0.5)


def test_rope_append_rows_do_not_depend_on_each_other(ops):
    q, k, v = run_rope(ops, [7, 300], 9, 8, 2, 128, 512, counts=[9, 4])
    rng = np.random.default_rng(9)
    qkv = normal(rng, 2, 9, 12 * 128)
    gains = [(1 + 0.3 * normal(np.random.default_rng(1), 128)).cuda() for _ in range(2)]
    lone = []
    both = [torch.zeros_like(k) for _ in range(4)]
    all_q = ops.rope_append(qkv.cuda(), whole([7, 300]), both[0], both[1], 8, 2, 128, 1e4, *gains)
    for t in range(9):
        lone.append(ops.rope_append(qkv[:, t:t + 1].contiguous().cuda(), whole([7 + t, 300 + t]), both[2], both[3], 8, 2,
                                    128, 1e4, *gains))
    assert torch.equal(torch.cat(lone, 1), all_q)
    assert torch.equal(both[0], both[2]) and torch.equal(both[1], both[3])


# --------------------------------------------------------------------------
# 8-bit rows


def run_quantize(ops, held, lengths, Hkv, dh, block, rows, max_seq, change=None, layers=None, seed=0):
    rng = np.random.default_rng(seed)
    B = len(held)
    kv = [normal(rng, B, Hkv, rows, dh) * torch.from_numpy(10.0 ** rng.uniform(-4, 3, (1, Hkv, 1, 1))) for _ in range(2)]
    kv = [x.float().bfloat16() for x in kv]
    if change:
        change(*kv)
    mid = 0 if layers is None else layers // 2
    wide = (B, 1 if layers is None else layers, Hkv)
    eight = [torch.from_numpy(rng.integers(0, 256, (*wide, max_seq, dh)).astype(np.uint8)).cuda() for _ in range(2)]
    scales = [torch.from_numpy(rng.random((*wide, max_seq // block)).astype(np.float32)).cuda() for _ in range(2)]
    was8, was_s = [x.clone() for x in eight], [x.clone() for x in scales]
    src = [torch.zeros(*wide, rows, dh, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    for s, x in zip(src, kv):
        s[:, mid] = x.cuda()
    new = ops.cache_quantize(*(x[:, mid] for x in src), whole(held), whole(lengths),
                             *(x.view(torch.float8_e4m3fn)[:, mid] for x in eight), *(x[:, mid] for x in scales))
    want = []
    for b, (h, n) in enumerate(zip(held, lengths)):
        good = h >= 0 and h % block == 0 and h <= max_seq and n <= max_seq and n - h <= rows
        blocks = range(h // block, n // block) if good else ()
        want.append(h + block * len(blocks))
        for x, w8, ws in zip(kv, was8, was_s):
            x = x.double().numpy()[b]
            for c in blocks:
                r = x[:, np.arange(c * block, c * block + block) % rows]
                for i in range(Hkv):
                    s = O.block_scale(r[i])
                    ws[b, mid, i, c] = s
                    w8[b, mid, i, c * block:(c + 1) * block] = torch.from_numpy(O.to_e4m3(r[i] / s)).cuda()
    assert new.tolist() == want
    for got, w in zip(eight, was8):
        # (NaN keeps no sign)
        nan = (w & 0x7F) == 0x7F
        assert torch.equal(torch.where(nan, got & 0x7F, got), torch.where(nan, w & 0x7F, w))
    for got, w in zip(scales, was_s):
        assert torch.equal(got, w)


@pytest.mark.parametrize("Hkv,dh,block", [(2, 64, 32), (3, 128, 64), (1, 128, 128), (5, 64, 128), (2, 128, 32)])
@pytest.mark.parametrize("held,lengths,rows", [([0], [300], 300), ([0], [31], 64), ([128, 256], [255, 512], 256),
                                               ([0, 128, 0, 384, 128], [0, 128, 129, 511, 100], 131),
                                               ([0], [0], 1)])
def test_cache_quantize(ops, Hkv, dh, block, held, lengths, rows):
    run_quantize(ops, held, lengths, Hkv, dh, block, rows, 512)


def test_cache_quantize_strange_values(ops):
    def change(k, v):
        k[0, 0, 3, 5], k[0, 0, 40, 6], k[0, 1, 2, 2] = float("inf"), float("-inf"), NAN
        v[0, 0, :32] = 0.0
        v[0, 1, 32:64] = NAN
        v[1] = v[1] * 1e-36                             # below the smallest scale
        k[1, 0] = 3e38                                  # near the type's largest
        k[1, 1, 5] = 448.0 * 2.0 ** 3                   # the border of a scale
        k[1, 1, :5] = k[1, 1, 6:] = 0.0
    run_quantize(ops, [0, 0], [96, 64], 2, 64, 32, 100, 128, change)


def test_cache_quantize_refuses_senseless_sequences_alone(ops):
    run_quantize(ops, [-32, 0, 16, 512 + 32, 0, 64, 32], [64, 64, 96, 600, 513, 64 + 101, 32 + 100], 2, 64, 32, 100,
                 512)
    run_quantize(ops, [0, 2 ** 31 - 32], [-2 ** 31, 2 ** 31 - 1], 2, 64, 32, 100, 512)


def test_cache_quantize_many_sequences_and_layers(ops):
    rng = np.random.default_rng(5)
    held = [int(x) * 32 for x in rng.integers(0, 4, 512)]
    run_quantize(ops, held, [h + int(x) for h, x in zip(held, rng.integers(0, 100, 512))], 1, 64, 32, 128, 256)
    run_quantize(ops, [0, 64], [200, 300], 3, 128, 64, 256, 320, layers=3)


def test_eight_bits_move_once(ops):
    # moved in two steps or in one: the same bits
    rng = np.random.default_rng(6)
    k, v = (normal(rng, 2, 2, 512, 128).bfloat16().cuda() for _ in range(2))
    outs = []
    for steps in (([300, 500],), ([70, 64], [200, 200], [300, 500])):
        r = [torch.zeros(2, 2, 512, 128, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2)]
        r += [torch.zeros(2, 2, 8, device="cuda") for _ in range(2)]
        held = whole([0, 0])
        for n in steps:
            held = ops.cache_quantize(k, v, held, whole(n), *r)
        assert held.tolist() == [256, 448]
        outs.append(r)
    for x, y in zip(*outs):
        assert torch.equal(bits(x), bits(y))


# --------------------------------------------------------------------------
# attention


class Attn:
    """Seeded inputs of one call; rows that no token sees hold NaN."""

    def __init__(self, lengths, T, H, Hkv, dh, rows, held=None, block=32, max_seq=None, counts=None, window=0,
                 sinks=0, seed=0, std=1.0, layers=None, scale=None):
        rng = np.random.default_rng(seed + T + sum(lengths))
        B = len(lengths)
        self.lengths, self.T, self.H, self.Hkv, self.dh, self.rows = lengths, T, H, Hkv, dh, rows
        self.held, self.block, self.window, self.sinks = held, block, window, sinks
        self.counts, self.scale = counts, scale
        self.q = (normal(rng, B, T, H, dh) * std).bfloat16()
        ends = [n + (T if counts is None else counts[b]) for b, n in enumerate(lengths)]
        most = max(max(ends), 1)
        self.K = np.full((B, Hkv, most, dh), np.nan)      # the rows' values
        self.V = self.K.copy()
        self.seen = np.zeros((B, most), bool)
        for b, n in enumerate(lengths):
            for t in range(ends[b] - n):
                self.seen[b, O.seen_rows(n + t, window, sinks)] = True
        ring = [torch.full((B, Hkv, rows, dh), NAN, dtype=torch.bfloat16) for _ in range(2)]
        if held is not None:
            max_seq = max_seq or -(-max(max(held), 1) // block) * block
            e8 = [np.full((B, Hkv, max_seq, dh), 0x7F, np.uint8) for _ in range(2)]
            sc = [np.full((B, Hkv, max_seq // block), np.nan, np.float32) for _ in range(2)]
        for b in range(B):
            h = held[b] if held is not None else 0
            for i, x in enumerate((self.K, self.V)):
                if h:
                    n = -(-h // block)
                    code = O.to_e4m3(np.clip(rng.standard_normal((Hkv, n * block, dh)) * 90, -448, 448))
                    s = (2.0 ** rng.integers(-9, -5, (Hkv, n)) * rng.uniform(0.7, 1.4, (Hkv, n))).astype(np.float32)
                    x[b, :, :h] = (O.from_e4m3(code) * np.repeat(s, block, 1)[..., None])[:, :h]
                    code[:, [not self.seen[b, j] if j < h else True for j in range(n * block)]] = 0x7F
                    e8[i][b, :, :n * block] = code
                    used = [self.seen[b, c * block:min((c + 1) * block, h)].any() for c in range(n)]
                    sc[i][b, :, :n] = np.where(used, s, np.nan)
                for j in range(h, ends[b]):
                    if self.seen[b, j]:
                        r = normal(rng, Hkv, dh).bfloat16()
                        ring[i][b, :, j % rows] = r
                        x[b, :, j] = r.double().numpy()
        wide = (lambda t: t.cuda()) if layers is None else (
            lambda t: torch.stack([torch.full_like(t, NAN) if t.dtype != torch.uint8 else t * 0 + 0x7F
                                   if i != layers // 2 else t for i in range(layers)], 1).cuda()[:, layers // 2]
            if t.dtype == torch.uint8 else
            torch.stack([torch.full_like(t, NAN) if i != layers // 2 else t for i in range(layers)], 1).cuda()[:, layers // 2])
        self.k, self.v = wide(ring[0]), wide(ring[1])
        self.kw = {}
        if held is not None:
            self.kw = dict(zip(("k8", "v8"), (wide(torch.from_numpy(x)).view(torch.float8_e4m3fn) for x in e8)))
            self.kw.update(zip(("k_scale", "v_scale"), (wide(torch.from_numpy(x)) for x in sc)))
            self.kw["held"] = whole(held)
        if counts is not None:
            self.kw["counts"] = whole(counts)

    def call(self, ops, **kw):
        return ops.cache_attention(self.q.cuda(), self.k, self.v, whole(self.lengths), window=self.window,
                                   sinks=self.sinks, scale=self.scale, **{**self.kw, **kw})

    def check(self, out):
        got = out.double().cpu().numpy()
        G, scale = self.H // self.Hkv, self.scale or 1 / np.sqrt(self.dh)
        worst = 0.0
        for b, n in enumerate(self.lengths):
            c = self.T if self.counts is None else self.counts[b]
            assert not got[b, c:].any(), "rows behind the sequence's tokens"
            for t in range(c):
                rows = O.seen_rows(n + t, self.window, self.sinks)
                for h in range(self.H):
                    q = self.q[b, t, h].double().numpy()
                    K, V = self.K[b, h // G], self.V[b, h // G]
                    ref, spread = O.attend(q, K, V, rows, scale)
                    size = (2.0 ** -17 * np.abs(q).max() * np.abs(K[rows]).sum(1) +
                            2 * self.dh * 2.0 ** -24 * np.abs(K[rows]) @ np.abs(q)).max()
                    d = abs(scale) * size + 1e-6
                    tol = U * np.abs(ref) + (U + 2 * d) * spread + 1e-30
                    off = np.abs(got[b, t, h] - ref) / tol
                    assert np.all(off <= 1), (b, t, h, off.max())
                    worst = max(worst, off.max())
        return worst


HEADS = [(4, 4, 64), (8, 2, 64), (6, 2, 128), (8, 1, 128), (3, 3, 128)]


@pytest.mark.parametrize("H,Hkv,dh", HEADS)
@pytest.mark.parametrize("lengths,T,rows,held", [
    ([0], 1, 1, None), ([0], 5, 9, None), ([1, 0, 130], 2, 256, None), ([127], 1, 128, [96]), ([128], 1, 128, [128]),
    ([129, 300], 16, 128, [64, 288]), ([500, 3, 257], 3, 1000, [0, 0, 256]), ([640], 4, 128, [640]),
    ([1000, 31], 7, 384, [704, 0])])
def test_cache_attention(ops, H, Hkv, dh, lengths, T, rows, held):
    a = Attn(lengths, T, H, Hkv, dh, rows, held)
    a.check(a.call(ops))


@pytest.mark.parametrize("block", [32, 64, 128])
@pytest.mark.parametrize("H,Hkv,dh,lengths,T,rows,held,window,sinks", [
    (8, 2, 128, [900], 1, 128, [896], 100, 4), (8, 2, 128, [900, 77], 5, 256, [768, 0], 200, 0),
    (4, 4, 64, [900, 1000], 8, 256, [768, 896], 1, 3), (4, 1, 64, [300], 16, 256, [128], 7, 200),
    (4, 2, 128, [515], 3, 128, [512], 257, 130), (4, 2, 128, [260], 3, 300, None, 16, 5),
    (16, 2, 64, [1500], 2, 128, [1408], 128, 64), (2, 2, 128, [200, 200], 4, 128, [128, 128], 5000, 2),
    (2, 1, 128, [400], 16, 128, [384], 1, 0)])
def test_windows(ops, block, H, Hkv, dh, lengths, T, rows, held, window, sinks):
    if held is not None:
        held = [h // block * block for h in held]
        rows = max(rows, 256)
    a = Attn(lengths, T, H, Hkv, dh, rows, held, block, window=window, sinks=sinks)
    a.check(a.call(ops))


@pytest.mark.parametrize("H,Hkv,dh,T", [(128, 1, 64, 1), (16, 1, 128, 8), (2, 2, 128, 128), (32, 1, 64, 1),
                                        (33, 1, 64, 1), (64, 1, 128, 1), (65, 1, 64, 1), (8, 8, 64, 100),
                                        (24, 2, 128, 10), (5, 1, 128, 25)])
def test_rows_up_to_a_tile(ops, H, Hkv, dh, T):
    a = Attn([300, 290], T, H, Hkv, dh, 256, [256, 224], counts=[T, max(1, T - 3)])
    a.check(a.call(ops))


def test_uneven_sequences(ops):
    rng = np.random.default_rng(3)
    lengths = [int(x) for x in rng.integers(0, 700, 37)]
    held = [max(0, n - int(x)) // 32 * 32 for n, x in zip(lengths, rng.integers(0, 64, 37))]
    counts = [int(x) for x in rng.integers(0, 4, 37)]
    a = Attn(lengths, 3, 4, 2, 64, 128, held, counts=counts)
    a.check(a.call(ops))
    a = Attn(lengths, 3, 4, 2, 64, 128, held, counts=counts, window=90, sinks=5, layers=3)
    a.check(a.call(ops))


def test_many_short_sequences(ops):
    rng = np.random.default_rng(4)
    lengths = [int(x) for x in rng.integers(0, 9, 512)]
    a = Attn(lengths, 1, 2, 1, 64, 10)
    a.check(a.call(ops))


def plain_attention(a_q, K, V, length, scale, window=0, sinks=0):
    """One sequence in 64 bits as torch operations: q [T, H, dh], K, V [Hkv, n,
    dh] -> the result, sum p |v|, and a bound of the scores' error."""
    T, H, dh = a_q.shape
    Hkv, n = K.shape[:2]
    q = a_q.double().view(T, Hkv, H // Hkv, dh).permute(1, 2, 0, 3)
    s = scale * (q @ K[:, None].transpose(2, 3))
    j, pos = torch.arange(n, device=q.device), length + torch.arange(T, device=q.device)[:, None]
    hidden = j > pos
    if window:
        hidden |= (j >= sinks) & (j <= pos - window)
    p = torch.softmax(s.masked_fill(hidden, -float("inf")), -1)
    d = scale * (2.0 ** -17 * q.abs().amax() * K.abs().sum(-1).amax() +
                 2 * dh * 2.0 ** -24 * (q.abs() @ K[:, None].abs().transpose(2, 3)).amax()) + 1e-6
    back = lambda x: x.permute(2, 0, 1, 3).reshape(T, H, dh)  # noqa: E731
    return back(p @ V[:, None]), back(p @ V[:, None].abs()), d.item()


@pytest.mark.parametrize("lengths,T,H,Hkv,dh,window,std", [
    ([131000], 1, 64, 8, 128, 0, 1.5), ([60000, 3, 9000], 3, 8, 2, 64, 0, 3.0), ([9000] * 9, 9, 16, 2, 128, 0, 1.5),
    ([20000, 30001], 5, 6, 6, 128, 0, 4.0), ([40000, 17000], 16, 8, 1, 128, 0, 1.0), ([30000], 2, 40, 40, 128, 9000, 2.0),
    ([50001], 40, 3, 1, 64, 20011, 2.0), ([700] * 300, 1, 8, 2, 64, 0, 2.0)])
def test_long_contexts(ops, lengths, T, H, Hkv, dh, window, std):
    # a CTA has many tiles, and runs of several sequences and heads
    g = torch.Generator(device="cuda").manual_seed(T + H)
    B, block, rows, sinks = len(lengths), 64, 256, 7 if window else 0
    S = -(-max(lengths) // block) * block
    held = [max(0, n - 31) // block * block for n in lengths]
    q = (torch.randn(B, T, H, dh, generator=g, device="cuda") * std).bfloat16()
    k, v = (torch.randn(B, Hkv, rows, dh, generator=g, device="cuda").bfloat16() for _ in range(2))
    k8, v8 = ((torch.randn(B, Hkv, S, dh, generator=g, device="cuda") * 90).clamp_(-448, 448).to(torch.float8_e4m3fn)
              for _ in range(2))
    ks, vs = (torch.rand(B, Hkv, S // block, generator=g, device="cuda") / 90 + 0.004 for _ in range(2))
    out = ops.cache_attention(q, k, v, whole(lengths), k8=k8, v8=v8, k_scale=ks, v_scale=vs, held=whole(held),
                              window=window, sinks=sinks).double()
    for b in range(0, B, max(1, B // 9)):
        at = torch.arange(held[b], lengths[b] + T, device="cuda") % rows
        K, V = (torch.cat((e[b, :, :held[b]].double() * s[b, :, :held[b] // block].double().repeat_interleave(block, 1)[..., None],
                           x[b, :, at].double()), 1) for e, s, x in ((k8, ks, k), (v8, vs, v)))
        ref, spread, d = plain_attention(q[b], K, V, lengths[b], dh ** -0.5, window, sinks)
        off = (out[b] - ref).abs() / (U * ref.abs() + (U + 2 * d) * spread)
        assert off.max().item() <= 1, (b, off.max().item())


def test_scores_far_apart(ops):
    # one key takes nearly all, then a larger one comes; and 16 units of scale
    a = Attn([700], 2, 4, 2, 128, 128, [640], std=8.0)
    a.check(a.call(ops))
    a = Attn([700], 2, 4, 2, 64, 128, [640], scale=2.0)
    a.check(a.call(ops))
    a = Attn([300], 2, 4, 2, 64, 302, scale=-0.5)
    a.check(a.call(ops))


@pytest.mark.parametrize("T,H,Hkv", [(1, 4, 1), (3, 4, 1), (9, 4, 1)])
@pytest.mark.parametrize("far", [-1e30, -2e38, 2e38])
def test_scores_near_the_ends_of_the_range(ops, T, H, Hkv, far):
    # equal scores, however far from 0, weigh their rows alike: 2^k sums are exact
    dh, n, held = 64, 300, 256
    q = torch.zeros(1, T, H, dh, device="cuda").bfloat16()
    q[..., 0] = 2.0 ** 60 if far > 0 else -2.0 ** 60
    row = abs(far) / 2.0 ** 60
    e = int(np.floor(np.log2(row)))
    rng = np.random.default_rng(3)
    k = torch.zeros(1, Hkv, 512, dh, device="cuda").bfloat16()
    k[..., 0] = 2.0 ** e
    v = normal(rng, 1, Hkv, 512, dh).bfloat16().cuda()
    k8 = torch.zeros(1, Hkv, held, dh, device="cuda").to(torch.float8_e4m3fn)
    k8[..., 0] = 1.0
    v8 = normal(rng, 1, Hkv, held, dh).to(torch.float8_e4m3fn).cuda()
    ks = torch.full((1, Hkv, held // 64), 2.0 ** e, device="cuda")
    vs = torch.ones_like(ks)
    out = ops.cache_attention(q, k, v, whole([n]), k8=k8, v8=v8, k_scale=ks, v_scale=vs, held=whole([held]), scale=1.0)
    V = torch.cat((v8.double()[0, 0], v.double()[0, 0, held:n + T]))
    for t in range(T):
        want, spread = V[:n + 1 + t].mean(0), V[:n + 1 + t].abs().mean(0)
        off = (out[0, t].double() - want).abs() / (U * want.abs() + U * spread + 1e-30)
        assert off.max().item() <= 1, off.max().item()


def test_a_mass_of_small_weights_beside_a_large_one(ops):
    # a first key 12 above 20000 others, whose sum is a tenth of it: none of
    # them may be lost
    n, H, dh = 20000, 2, 64
    code = torch.zeros(1, 1, n + 96, dh, dtype=torch.uint8, device="cuda")
    k8 = code.view(torch.float8_e4m3fn)
    k8[:, :, 0, 0] = 12.0
    v8 = torch.zeros_like(code).view(torch.float8_e4m3fn)
    v8[:, :, 1:, 1] = 1.0
    one = torch.ones(1, 1, (n + 96) // 32, device="cuda")
    q = torch.zeros(1, 1, H, dh, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 8.0
    ring = torch.zeros(1, 1, 128, dh, dtype=torch.bfloat16, device="cuda")
    out = ops.cache_attention(q, ring, ring, whole([n]), k8=k8, v8=v8, k_scale=one, v_scale=one, held=whole([n]))
    rest = (n - 1) * np.exp(-12.0)
    want = rest / (1 + rest + np.exp(-12.0))
    assert abs(out[0, 0, 0, 1].item() - want) <= 3 * U * want
    assert out[0, 0, 0, 2:].abs().max().item() == 0


@pytest.mark.parametrize("what", [NAN, float("inf"), float("-inf")])
def test_rows_that_a_token_does_not_see_may_hold_anything(ops, what):
    # drafted rows, and rows that leave the window from one token to the next
    H, Hkv, dh, T = 4, 2, 64, 6
    a = Attn([200], T, H, Hkv, dh, 512, [128], window=100, sinks=2)
    clean = a.call(ops)
    a.check(clean)
    k, v = a.k.clone(), a.v.clone()
    a.v[:, :, 203, 7] = what
    a.k[:, :, 204, 3] = what
    out = a.call(ops)
    assert torch.equal(out[:, :3], clean[:, :3])
    cols = [i for i in range(dh) if i != 7]
    assert torch.equal(out[:, 3, :, cols], clean[:, 3, :, cols])
    assert not torch.isfinite(out[:, 3, :, 7]).any()
    if what != what:
        assert torch.isnan(out[:, 4:]).all()
    a.k, a.v = k, v
    # rows 101 .. 105 leave the window one by one; 8-bit rows hold NaN there
    low = 101
    e = a.kw["v8"].view(torch.uint8)
    was = e.clone()
    e[:, :, low + 1, 9] = 0x7F
    out = a.call(ops)
    assert torch.isnan(out[:, :2, :, 9]).all()
    assert torch.equal(out[:, 2:], clean[:, 2:])
    cols = [i for i in range(dh) if i != 9]
    assert torch.equal(out[..., cols], clean[..., cols])
    e.copy_(was)
    e = a.kw["k8"].view(torch.uint8)
    e[:, :, low + 2, 9] = 0x7F
    out = a.call(ops)
    assert torch.isnan(out[:, :3]).all() and torch.equal(out[:, 3:], clean[:, 3:])


def test_values_that_are_not_finite_reach_their_column(ops):
    a = Attn([300], 2, 4, 2, 128, 256, [256])
    clean = a.call(ops)
    a.kw["v8"].view(torch.uint8)[:, :, 50, 11] = 0x7F
    a.v[:, :, 280 % 256, 12] = float("inf")
    out = a.call(ops)
    assert torch.isnan(out[..., 11]).all() and torch.isinf(out[..., 12]).all()
    cols = [i for i in range(128) if i not in (11, 12)]
    assert torch.equal(out[..., cols], clean[..., cols])


def test_queries_that_are_not_finite_or_zero(ops):
    a = Attn([300], 4, 4, 2, 64, 256, [256])
    clean = a.call(ops)
    a.q[0, 1, 2, 5] = float("inf")
    a.q[0, 2, 0, 1] = NAN
    a.q[0, 3] = 0.0
    out = a.call(ops)
    assert torch.isnan(out[0, 1, 2]).all() and torch.isnan(out[0, 2, 0]).all()
    assert torch.equal(out[0, 0], clean[0, 0]) and torch.equal(out[0, 1, [0, 1, 3]], clean[0, 1, [0, 1, 3]])
    mean = torch.from_numpy(a.V[0, :, :304]).mean(1)
    assert (out[0, 3].cpu().double() - mean.repeat_interleave(2, 0)).abs().max() <= 0.02
    a.q = (a.q.nan_to_num(0, 0, 0) * 1e-38).bfloat16()
    assert torch.isfinite(a.call(ops)).all()
    a.q = torch.full_like(a.q, 3e38)
    assert torch.isnan(a.call(ops)).any() or torch.isfinite(a.call(ops)).all()


def test_scales_far_apart(ops):
    # values of 2^-100 and of 2^100: what the others weigh stays
    a = Attn([256], 1, 2, 1, 64, 128, [256], block=128)
    a.kw["v_scale"][:, :, 0] = 2.0 ** -100
    a.V[:, :, :128] = 0.0
    a.check(a.call(ops))
    a.kw["v_scale"][:, :, 0] = 0.0
    a.check(a.call(ops))
    a.kw["k_scale"][:, :, 1] = 0.0
    a.K[:, :, 128:256] = 0.0
    a.check(a.call(ops))


@pytest.mark.parametrize("T,H", [(1, 2), (3, 4), (5, 8)])
@pytest.mark.parametrize("e", [-115, -64, 64, 115, 119])
def test_scales_near_the_ends_of_the_range(ops, T, H, e):
    rng = np.random.default_rng(400 + e)
    n, dh = 512 - T, 64
    q = normal(rng, 1, T, H, dh).bfloat16().cuda()
    k8, v8 = (normal(rng, 1, 1, 512, dh).cuda().to(torch.float8_e4m3fn) for _ in range(2))
    ks = torch.ones(1, 1, 512 // 32, device="cuda")
    vs = torch.from_numpy(2.0 ** rng.integers(e - 5, e + 1, (1, 1, 512 // 32))).float().cuda()
    ring = torch.full((1, 1, 128, dh), NAN, device="cuda").bfloat16()
    out = ops.cache_attention(q, ring, ring, whole([n]), k8=k8, v8=v8, k_scale=ks, v_scale=vs, held=whole([512]))
    V = v8.double()[0, 0] * vs.double()[0, 0].repeat_interleave(32)[:, None]
    for t in range(T):
        p = torch.softmax(q[0, t].double() @ k8.double()[0, 0, :n + 1 + t].T / 8.0, -1)
        want, spread = p @ V[:n + 1 + t], p @ V[:n + 1 + t].abs()
        # the result's rounding, and the weights' to fp16 (2^-11; the sums' are far below)
        off = (out[0, t].double() - want).abs() / (U * want.abs() + 2.0 ** -10 * spread)
        assert off.max().item() <= 1, off.max().item()


def test_senseless_sequences_are_nan_and_alone(ops):
    good = Attn([200, 150, 90], 2, 4, 2, 64, 128, [128, 96, 64])
    want = good.call(ops)
    good.check(want)
    k8 = {x: torch.cat([good.kw[x].view(torch.uint8)] * 3).view(torch.float8_e4m3fn) for x in ("k8", "v8")}
    sc = {x: torch.cat([good.kw[x]] * 3) for x in ("k_scale", "v_scale")}
    q, k, v = (torch.cat([x.cuda()] * 3) for x in (good.q, good.k, good.v))
    lengths = [200, 150, 90, -1, 2 ** 31 - 1, 100, 2 ** 31 - 300, 500, 90]
    held = [128, 96, 64, 0, 0, 103, -32, 128, 160]
    counts = [2, 2, 2, 2, 2, 2, 2, 2, 2]
    out = ops.cache_attention(q, k, v, whole(lengths), held=whole(held), counts=whole(counts), **k8, **sc)
    assert torch.equal(out[:3], want) or (out[:3].float() - want.float()).abs().max() < 0.05
    good.check(out[:3])
    assert torch.isnan(out[3:]).all()
    counts = [2, -1, 3, 0, 2, 2, 2, 2, 2]
    out = ops.cache_attention(q, k, v, whole(lengths), held=whole(held), counts=whole(counts), **k8, **sc)
    assert torch.isnan(out[1:3]).all() and torch.isnan(out[3:]).all()
    # a ring whose rows are no multiple of 128 must not have turned over
    r = k[:1, :, :100].contiguous()
    out = ops.cache_attention(q[:1], r, r, whole([101]))
    assert torch.isnan(out).all()
    assert torch.isfinite(ops.cache_attention(q[:1], r.nan_to_num(0), r.nan_to_num(0), whole([98]))).all()


def test_calls_repeat_their_bits_and_ignore_the_workspace(ops):
    import self_speculative_decoding_gb300 as ssd
    from self_speculative_decoding_gb300 import _abi
    lib = _abi.lib()
    a = Attn([700, 340], 3, 8, 2, 128, 256, [512, 320])
    want = a.call(ops)
    a.check(want)
    need = lib.ssd_op_cache_attention_workspace(2, 3, 8, 2, 128)
    q, lengths = a.q.cuda(), whole(a.lengths)
    k8, v8, ks, vs, held = (a.kw[x] for x in ("k8", "v8", "k_scale", "v_scale", "held"))
    for fill in (0, 0xFF):
        ws = torch.full((need + 256,), fill, dtype=torch.uint8, device="cuda")
        out = torch.empty_like(want)
        st = lib.ssd_op_cache_attention(
            q.data_ptr(), 2, 3, lengths.data_ptr(), None, a.k.data_ptr(), a.v.data_ptr(), 256, 2 * 256 * 128,
            k8.data_ptr(), v8.data_ptr(), ks.data_ptr(), vs.data_ptr(), held.data_ptr(), k8.shape[2], 32,
            2 * k8.shape[2] * 128, 2 * ks.shape[2], 0, 0, 8, 2, 128, 128 ** -0.5, out.data_ptr(), ws.data_ptr(),
            need, ssd.stream_handle())
        assert st == 0
        assert torch.equal(out, want)
        assert bool((ws[need:] == fill).all())


@pytest.mark.parametrize("lengths,T,H,Hkv,dh,counts", [
    ([30000], 1, 16, 2, 128, None),                    # one pair over many CTAs
    ([2000, 0, 700], 2, 24, 24, 64, [2, 0, 1]),        # many pairs, tokens left out
    ([5000, 300], 3, 16, 4, 128, None),                # twelve rows
    ([9000, 4000, 10], 9, 16, 2, 128, [9, 3, 9])])     # 72 rows
def test_a_wait_that_runs_out_marks_its_rows(ops, lengths, T, H, Hkv, dh, counts):
    from self_speculative_decoding_gb300 import _abi
    call = _abi.lib().ssd_debug_cache_give_up
    B, rows, block = len(lengths), 256, 64
    g = torch.Generator(device="cuda").manual_seed(T)
    q = torch.randn(B, T, H, dh, generator=g, device="cuda").bfloat16()
    k, v = (torch.randn(B, Hkv, rows, dh, generator=g, device="cuda").bfloat16() for _ in range(2))
    S = -(-max(lengths) // block) * block
    held = whole([max(0, n - 100) // block * block for n in lengths])
    k8, v8 = (torch.randn(B, Hkv, S, dh, generator=g, device="cuda").to(torch.float8_e4m3fn) for _ in range(2))
    ks, vs = (torch.ones(B, Hkv, S // block, device="cuda") for _ in range(2))
    def run():  # noqa: E306
        return ops.cache_attention(q, k, v, whole(lengths), k8=k8, v8=v8, k_scale=ks, v_scale=vs, held=held,
                                   counts=None if counts is None else whole(counts))
    want = run()
    assert torch.isfinite(want).all()
    live = torch.ones(B, T, dtype=torch.bool, device="cuda")
    for b, c in enumerate(counts or ()):
        live[b, c:] = False
    pairs = 0
    try:
        for cta in (0, 1, 40, 140):
            call(cta)
            out = run()
            call(-1)
            lost = torch.isnan(out).permute(0, 2, 1, 3).reshape(B, Hkv, H // Hkv, T, dh)
            for b in range(B):
                for h in range(Hkv):
                    x = lost[b, h][:, live[b]]
                    assert x.all() or not x.any()
                    pairs += bool(x.numel() and x.any())
                    assert not lost[b, h][:, ~live[b]].any()
            assert torch.equal(out[~torch.isnan(out)], want[~torch.isnan(out)])
            assert torch.equal(run(), want)
    finally:
        call(-1)
    assert pairs >= 4 and pairs <= 4 * max(2, 2 * B * Hkv // 100 + 3)


def test_graphs_follow_the_lengths(ops):
    a = Attn([700, 340], 3, 8, 2, 128, 1024)
    a.k.nan_to_num_(0)
    a.v.nan_to_num_(0)
    lengths, q = whole(a.lengths), a.q.cuda()
    side, outs, graphs = torch.cuda.Stream(), [], []
    ops.cache_attention(q, a.k, a.v, lengths)
    torch.cuda.synchronize()
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            outs.append(ops.cache_attention(q, a.k, a.v, lengths))
        graphs.append(g)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for n in ([700, 340], [1, 0], [1021, 1000], [128, 127]):
        lengths.copy_(whole(n))
        want = ops.cache_attention(q, a.k, a.v, lengths)
        torch.cuda.synchronize()
        for s, g in zip((s1, s2), graphs):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want) and torch.equal(outs[1], want)


def test_offsets_beyond_32_bits(ops):
    Hkv, dh, S, n = 9, 128, 2_400_000, 1000
    k8, v8 = (torch.zeros(1, Hkv, S, dh, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2))
    ks, vs = (torch.ones(1, Hkv, S // 64, device="cuda") for _ in range(2))
    rng = np.random.default_rng(8)
    k, v = (normal(rng, 1, Hkv, 2048, dh).bfloat16().cuda() for _ in range(2))
    held = ops.cache_quantize(k, v, whole([0]), whole([n]), k8, v8, ks, vs)
    assert held.tolist() == [960]
    q = normal(rng, 1, 1, 2 * Hkv, dh).bfloat16().cuda()
    out = ops.cache_attention(q, k, v, whole([n]), k8=k8, v8=v8, k_scale=ks, v_scale=vs, held=held)
    small = [x[:, :, :960].contiguous() for x in (k8.view(torch.uint8), v8.view(torch.uint8))]
    want = ops.cache_attention(q, k, v, whole([n]), k8=small[0].view(torch.float8_e4m3fn),
                               v8=small[1].view(torch.float8_e4m3fn), k_scale=ks[:, :, :15].contiguous(),
                               v_scale=vs[:, :, :15].contiguous(), held=held)
    assert torch.equal(out, want)
    # rows far along one head's cache, told apart by their values
    far = 2_300_032
    v8.view(torch.uint8)[:, :, :far] = 0x38                              # 1.0
    out = ops.cache_attention(q * 0, k, v, whole([far]), k8=k8, v8=v8, k_scale=ks, v_scale=vs, held=whole([far]))
    assert (out.float() - 1).abs().max().item() < 0.01
    k8.view(torch.uint8)[:, :, far - 70] = 0x38
    v8.view(torch.uint8)[:, :, far - 70] = 0x40                          # 2.0
    out = ops.cache_attention(q.abs() * 0 + 3, k, v, whole([far]), k8=k8, v8=v8, k_scale=ks, v_scale=vs,
                              held=whole([far]))
    assert (out.float() - 2).abs().max().item() < 0.02


# --------------------------------------------------------------------------
# verification


def run_verify(ops, p, q, drafts, au, su, counts=None):
    B, d1, V = p.shape
    on = lambda x, t: torch.from_numpy(np.ascontiguousarray(x)).to(t).cuda()  # noqa: E731
    tokens, n = ops.verify_drafts(on(p, torch.float32), on(drafts, torch.int32), on(au, torch.float32),
                                  on(su, torch.float32), q=None if q is None else on(q, torch.float32),
                                  counts=None if counts is None else whole(counts))
    tokens, n = tokens.tolist(), n.tolist()
    for b in range(B):
        c = d1 - 1 if counts is None else min(max(counts[b], 0), d1 - 1)
        f = lambda x: np.asarray(x, np.float32).astype(np.float64)  # noqa: E731
        want = O.verify(f(p[b, :c + 1]), None if q is None else f(q[b]), drafts[b, :c], f(au[b]), float(f(su[b])))
        assert tokens[b] == want + [-1] * (d1 - len(want)), (b, tokens[b], want)
        assert n[b] == len(want)
    return tokens, n


def probabilities(rng, *shape, sharp=2.0):
    z = rng.standard_normal(shape) * sharp
    e = np.exp(z - z.max(-1, keepdims=True))
    return (e / e.sum(-1, keepdims=True)).astype(np.float32)


@pytest.mark.parametrize("V", [1, 2, 31, 32, 33, 513, 1000, 4099, 32000, 128003])
@pytest.mark.parametrize("given", [True, False])
def test_verify_drafts(ops, V, given):
    rng = np.random.default_rng(V)
    B, d = (33, 5) if V < 5000 else (7, 3)
    p = probabilities(rng, B, d + 1, V)
    q = None
    if given:
        q = 0.5 * probabilities(rng, B, d, V) + 0.5 * p[:, :d]
    drafts = np.array([[rng.choice(V, p=(p[b, j].astype(np.float64) / p[b, j].astype(np.float64).sum())) for j in range(d)] for b in range(B)])
    run_verify(ops, p, q, drafts, rng.random((B, d)), rng.random(B))
    run_verify(ops, p, q, drafts, rng.random((B, d)) * 0.5, rng.random(B), [int(x) for x in rng.integers(-1, d + 2, B)])


def test_verify_drafts_borders(ops):
    # exact sums: every multiple of 1/64, at the border itself and one step below
    V = 64
    p = np.full((2 * V, 1, V), 1 / V)
    su = np.repeat(np.arange(V) / V, 2).astype(np.float32)
    su[1::2] = np.nextafter(su[1::2] + np.float32(1 / V), np.float32(0))
    run_verify(ops, p, None, np.zeros((2 * V, 0), int), np.zeros((2 * V, 0)), su)
    # u q = p: not accepted; the next below: accepted
    p = np.zeros((2, 2, 4)) + 0.25
    q = np.zeros((2, 1, 4)) + 0.25
    q[:, 0] = (0.5, 0.5, 0.0, 0.0)
    au = np.array([[0.5], [np.nextafter(np.float32(0.5), np.float32(0))]])
    tokens, n = run_verify(ops, p, q, np.array([[0], [0]]), au, np.array([0.0, 0.9]))
    assert n == [1, 2] and tokens[0][0] == 2


def test_verify_drafts_edges(ops):
    rng = np.random.default_rng(2)
    B, d, V = 10, 3, 300
    p, q = probabilities(rng, B, d + 1, V), probabilities(rng, B, d, V)
    drafts = rng.integers(0, V, (B, d))
    drafts[0, 0], drafts[1, 1], drafts[2, 0] = -1, V, 2 ** 31 - 1
    q[3, 0] = p[3, 0]                       # nothing left, and u makes it so
    p[4, 0] = 0.0                           # nothing at all
    p[5, 0, 7], q[5, 0, 9], p[6, 0, 3] = np.nan, np.nan, -1.0
    p[7, 0] = q[7, 0] * 0.5                 # less everywhere
    au = np.full((B, d), 0.999999)
    su = rng.random(B)
    su[8], su[9] = 1.0, 2.0
    for qq in (q, None):
        run_verify(ops, p, qq, drafts, au, su)
    p[6, :, 5] = np.inf
    tokens, n = run_verify(ops, p, None, np.full((B, d), 8), np.ones((B, d)), su)
    assert n[6] == 0 and n[4] == 0


def test_verify_many_drafts_and_sequences(ops):
    rng = np.random.default_rng(3)
    p = probabilities(rng, 3, 1025, 40)
    run_verify(ops, p, None, p[:, :1024].argmax(-1), rng.random((3, 1024)) * 1e-3, rng.random(3))
    p = probabilities(rng, 512, 3, 50)
    run_verify(ops, p, probabilities(rng, 512, 2, 50), rng.integers(0, 50, (512, 2)), rng.random((512, 2)), rng.random(512))


# --------------------------------------------------------------------------
# streams, threads, a whole run


def test_another_stream_and_a_given_output(ops):
    a = Attn([300, 40], 2, 4, 2, 64, 256, [256, 0])
    want = a.call(ops)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out = torch.empty_like(want)
        assert a.call(ops, out=out) is not None
    s.synchronize()
    assert torch.equal(out, want)


def test_two_threads_and_streams_at_once(ops):
    # calls that start beside one another's ends, from two threads, say what they say alone
    import threading
    def work(seed):  # noqa: E306
        rng = np.random.default_rng(seed)
        H, Hkv, dh, V, T = (16, 2, 128, 5000, 3) if seed else (8, 8, 64, 32000, 1)
        k, v = (torch.zeros(3, Hkv, 1024, dh, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        k8, v8 = (torch.zeros(3, Hkv, 1024, dh, device="cuda").to(torch.float8_e4m3fn) for _ in range(2))
        ks, vs = (torch.ones(3, Hkv, 1024 // 64, device="cuda") for _ in range(2))
        lengths, held = whole([0, 0, 0]), whole([0, 0, 0])
        p = torch.from_numpy(probabilities(rng, 3, T + 1, V).astype(np.float32)).cuda()
        au, su = (torch.from_numpy(rng.random(n).astype(np.float32)).cuda() for n in ((3, T), 3))
        drafts = torch.from_numpy(rng.integers(0, V, (3, T)).astype(np.int32)).cuda()
        qkv = [normal(rng, 3, 200, (H + 2 * Hkv) * dh).cuda()] + [normal(rng, 3, T, (H + 2 * Hkv) * dh).cuda()
                                                                  for _ in range(30)]
        said = []
        for x in qkv:
            q = ops.rope_append(x, lengths, k, v, H, Hkv, dh, 1e4)
            if x.shape[1] == T:
                said.append(ops.cache_attention(q, k, v, lengths, k8, v8, ks, vs, held, window=150, sinks=3))
                said += ops.verify_drafts(p, drafts, au, su)
            lengths = lengths + x.shape[1]
            held = ops.cache_quantize(k, v, held, lengths, k8, v8, ks, vs)
        return said + [k, v, bits(k8), bits(v8), ks, vs, held]

    want = [work(i) for i in range(2)]
    torch.cuda.synchronize()
    got, errors = [None, None], []

    def run(i):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                got[i] = work(i)
            s.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for w, g in zip(want, got):
        assert all(torch.isfinite(x.float()).all() for x in w[:1])
        assert len(w) == len(g) and all(torch.equal(x, y) for x, y in zip(w, g))


def test_arguments_of_the_python_calls(ops):
    a = Attn([300, 40], 2, 4, 2, 64, 256, [256, 0])
    q, k, v, n = a.q.cuda(), a.k, a.v, whole(a.lengths)
    for bad in (dict(k8=None), dict(held=None), dict(v_scale=a.kw["v_scale"][:, :, :1].contiguous()),
                dict(counts=whole([1])), dict(out=q.float()), dict(held=a.kw["held"].long()),
                dict(k8=a.kw["k8"].view(torch.uint8))):
        with pytest.raises((ValueError, RuntimeError)):
            a.call(ops, **bad)
    for args in ((q.float(), k, v, n), (q, k.float(), v, n), (q, k, v[:, :1], n), (q, k, v, n.cpu()),
                 (q[..., :32], k, v, n), (q, k.transpose(1, 2), v, n), (q, k[:1], v[:1], n)):
        with pytest.raises((ValueError, RuntimeError)):
            ops.cache_attention(*args)
    with pytest.raises((ValueError, RuntimeError)):
        ops.rope_append(torch.zeros(2, 300, 8 * 64, device="cuda"), n, k, v, 4, 2, 64, 1e4)
    with pytest.raises((ValueError, RuntimeError)):
        ops.verify_drafts(torch.zeros(2, 3, 9, device="cuda"), whole([[1, 2]]), torch.zeros(2, 2, device="cuda"),
                          torch.zeros(2, device="cuda"))
    with pytest.raises((ValueError, RuntimeError)):
        ops.cache_quantize(k, v, n, n, a.kw["k8"], a.kw["v8"], a.kw["k_scale"], a.kw["v_scale"], held_out=n)


def test_rounds_of_drafting_as_a_graph(ops):
    """Rounds of two sequences, a layer each: drafts through a window over the
    8-bit cache, a verify pass over all of it, verification, rows to 8 bits;
    replayed from a graph they say the same, and the caches hold the rows of the
    tokens that were said."""
    B, d, H, Hkv, dh, V, block, rows, S = 2, 3, 4, 2, 64, 200, 32, 128, 512
    rng = np.random.default_rng(11)
    embed = normal(rng, V, (H + 2 * Hkv) * dh).cuda()
    head = (normal(rng, H * dh, V) * 0.2).cuda()
    gq, gk = ((1 + 0.2 * normal(rng, dh)).cuda() for _ in range(2))
    k, v = (torch.zeros(B, Hkv, rows, dh, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k8, v8 = (torch.zeros(B, Hkv, S, dh, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2))
    ks, vs = (torch.ones(B, Hkv, S // block, device="cuda") for _ in range(2))
    lengths, held = whole([0, 0]), whole([0, 0])
    last = whole([5, 9])
    u = torch.zeros(B, 2 * d + 1, device="cuda")         # the round's random numbers

    def layer(tok, at, **window):
        q = ops.rope_append(embed[tok.long()], at, k, v, H, Hkv, dh, 1e4, gq, gk)
        o = ops.cache_attention(q, k, v, at, k8=k8, v8=v8, k_scale=ks, v_scale=vs, held=held, **window)
        return torch.softmax(o.flatten(2).float() @ head, -1)

    def round_():
        drafts, probs, tok = [], [], last
        for j in range(d):
            pr = layer(tok[:, None], lengths + j, window=40, sinks=2)[:, 0]
            past = (pr.double().cumsum(1) > u[:, d + j:d + j + 1].double()).int().argmax(1).int()
            drafts.append(past)
            probs.append(pr)
            tok = past
        drafts = torch.stack(drafts, 1).contiguous()
        p = layer(torch.cat((last[:, None], drafts), 1), lengths)
        tokens, n = ops.verify_drafts(p.contiguous(), drafts, u[:, :d].contiguous(), u[:, 2 * d].contiguous(),
                                      q=torch.stack(probs, 1).contiguous())
        lengths.add_(n)
        last.copy_(tokens.gather(1, (n - 1).clamp(min=0).long()[:, None])[:, 0].clamp(0, V - 1))
        held.copy_(ops.cache_quantize(k, v, held, lengths, k8, v8, ks, vs))
        return tokens, n

    def reset():
        for x in (k, v, lengths, held):
            x.zero_()
        k8.view(torch.uint8).zero_()
        v8.view(torch.uint8).zero_()
        last.copy_(whole([5, 9]))

    us = [torch.from_numpy(np.random.default_rng(100 + i).random((B, 2 * d + 1)).astype(np.float32)).cuda()
          for i in range(60)]
    runs = []
    for graphed in (False, True):
        reset()
        said = [[], []]
        if graphed:
            u.copy_(us[0])
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                round_()
            side.synchronize()
            reset()
            torch.cuda.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                out = round_()
            torch.cuda.synchronize()
        for x in us:
            u.copy_(x)
            if graphed:
                g.replay()
            else:
                out = round_()
            for b in range(B):
                said[b] += out[0][b, :out[1][b]].tolist()
        assert [len(s) for s in said] == lengths.tolist() and held.tolist() == [n // block * block for n in lengths.tolist()]
        runs.append(said)
    assert runs[0] == runs[1]
    # the rows that a plain program would hold
    for b, said in enumerate(runs[0]):
        seq = [[5, 9][b]] + said[:-1]                    # the token of each row
        x = embed[torch.tensor(seq, device="cuda")].double().cpu().numpy().reshape(len(seq), H + 2 * Hkv, dh)
        n8 = len(seq) // block * block
        for i in range(Hkv):
            K = np.stack([O.rotate(O.head_norm(x[p, H + i], gk.double().cpu().numpy(), 1e-5), p, 1e4) for p in range(len(seq))])
            for mine, want, s in ((k8, K, ks), (v8, x[:, H + Hkv + i], vs)):
                s = np.repeat(s[b, i, :n8 // block].double().cpu().numpy(), block)[:, None]
                got, want = mine[b, i, :n8].double().cpu().numpy() * s, want[:n8]
                # e4m3's half step, and bf16's before it; below the smallest
                # normal value a half step of 2^-10 scales
                assert np.all(np.abs(got - want) <= np.abs(want) * (2.0 ** -4 + 2 * U) + 2.0 ** -10 * s)
    assert min(len(s) for s in runs[0]) >= 64            # blocks were moved, the ring turned over
