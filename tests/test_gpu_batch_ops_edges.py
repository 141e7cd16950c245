"""The calls of several sequences on the GPU, at the edges of what they promise:
equal calls, values that are not finite, scales far apart, the ends of fp32."""

from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import batch as O

pytestmark = pytest.mark.gpu

U = 2.0 ** -8                          # half a bf16 step, relative to the value
NAN = float("nan")


@pytest.fixture(scope="module")
def ops():
    import __graft_entry__ as g
    g.build()
    import self_speculative_decoding_gb300 as ssd
    return ssd.ops


def whole(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# --------------------------------------------------------------------------
# buffers side by side


@pytest.mark.parametrize("name", ["lengths", "counts", "positions", "q_gain", "k_gain", "qkv"])
@pytest.mark.parametrize("next_to", ["out", "k", "v"])
def test_rope_append_inputs_that_end_where_outputs_begin(ops, name, next_to):
    B, T, H, Hkv, dh, rows = 4, 160, 2, 1, 64, 160
    g = torch.Generator(device="cuda").manual_seed(3)

    def inputs():
        g.manual_seed(3)
        return dict(qkv=torch.randn(B, T, (H + 2 * Hkv) * dh, generator=g, device="cuda"), lengths=whole([3, 0, 200, 7]),
                    k=torch.zeros(B, Hkv, rows, dh, device="cuda").bfloat16(),
                    v=torch.zeros(B, Hkv, rows, dh, device="cuda").bfloat16(), counts=whole([160, 0, 5, 31]),
                    positions=whole([9, 8, 7, 6]), q_gain=torch.rand(dh, generator=g, device="cuda") + 0.5,
                    k_gain=torch.rand(dh, generator=g, device="cuda") + 0.5,
                    out=torch.zeros(B, T, H, dh, device="cuda").bfloat16())

    def call(a):
        return ops.rope_append(a["qkv"], a["lengths"], a["k"], a["v"], H, Hkv, dh, 1e4, a["q_gain"], a["k_gain"],
                               counts=a["counts"], positions=a["positions"], out=a["out"])

    want, a = inputs(), inputs()
    call(want)
    # the two in one buffer, the output right behind the input
    x, y = a[name], a[next_to]
    nx, ny = x.numel() * x.element_size(), y.numel() * y.element_size()
    assert nx % 16 == 0
    buf = torch.zeros(nx + ny, dtype=torch.uint8, device="cuda")
    a[name] = buf[:nx].view(x.dtype).view(x.shape).copy_(x)
    a[next_to] = buf[nx:].view(y.dtype).view(y.shape).copy_(y)
    call(a)
    for k in want:
        assert torch.equal(a[k], want[k]), k


def test_all_caches_of_a_sequence_in_one_piece(ops):
    # k, v, their 8-bit rows and scales of each sequence one behind the other
    B, T, H, Hkv, dh, rows, max_seq, block = 3, 90, 6, 2, 64, 128, 256, 32
    g = torch.Generator(device="cuda").manual_seed(4)
    qkv = torch.randn(B, T, (H + 2 * Hkv) * dh, generator=g, device="cuda")
    parts = [("k", torch.bfloat16, (Hkv, rows, dh)), ("v", torch.bfloat16, (Hkv, rows, dh)),
             ("k8", torch.float8_e4m3fn, (Hkv, max_seq, dh)), ("v8", torch.float8_e4m3fn, (Hkv, max_seq, dh)),
             ("ks", torch.float32, (Hkv, max_seq // block)), ("vs", torch.float32, (Hkv, max_seq // block))]
    sizes = [torch.empty(0, dtype=t).element_size() * int(np.prod(shape)) for _, t, shape in parts]
    piece = torch.zeros(B, sum(sizes), dtype=torch.uint8, device="cuda")
    one = {n: x.view(t).view(B, *shape) for (n, t, shape), x in zip(parts, piece.split(sizes, 1))}
    apart = {n: torch.zeros(B, *shape, device="cuda").to(t) for n, t, shape in parts}

    def run(c):
        start = whole([0, 7, 30])
        q = ops.rope_append(qkv, start, c["k"], c["v"], H, Hkv, dh, 1e4)
        held = ops.cache_quantize(c["k"], c["v"], whole([0, 0, 0]), start + T, c["k8"], c["v8"], c["ks"], c["vs"])
        out = ops.cache_attention(q[:, -3:].contiguous(), c["k"], c["v"], start + T - 3, c["k8"], c["v8"], c["ks"], c["vs"], held)
        return q, held, out, *(x.contiguous().view(torch.uint8) for x in c.values())

    for x, y in zip(run(one), run(apart)):
        assert torch.equal(x, y)
    # in each other's way they are refused
    bad = dict(one, k8=piece[:, 16:16 + sizes[2]].view(torch.float8_e4m3fn).view(B, Hkv, max_seq, dh))
    with pytest.raises((ValueError, RuntimeError)):
        ops.cache_quantize(bad["k"], bad["v"], whole([0, 0, 0]), whole([90] * 3), bad["k8"], bad["v8"], bad["ks"], bad["vs"])


# --------------------------------------------------------------------------
# rotation


@pytest.mark.parametrize("H,Hkv,dh", [(40, 4, 128), (7, 3, 64)])
@pytest.mark.parametrize("norms", [False, True])
def test_rope_append_of_many_tokens_gives_each_token_alone(ops, H, Hkv, dh, norms):
    # calls of few and of many tokens go by different grains
    B, T = 3, 400
    g = torch.Generator(device="cuda").manual_seed(dh)
    qkv = torch.randn(B, T, (H + 2 * Hkv) * dh, generator=g, device="cuda")
    gains = [torch.rand(dh, generator=g, device="cuda") + 0.5 for _ in range(2)] if norms else [None, None]
    k, v, k1, v1 = (torch.zeros(B, Hkv, 1000, dh, device="cuda").bfloat16() for _ in range(4))
    start = whole([0, 131, 600])
    q = ops.rope_append(qkv, start, k, v, H, Hkv, dh, 1e4, *gains)
    lone = [ops.rope_append(qkv[:, t:t + 1].contiguous(), start + t, k1, v1, H, Hkv, dh, 1e4, *gains) for t in range(T)]
    assert torch.equal(torch.cat(lone, 1).view(torch.int16), q.view(torch.int16))
    assert torch.equal(k1, k) and torch.equal(v1, v)


# --------------------------------------------------------------------------
# verification


@pytest.mark.parametrize("B,d,V,given", [(1, 4, 1024, True), (16, 3, 32000, False), (48, 2, 128003, True),
                                         (300, 1, 5000, True)])
def test_verify_drafts_says_the_same_every_time(ops, B, d, V, given):
    # the search in the CTA that has the token must not disturb the choice of that CTA
    g = torch.Generator(device="cuda").manual_seed(V)
    p = torch.softmax(torch.randn(B, d + 1, V, generator=g, device="cuda") * 2, -1)
    q = torch.softmax(torch.randn(B, d, V, generator=g, device="cuda") * 2, -1) if given else None
    drafts = torch.randint(0, V, (B, d), generator=g, device="cuda", dtype=torch.int32)
    au = torch.full((B, d), 0.999, device="cuda")
    su = torch.rand(B, generator=g, device="cuda")
    y = drafts[:, :1].long()
    rest = p[:, 0].double() - (q[:, 0].double() if given else 0.0)
    if not given:
        rest.scatter_(1, y, 0.0)
    part = rest.clamp(min=0.0).cumsum(1)
    sure = au[:, 0].double() * (q[:, 0].gather(1, y)[:, 0].double() if given else 1.0)
    out = ~(sure < p[:, 0].gather(1, y)[:, 0].double())          # the first draft is rejected
    want = (part > su.double()[:, None] * part[:, -1:]).int().argmax(1).int()
    first = ops.verify_drafts(p, drafts, au, su, q=q)
    assert torch.equal(first[0][out, 0], want[out])
    same = torch.ones((), dtype=torch.bool, device="cuda")
    for _ in range(200):
        for a, b in zip(ops.verify_drafts(p, drafts, au, su, q=q), first):
            same &= (a == b).all()
    assert same.item()


@pytest.mark.parametrize("e", [-149, -130, -100, 0, 70, 100, 118])
def test_verify_drafts_of_weights_of_any_size(ops, e):
    # weights that sum to anything: what is accepted and drawn depends on their ratios; with
    # e = 118 every row sums to more than fp32 holds, and nothing is drawn
    B, d, V = 64, 3, 50
    rng = np.random.default_rng(e + 200)
    scale = 2.0 ** e
    p = np.ldexp(rng.integers(1, 1 << 9, (B, d + 1, V)).astype(np.float32), e)
    q = np.ldexp(rng.integers(1, 1 << 9, (B, d, V)).astype(np.float32), e)
    drafts = rng.integers(0, V, (B, d))
    au, su = rng.random((B, d)).astype(np.float32), rng.random(B).astype(np.float32)
    # ties: u q = p exactly, and one step below
    for b in range(0, B, 4):
        q[b, 0], p[b, 0] = np.float32(scale * 256), np.float32(scale * 128)
        au[b, 0] = 0.5 if b % 8 else np.nextafter(np.float32(0.5), np.float32(0))
    on = lambda x, t: torch.from_numpy(np.ascontiguousarray(x)).to(t).cuda()  # noqa: E731
    tokens, n = ops.verify_drafts(on(p, torch.float32), on(drafts, torch.int32), on(au, torch.float32),
                                  on(su, torch.float32), q=on(q, torch.float32))
    for b in range(B):
        want = O.verify(p[b].astype(np.float64), q[b].astype(np.float64), drafts[b], au[b].astype(np.float64), float(su[b]))
        want = want[:-1] if e == 118 else want
        assert tokens[b].tolist() == want + [-1] * (d + 1 - len(want)), b
        assert n[b].item() == len(want)


@pytest.mark.parametrize("V", [40, 3000, 40000])
@pytest.mark.parametrize("u", [-1e-30, -0.5, -0.0, float("-inf"), NAN])
def test_verify_drafts_below_the_range(ops, V, u):
    # as 0: the first entry over 0, wherever it lies
    p = torch.zeros(6, 1, V, device="cuda")
    at = [0, 1, V // 3, V // 2, V - 2, V - 1]
    for b, v in enumerate(at):
        p[b, 0, v:] = torch.rand(V - v, device="cuda") + 0.1
    tokens, n = ops.verify_drafts(p, torch.zeros(6, 0, dtype=torch.int32, device="cuda"), torch.zeros(6, 0, device="cuda"),
                                  torch.full((6,), u, device="cuda"))
    assert tokens[:, 0].tolist() == at and n.tolist() == [1] * 6


def stubborn_entries(n, seed):
    """n fp32 entries whose sum in order, with the rounding errors added up in
    fp32, is off by some 2^-35 always to the same side."""
    f, rng = np.float32, np.random.default_rng(seed)
    some = (f(2.0 ** -20) * (1 + rng.integers(0, 1 << 23, 512) / f(1 << 23))).astype(f)
    s, c, entries = f(1), f(0), [f(1)]
    for _ in range(n - 1):
        t = (s + some).astype(f)
        part = (t - s).astype(f)
        err = ((s - (t - part).astype(f)).astype(f) + (some - part).astype(f)).astype(f)
        now = (c + err).astype(f)
        k = int(np.argmax(now.astype(np.float64) - (np.float64(c) + err.astype(np.float64))))
        entries.append(some[k])
        s, c = t[k], now[k]
    return np.array(entries, f), float(s) + float(c)


@pytest.mark.parametrize("B", [1, 512])
def test_verify_drafts_sums_many_entries(ops, B):
    # a border as near to U sum p as 2^-36 of it: one CTA's 16 runs of 8000 entries, a
    # lane's every 32nd; the runs of the second half sum to 256 times `lane`
    V, n = 128000, 250
    lane, by_fp32 = stubborn_entries(n, 5)
    half = [Fraction(float(x)) for x in lane]
    true = 256 * sum(half)
    off = 256 * (Fraction(by_fp32) - sum(half))
    assert abs(off) > 2.0 ** -36 * true
    p = np.zeros(V, np.float32)
    p[V // 2:] = np.repeat(lane, 32)[None].repeat(8, 0).reshape(-1)
    # the first half: the same sum and half of what fp32 is off by, in a few entries
    left, at = true + off / 2, 0
    while left > true * Fraction(1, 2 ** 44):
        p[at] = np.float32(np.nextafter(np.float32(left), np.float32(0)))
        left -= Fraction(float(p[at]))
        at += 1
    first = sum(Fraction(float(x)) for x in p[:at])
    want = at - 1 if first > (first + true) / 2 else V // 2
    tokens, count = ops.verify_drafts(torch.from_numpy(p).cuda().expand(B, 1, V).contiguous(),
                                      torch.zeros(B, 0, dtype=torch.int32, device="cuda"), torch.zeros(B, 0, device="cuda"),
                                      torch.full((B,), 0.5, device="cuda"))
    assert (count == 1).all().item() and (tokens == want).all().item(), (tokens[0].item(), want)


# --------------------------------------------------------------------------
# attention: values that are not finite, which some tokens see


def caches(g, B, Hkv, dh, rows, max_seq, block):
    """Seeded bf16 rings and 8-bit caches with scales."""
    k, v = (torch.randn(B, Hkv, rows, dh, generator=g, device="cuda").bfloat16() for _ in range(2))
    k8, v8 = ((torch.randn(B, Hkv, max_seq, dh, generator=g, device="cuda") * 90).clamp_(-448, 448).to(torch.float8_e4m3fn)
              for _ in range(2))
    ks, vs = (torch.rand(B, Hkv, max_seq // block, generator=g, device="cuda") / 90 + 0.004 for _ in range(2))
    return k, v, dict(k8=k8, v8=v8, k_scale=ks, v_scale=vs)


@pytest.mark.parametrize("what", [NAN, float("inf"), float("-inf")])
@pytest.mark.parametrize("T,G", [(2, 1), (3, 1), (4, 1), (2, 2), (4, 2), (3, 5)])
@pytest.mark.parametrize("B,Hkv,n,held,window", [
    (64, 8, 20, 0, 0),             # pairs of one tile, several of a CTA: either group's
    (1, 2, 250, 0, 0),             # the drafted rows in the second tile of two
    (2, 3, 509, 480, 0),           # in the fourth and fifth
    (40, 5, 300, 288, 280),        # rows that leave the window as well
])
def test_values_that_some_tokens_see_reach_them(ops, B, Hkv, n, held, window, T, G, what):
    dh, block = 64, 32
    g = torch.Generator(device="cuda").manual_seed(T * 10 + G)
    k, v, kw = caches(g, B, Hkv, dh, 512, 512, block)
    q = torch.randn(B, T, Hkv * G, dh, generator=g, device="cuda").bfloat16()
    kw["held"] = whole([held] * B)

    def run():
        return ops.cache_attention(q, k, v, whole([n] * B), window=window, **kw)

    clean = run()
    assert torch.isfinite(clean).all()
    rng = np.random.default_rng(T)
    v_was, e, e_was = v.clone(), kw["v8"].view(torch.uint8), kw["v8"].view(torch.uint8).clone()
    low = max(0, n + 1 - window) if window else 0
    for share in (0.02, 0.3, 1.0):               # of the pairs
        for row in [n + T - 1, n + 1] + ([low, low + T - 2] if window else []):
            hit = torch.from_numpy(rng.random((B, Hkv)) < share).cuda()
            v.copy_(v_was)
            e.copy_(e_was)
            if row >= held:
                at = row % 512
                v[:, :, at, 7] = torch.where(hit, torch.full_like(v[:, :, at, 7], what), v[:, :, at, 7])
            else:
                e[:, :, row, 7] = torch.where(hit, torch.full_like(e[:, :, row, 7], 0x7F), e[:, :, row, 7])
            out = run()
            pos = n + torch.arange(T, device="cuda")
            sees = (row <= pos) & ((row > pos - window) if window else True)
            lost = hit.repeat_interleave(G, 1)[:, None] & sees[None, :, None]        # [B, T, H]
            assert not torch.isfinite(out[..., 7][lost]).any(), (share, row)
            assert torch.equal(out[..., 7][~lost], clean[..., 7][~lost])
            cols = [i for i in range(dh) if i != 7]
            assert torch.equal(out[..., cols], clean[..., cols])


@pytest.mark.parametrize("T,G", [(2, 1), (3, 4), (3, 9), (9, 8)])
@pytest.mark.parametrize("B", [1, 90])
def test_a_zero_keeps_its_sign_beside_them(ops, B, T, G):
    # results that round to -0 stay -0 where other columns hold NaN
    Hkv, dh, n = 2, 64, 300
    g = torch.Generator(device="cuda").manual_seed(T)
    k, v = (torch.randn(B, Hkv, 384, dh, generator=g, device="cuda").bfloat16() for _ in range(2))
    v[..., 5] = -2.0 ** -133
    v[:, :, :n - 1, 5] = 0.0
    q = torch.randn(B, T, Hkv * G, dh, generator=g, device="cuda").bfloat16()
    clean = ops.cache_attention(q, k, v, whole([n] * B))
    v[:, :, n + T - 1, 7] = NAN                      # the last token's own
    out = ops.cache_attention(q, k, v, whole([n] * B))
    cols = [i for i in range(dh) if i != 7]
    assert torch.equal(out[..., cols].view(torch.int16), clean[..., cols].view(torch.int16))
    assert (clean[..., 5].view(torch.int16) == -32768).any().item()

# --------------------------------------------------------------------------
# attention: value scales far apart


def exact_rows(q, K, S, V8, length, scale, window=0):
    """One sequence in 64 bits: q [T, H, dh], K [Hkv, n, dh] values, V = S[..., None] *
    V8 -> the result, sum p |v|, and the largest p s of each row."""
    T, H, dh = q.shape
    Hkv, n = K.shape[:2]
    x = q.double().view(T, Hkv, H // Hkv, dh).permute(1, 2, 0, 3)
    s = scale * (x @ K[:, None].transpose(2, 3))
    j, pos = torch.arange(n, device="cuda"), length + torch.arange(T, device="cuda")[:, None]
    hidden = (j > pos) | ((j <= pos - window) if window else False)
    p = torch.softmax(s.masked_fill(hidden, -float("inf")), -1)
    back = lambda t: t.permute(2, 0, 1, 3).reshape(T, H, -1)  # noqa: E731
    V = S[..., None] * V8
    return back(p @ V[:, None]), back(p @ V.abs()[:, None]), back((p * S.abs()[:, None, None]).amax(-1, keepdim=True))


def check_scales(ops, q, k8, v8, ks, vs, n, held, k, v, window=0, scale=None):
    """The call against 64 bits.  Off by: the result's own rounding U |o|; each weight's
    in fp16, 2^-11 of it, or (below 2^-18 of the largest) half a step of 2^-28 of the
    largest; bf16 rows' weights U; scores 2^-16 with values of this size, a factor of
    2^-15 on a probability and its sum."""
    B, T, H, dh = q.shape
    block = k8.shape[2] // ks.shape[2]
    out = ops.cache_attention(q, k, v, whole([n] * B), k8=k8, v8=v8, k_scale=ks, v_scale=vs, held=whole([held] * B),
                              window=window, scale=scale).double()
    for b in range(0, B, max(1, B // 5)):
        ring = torch.arange(held, n + T, device="cuda") % k.shape[2]
        each = lambda s: s[b].double().repeat_interleave(block, 1)[:, :held]  # noqa: E731
        K = torch.cat((k8[b, :, :held].double() * each(ks)[..., None], k[b, :, ring].double()), 1)
        V8 = torch.cat((v8[b, :, :held].double(), v[b, :, ring].double()), 1)
        S = torch.cat((each(vs), torch.ones_like(K[:, held:, 0])), 1)
        ref, spread, most = exact_rows(q[b], K, S, V8, n, dh ** -0.5 if scale is None else scale, window)
        tol = U * ref.abs() + (2.0 ** -11 + 2.0 ** -14 + (U if held < n + T else 0.0)) * spread + (
            (n + T) * 2.0 ** -29 * most * V8.abs().amax())
        off = (out[b] - ref).abs() / (tol + 1e-37)
        assert (off <= 1).all().item(), (b, off.max().item())


ROWS = [(1, 1), (2, 2), (3, 4), (5, 3), (7, 4), (9, 8)]          # tokens, query heads a K/V head
PAIRS = [(3, 2), (40, 5)]              # sequences, heads: a CTA for each tile or so; all of a pair's tiles in one


@pytest.mark.parametrize("B,Hkv", PAIRS)
@pytest.mark.parametrize("T,G", ROWS)
@pytest.mark.parametrize("heavy", ["first", "last", "middle"])
@pytest.mark.parametrize("apart", [-38, -30, -12, 12, 30, 38])
def test_weight_on_blocks_of_another_scale(ops, B, Hkv, T, G, heavy, apart):
    # all the weight lies in one block whose value scale is 2^apart of the others'
    dh, block, n = 64, 32, 1500
    g = torch.Generator(device="cuda").manual_seed(abs(apart) + T)
    held = (n + T) // block * block
    k, v = (torch.randn(B, Hkv, 128, dh, generator=g, device="cuda").bfloat16() for _ in range(2))
    k8 = torch.randn(B, Hkv, held, dh, generator=g, device="cuda").mul_(0.5)
    v8 = torch.randn(B, Hkv, held, dh, generator=g, device="cuda").mul_(90).clamp_(-448, 448).to(torch.float8_e4m3fn)
    at = {"first": 0, "middle": held // block // 2, "last": held // block - 2}[heavy]
    k8[..., 0] = -30.0                               # scores far below the block's
    k8[:, :, at * block:(at + 1) * block, 0] = 30.0
    k[..., 0] = -30.0
    q = torch.randn(B, T, Hkv * G, dh, generator=g, device="cuda")
    q[..., 0] = 8.0
    ks = torch.ones(B, Hkv, held // block, device="cuda")
    vs = torch.full((B, Hkv, held // block), 0.01, device="cuda")
    vs[:, :, at] = 0.013 * 2.0 ** apart
    v.mul_(1e-30)
    check_scales(ops, q.bfloat16(), k8.to(torch.float8_e4m3fn), v8, ks, vs, n, held, k, v)


@pytest.mark.parametrize("B,Hkv", PAIRS)
@pytest.mark.parametrize("T,G", ROWS)
@pytest.mark.parametrize("e", [3, 12, 19])
@pytest.mark.parametrize("lengths", [40, 700, 5000])
def test_scales_at_random(ops, B, Hkv, T, G, e, lengths):
    dh, block = 128, 64
    g = torch.Generator(device="cuda").manual_seed(e + T)
    held = lengths // block * block
    max_seq = max(block, held)
    k, v = (torch.randn(B, Hkv, 256, dh, generator=g, device="cuda").bfloat16() for _ in range(2))
    k8, v8 = (torch.randn(B, Hkv, max_seq, dh, generator=g, device="cuda").mul_(a).clamp_(-448, 448).to(torch.float8_e4m3fn)
              for a in (1.0, 90.0))
    ks = torch.ones(B, Hkv, max_seq // block, device="cuda")
    vs = torch.exp2(torch.randint(-e, e + 1, ks.shape, generator=g, device="cuda").float()) * (
        1.0 + torch.rand(ks.shape, generator=g, device="cuda"))
    q = torch.randn(B, T, Hkv * G, dh, generator=g, device="cuda").mul_(2.0).bfloat16()
    check_scales(ops, q, k8, v8, ks, vs, lengths, held, k, v)
    if held:
        check_scales(ops, q, k8, v8, ks, vs, held - T, held, k, v)


@pytest.mark.parametrize("T,G", [(1, 2), (2, 8), (9, 8)])
@pytest.mark.parametrize("large", ["first", "last"])
def test_a_tail_of_small_weights_beside_a_large_scale(ops, T, G, large):
    # a block of scale 1 without weight; the others 2^12 below, one key of which takes
    # most, and the rest (12 below it) a tenth of that in all: none may be lost
    n, dh, block = 20000, 64, 32
    held = n + T + block - (n + T) % block
    k8 = torch.zeros(1, 1, held, dh, device="cuda")
    at = 0 if large == "first" else (n // block - 1)
    k8[:, :, at * block:(at + 1) * block, 0] = -12.0
    k8[:, :, 64, 0] = 12.0
    v8 = torch.zeros_like(k8)
    v8[..., 1] = 1.0
    v8[:, :, 64, 1] = 0.0
    v8[:, :, at * block:(at + 1) * block, 1] = 448.0
    ks = torch.ones(1, 1, held // block, device="cuda")
    vs = torch.full_like(ks, 2.0 ** -12)
    vs[:, :, at] = 1.0
    q = torch.zeros(1, T, G, dh, device="cuda").bfloat16()
    q[..., 0] = 8.0
    ring = torch.zeros(1, 1, 128, dh, device="cuda").bfloat16()
    out = ops.cache_attention(q, ring, ring, whole([n]), k8=k8.to(torch.float8_e4m3fn), v8=v8.to(torch.float8_e4m3fn),
                              k_scale=ks, v_scale=vs, held=whole([n]))
    # (rows n .. are the ring's: scores and values of 0)
    for t in range(T):
        tail = n - 1 - block
        total = 1 + (tail + t + 1) * np.exp(-12.0) + block * np.exp(-24.0)
        want = 2.0 ** -12 * tail * np.exp(-12.0) / total + 448 * block * np.exp(-24.0) / total
        off = (out[0, t, :, 1].double() - want).abs().max().item() / want
        assert off <= 3 * U


@pytest.mark.parametrize("T,G", [(1, 2), (2, 8), (3, 10), (9, 8)])
@pytest.mark.parametrize("dh", [64, 128])
@pytest.mark.parametrize("at", [0, 3, 300])
def test_a_block_of_zeros_takes_the_weight(ops, T, G, dh, at):
    # zeros, whose scale is 1, take nearly all the weight; the rows beside them, whose
    # scale is 2^-12, have e^-12 each, and are the result
    n, block = 20000, 64
    held = n + T + block - (n + T) % block
    k8 = torch.zeros(1, 1, held, dh, device="cuda")
    k8[:, :, at * block:(at + 1) * block, 0] = 12.0
    v8 = torch.zeros_like(k8)
    v8[..., 1] = 1.0
    v8[:, :, at * block:(at + 1) * block] = 0.0
    v8[:, :, at * block:(at + 1) * block, 5] = -0.0
    ks = torch.ones(1, 1, held // block, device="cuda")
    vs = torch.full_like(ks, 2.0 ** -12)
    vs[:, :, at] = 1.0
    q = torch.zeros(1, T, G, dh, device="cuda").bfloat16()
    q[..., 0] = 8.0
    ring = torch.zeros(1, 1, 128, dh, device="cuda").bfloat16()
    out = ops.cache_attention(q, ring, ring, whole([n]), k8=k8.to(torch.float8_e4m3fn), v8=v8.to(torch.float8_e4m3fn),
                              k_scale=ks, v_scale=vs, held=whole([n // block * block]), scale=0.125)
    far = n // block * block                     # (rows from there on are the ring's: scores and values of 0)
    for t in range(T):
        tail = far - block
        total = block + (n + t + 1 - block) * np.exp(-12.0)
        want = 2.0 ** -12 * tail * np.exp(-12.0) / total
        off = (out[0, t, :, 1].double() - want).abs().max().item() / want
        assert off <= 3 * U and not out[0, t, :, 2:].any().item()


@pytest.mark.parametrize("B,Hkv", PAIRS)
@pytest.mark.parametrize("T,G", [(2, 1), (4, 2), (4, 4), (6, 5), (9, 8)])
def test_a_large_scale_that_some_tokens_see(ops, B, Hkv, T, G):
    # a block of large scale leaves the window token by token
    dh, block, n, window = 64, 32, 1000, 601
    g = torch.Generator(device="cuda").manual_seed(T)
    held = 960
    k, v = (torch.randn(B, Hkv, 256, dh, generator=g, device="cuda").bfloat16() for _ in range(2))
    k8, v8 = (torch.randn(B, Hkv, held, dh, generator=g, device="cuda").mul_(a).clamp_(-448, 448).to(torch.float8_e4m3fn)
              for a in (1.0, 90.0))
    ks = torch.ones(B, Hkv, held // block, device="cuda")
    vs = torch.full_like(ks, 0.01)
    low = n + 1 - window                             # 400: the first token's first row
    vs[:, :, low // block] = 2.0 ** 30
    q = torch.randn(B, T, Hkv * G, dh, generator=g, device="cuda").bfloat16()
    v8.view(torch.uint8)[:, :, low + T:(low // block + 1) * block] = 0
    check_scales(ops, q, k8, v8, ks, vs, n, held, k, v, window=window)


@pytest.mark.parametrize("T,G", [(1, 4), (2, 6), (3, 9), (4, 7), (5, 12)])
@pytest.mark.parametrize("first", [2.0 ** -86, 2.0 ** -100, 2.0 ** -126])
def test_means_of_many_rows_of_tiny_scales(ops, T, G, first):
    # more pairs than SMs: each is one CTA's, and its sums are divided there
    B, Hkv, dh, block, n = 20, 9, 64, 64, 4096     # (e^-128 2^40 is far below 2^-28)
    g = torch.Generator(device="cuda").manual_seed(T)
    k8 = torch.zeros(B, Hkv, n, dh, device="cuda").to(torch.float8_e4m3fn)
    v8 = (torch.rand(B, Hkv, n, dh, generator=g, device="cuda") * 400 + 40).to(torch.float8_e4m3fn)
    k8.view(torch.uint8)[:, :, :block] = 0xD8                    # -16 x 64: no weight
    ks = torch.ones(B, Hkv, n // block, device="cuda")
    vs = torch.full_like(ks, 2.0 ** -126)
    vs[:, :, 0] = first
    q = torch.ones(B, T, Hkv * G, dh, device="cuda").bfloat16()
    ring = torch.full((B, Hkv, 128, dh), NAN, device="cuda").bfloat16()
    out = ops.cache_attention(q, ring, ring, whole([n - T] * B), k8=k8, v8=v8, k_scale=ks, v_scale=vs,
                              held=whole([n] * B)).double()
    for t in range(T):
        m = n - T + 1 + t
        want = (v8[:, :, block:m].float().double().sum(2) / (m - block) * 2.0 ** -126).repeat_interleave(G, 1)
        off = ((out[:, t] - want).abs() / want).max().item()
        assert off <= U + 2.0 ** -10


@pytest.mark.parametrize("B,Hkv", PAIRS)
@pytest.mark.parametrize("T,G", ROWS)
@pytest.mark.parametrize("e", [-126, -115, -90, -60, -40, -25, -20])
@pytest.mark.parametrize("n", [150, 900])
def test_bf16_rows_behind_tiny_scales(ops, B, Hkv, T, G, e, n):
    dh, block = 64, 64
    g = torch.Generator(device="cuda").manual_seed(T - e)
    held = (n - 70) // block * block
    k, v = (torch.randn(B, Hkv, 256, dh, generator=g, device="cuda").bfloat16() for _ in range(2))
    k8, v8 = (torch.randn(B, Hkv, held, dh, generator=g, device="cuda").mul_(a).clamp_(-448, 448).to(torch.float8_e4m3fn)
              for a in (1.0, 90.0))
    ks = torch.ones(B, Hkv, held // block, device="cuda")
    vs = torch.full_like(ks, 2.0 ** e)
    q = torch.randn(B, T, Hkv * G, dh, generator=g, device="cuda").bfloat16()
    check_scales(ops, q, k8, v8, ks, vs, n, held, k, v)
    # and larger ones than usual; and as tiny as the others
    check_scales(ops, q, k8, v8, ks, vs, n, held, k, v * 2.0 ** 40)
    v = v * 2.0 ** max(e + 6, -100)
    check_scales(ops, q, k8, v8, ks, vs, n, held, k, v)


@pytest.mark.parametrize("T,G", ROWS)
def test_large_values_of_bf16_rows_alone(ops, T, G):
    # 2^11 times their sum is below 2^127
    B, Hkv, dh, n = 2, 2, 64, 1000
    g = torch.Generator(device="cuda").manual_seed(T)
    k, v = (torch.randn(B, Hkv, 1024, dh, generator=g, device="cuda") for _ in range(2))
    q = torch.randn(B, T, Hkv * G, dh, generator=g, device="cuda").bfloat16()
    k, v = k.bfloat16(), v.bfloat16()
    want = ops.cache_attention(q, k, v, whole([n] * B))
    out = ops.cache_attention(q, k, v * 2.0 ** 105, whole([n] * B))
    assert torch.equal(out, want * 2.0 ** 105)


# --------------------------------------------------------------------------
# queries that are not finite


@pytest.mark.parametrize("T,G", ROWS)
@pytest.mark.parametrize("n,held", [(0, None), (5, None), (900, None), (900, 0), (900, 832)])
def test_queries_that_are_not_finite_are_nan(ops, T, G, n, held):
    B, Hkv, dh, block = 40, 5, 64, 64
    g = torch.Generator(device="cuda").manual_seed(T + n)
    k, v, kw = caches(g, B, Hkv, dh, 1024, 1024, block)
    kw = {} if held is None else dict(kw, held=whole([held] * B))
    q = torch.randn(B, T, Hkv * G, dh, generator=g, device="cuda").bfloat16()
    clean = ops.cache_attention(q, k, v, whole([n] * B), **kw)
    rng = np.random.default_rng(T + n)
    for what in (float("inf"), float("-inf"), NAN):
        hit = torch.from_numpy(rng.random((B, T, Hkv * G)) < 0.3).cuda()
        bad = q.clone()
        bad[..., 11] = torch.where(hit, torch.full_like(q[..., 11], what), q[..., 11])
        for scale in (0.125, -0.125):
            out = ops.cache_attention(bad, k, v, whole([n] * B), scale=scale, **kw)
            assert torch.isnan(out[hit]).all()
            assert torch.isfinite(out[~hit]).all()
            if scale > 0:
                assert torch.equal(out[~hit], clean[~hit])


# --------------------------------------------------------------------------
# attention at random: odd lengths, any number of 8-bit rows, windows, rings, counts


def seen_mask(length, T, n, window, sinks):
    j, pos = torch.arange(n, device="cuda"), length + torch.arange(T, device="cuda")[:, None]
    seen = j <= pos
    return seen & ((j < sinks) | (j > pos - window)) if window else seen


@pytest.mark.parametrize("seed", range(60))
def test_attention_at_random(ops, seed):
    rng = np.random.default_rng(1000 + seed)
    pick = lambda *x: x[rng.integers(len(x))]  # noqa: E731
    dh, block = int(pick(64, 128)), int(pick(32, 64, 128))
    G = int(pick(1, 1, 2, 3, 4, 5, 8, 16))
    T = int(rng.integers(1, max(2, min(17, 128 // G + 1))))
    Hkv, B = int(pick(1, 2, 3, 5)), int(pick(1, 2, 3, 7, 40, 90))
    most = int(pick(3, 60, 300, 1500, 4000))
    lengths = rng.integers(0, most + 1, B)
    counts = rng.integers(0, T + 1, B) if seed % 3 else np.full(B, T)
    window = int(pick(0, 0, 1, 17, 130, 1000))
    sinks = int(rng.integers(0, 300)) if window and seed % 2 else int(pick(0, 3))
    ends = lengths + counts
    tail = rng.integers(0, 200, B)
    held = np.maximum(ends - tail, 0) if seed % 4 else np.maximum(lengths - tail, 0) // block * block
    # a ring that holds what is in bf16, or rows for the longest
    need = int(np.maximum(ends - held, 1).max())
    rows = -(-need // 128) * 128 if seed % 2 else max(int(ends.max()), 1)
    max_seq = -(-max(int(held.max()), 1) // block) * block
    g = torch.Generator(device="cuda").manual_seed(seed)
    std = float(pick(0.5, 1.5, 4.0))
    q = (torch.randn(B, T, Hkv * G, dh, generator=g, device="cuda") * std).bfloat16()
    k, v, kw = caches(g, B, Hkv, dh, rows, max_seq, block)
    out = ops.cache_attention(q, k, v, whole(lengths.tolist()), held=whole(held.tolist()), counts=whole(counts.tolist()),
                              window=window, sinks=sinks, **kw)
    again = ops.cache_attention(q, k, v, whole(lengths.tolist()), held=whole(held.tolist()), counts=whole(counts.tolist()),
                                window=window, sinks=sinks, **kw)
    assert torch.equal(out, again)
    out = out.double()
    for b in range(0, B, max(1, B // 7)):
        n, c, h = int(lengths[b]), int(counts[b]), int(held[b])
        assert not out[b, c:].any().item()
        if not c:
            continue
        at = torch.arange(h, n + c, device="cuda") % rows
        each = lambda s: s[b].double().repeat_interleave(block, 1)[:, :h, None]  # noqa: E731
        K, V = (torch.cat((kw[x + "8"][b, :, :h].double() * each(kw[x + "_scale"]), r[b, :, at].double()), 1)
                for x, r in (("k", k), ("v", v)))
        x = q[b, :c].double().view(c, Hkv, G, dh).permute(1, 2, 0, 3)
        s = dh ** -0.5 * (x @ K[:, None].transpose(2, 3))
        p = torch.softmax(s.masked_fill(~seen_mask(n, c, n + c, window, sinks), -float("inf")), -1)
        back = lambda t: t.permute(2, 0, 1, 3).reshape(c, Hkv * G, dh)  # noqa: E731
        ref, spread = back(p @ V[:, None]), back(p @ V[:, None].abs())
        # (as the tolerance of check_scales: U for a bf16 row's weight; a score's error, doubled)
        d = dh ** -0.5 * (2.0 ** -17 * x.abs().amax() * K.abs().sum(-1).amax() +
                          2 * dh * 2.0 ** -24 * (x.abs() @ K[:, None].abs().transpose(2, 3)).amax()) + 1e-6
        off = (out[b, :c] - ref).abs() / (U * ref.abs() + (U + 2 * d) * spread)
        assert (off <= 1).all().item(), (b, off.max().item())


def test_no_tokens_at_all(ops):
    g = torch.Generator(device="cuda").manual_seed(1)
    k, v, kw = caches(g, 5, 2, 64, 128, 256, 64)
    q = torch.randn(5, 3, 8, 64, generator=g, device="cuda").bfloat16()
    kw["held"] = whole([0, 64, 128, 0, 256])
    out = ops.cache_attention(q, k, v, whole([0, 64, 130, 7, 256]), counts=whole([0] * 5), **kw)
    assert not out.any().item()
    out = ops.rope_append(torch.randn(5, 3, 12 * 64, generator=g, device="cuda"), whole([0] * 5), k, v, 8, 2, 64, 1e4,
                          counts=whole([0] * 5))
    assert not out.any().item()


def test_calls_captured_from_streams_that_meet(ops):
    # rotation on one stream, verification on another, behind a copy and a fill; the
    # attention where the two meet
    B, T, H, Hkv, dh, V = 2, 3, 8, 2, 64, 500
    g = torch.Generator(device="cuda").manual_seed(2)
    k, v, kw = caches(g, B, Hkv, dh, 256, 256, 64)
    kw["held"] = whole([64, 128])
    qkv = torch.randn(B, T, (H + 2 * Hkv) * dh, generator=g, device="cuda")
    p = torch.softmax(torch.randn(B, T + 1, V, generator=g, device="cuda"), -1)
    drafts, au, su = whole([[1, 2, 3], [4, 5, 6]]), torch.zeros(B, T, device="cuda"), torch.rand(B, generator=g, device="cuda")
    lengths, n_in, x_in = whole([100, 140]), whole([100, 140]), qkv.clone()

    def calls(other):
        main = torch.cuda.current_stream()
        lengths.copy_(n_in)
        other.wait_stream(main)
        with torch.cuda.stream(other):
            qkv.copy_(x_in)
            q = ops.rope_append(qkv, lengths, k, v, H, Hkv, dh, 1e4)
        tokens, n = ops.verify_drafts(p, drafts, au, su)
        main.wait_stream(other)
        out = ops.cache_attention(q, k, v, lengths, **kw)
        new = ops.cache_quantize(k, v, kw["held"], lengths + n, kw["k8"].clone(), kw["v8"].clone(), kw["k_scale"].clone(),
                                 kw["v_scale"].clone())
        q.record_stream(main)
        return q, tokens, n, out, new

    other = torch.cuda.Stream()
    want = [x.clone() for x in calls(other)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = calls(other)
    for _ in range(20):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
