"""The calls of several sequences on the GPU, at the edges of what they promise:
equal calls, values that are not finite, scales far apart, the ends of fp32."""

import numpy as np
import pytest
import torch

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
