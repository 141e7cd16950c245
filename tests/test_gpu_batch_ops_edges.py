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
