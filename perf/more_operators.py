"""Timed cases of the operators of a drafting round over an 8-bit cache.

Four operators of a program that decodes several sequences at once: the norms
of the query and key heads with their rotation, appended to the caches; the
move of committed cache rows to 8 bits with a scale for each block of rows and
head; attention of a few tokens per sequence over such a cache, whole or
through a window with a few first rows that stay visible; and the verification
of drafted tokens from given random numbers.

``listed`` and ``draw`` give cases, ``prepare`` the tensors that a program has
in hand before the call, ``run`` one call: the plain torch form, or the
library's kernels where ``own`` is true.  ``exact`` is the definition in 64
bits and ``work`` the bytes and operations that a call cannot do without.
"""

import math
import random

import torch

own = False

THETA = 1.0e4
EPS = 1.0e-5


# --------------------------------------------------------------------------
# cases


def _rope(name, seqs, tokens, heads, kv_heads, dh, context, norms, ring, short=0):
    c = {"op": "rope", "seqs": seqs, "tokens": tokens, "heads": heads, "kv_heads": kv_heads, "dh": dh,
         "context": context, "norms": norms, "ring": ring, "short": short}
    return dict(c, name=name) if name else c


def _quantize(name, seqs, kv_heads, dh, block, max_seq, context, blocks, ring):
    c = {"op": "quantize", "seqs": seqs, "kv_heads": kv_heads, "dh": dh, "block": block,
         "max_seq": max_seq, "context": context, "blocks": blocks, "ring": ring}
    return dict(c, name=name) if name else c


def _attention(name, seqs, tokens, heads, kv_heads, dh, context, block, recent, ring, window=0, sinks=0,
               short=0, ragged=True):
    c = {"op": "attention", "seqs": seqs, "tokens": tokens, "heads": heads, "kv_heads": kv_heads, "dh": dh,
         "context": context, "block": block, "recent": recent, "ring": ring, "window": window,
         "sinks": sinks, "short": short, "ragged": ragged}
    return dict(c, name=name) if name else c


def _verify(name, seqs, drafts, vocab, agree, given=True, short=0):
    c = {"op": "verify", "seqs": seqs, "drafts": drafts, "vocab": vocab, "agree": agree, "given": given,
         "short": short}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one token of one sequence, grouped heads with norms: the plain decode
        # step, where the call's latency is all there is
        _rope("rope-one-token", 1, 1, 64, 8, 128, 16385, True, 256),
        # the prompts of four sequences, one head's cache per query head
        _rope("rope-prompts", 4, 2016, 40, 40, 128, 0, True, 2048, short=3),
        # a block or two of each of a few sequences of the tiny model
        _quantize("quantize-step", 5, 4, 64, 32, 512, 200, 2, 128),
        # the prompts of eight sequences at once
        _quantize("quantize-prompts", 8, 8, 128, 64, 16384, 0, 256, 16384),
        # the tiny model's verify: five tokens behind a short prompt
        _attention("attention-tiny", 1, 5, 4, 4, 64, 83, 32, 16, 128),
        # a draft step through a window of a long cache with four first rows
        _attention("attention-window", 1, 1, 64, 8, 128, 131000, 64, 128, 256, window=1023, sinks=4),
        # the plain decode step behind a long context
        _attention("attention-one-token", 1, 1, 64, 8, 128, 131000, 64, 128, 256),
        # a verify pass of eight drafts of sixteen sequences of uneven lengths,
        # some of which drafted less
        _attention("attention-verify", 16, 9, 64, 8, 128, 16385, 64, 64, 256, short=4),
        # one head's cache per query head, two tokens each, a window as well
        _attention("attention-mha", 8, 2, 40, 40, 128, 4095, 128, 100, 512, window=2048, sinks=8),
        # one sequence's drafts over the tiny vocabulary
        _verify("verify-tiny", 1, 4, 1024, 0.8),
        # many sequences over a large vocabulary of odd size
        _verify("verify-wide", 48, 8, 128003, 0.7, short=3),
        # drafts that were chosen greedily, without probabilities of their own
        _verify("verify-greedy", 16, 12, 32000, 0.9, given=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


HEADS = ((4, 4, 64), (8, 2, 64), (32, 32, 128), (40, 40, 128), (64, 8, 128), (12, 4, 128))


def draw(rng):
    kind = rng.choice(("rope", "quantize", "attention", "attention", "attention", "verify"))
    if kind == "rope":
        heads, kv_heads, dh = rng.choice(HEADS)
        rows = _log(rng, 1, 8064 * 120 // max(120, heads + 2 * kv_heads))
        seqs = _log(rng, 1, min(64, rows))
        tokens = max(1, rows // seqs)
        return _rope(None, seqs, tokens, heads, kv_heads, dh, rng.choice((0, _log(rng, 1, 131000))),
                     rng.random() < 0.6, 128 * rng.randint(-(-tokens // 128), -(-tokens // 128) + 3),
                     rng.randrange(0, tokens))
    if kind == "quantize":
        kv_heads, dh = rng.choice(((4, 64), (8, 128), (32, 128), (40, 128)))
        block = rng.choice((32, 64, 128))
        rows = _log(rng, 32, 16384 * 8 * 8 // kv_heads)
        seqs = _log(rng, 1, min(64, max(1, rows // block)))
        blocks = max(1, rows // seqs // block)
        context = block * rng.choice((0, rng.randrange(0, 64)))
        ring = 128 * -(-(blocks + 1) * block // 128)
        return _quantize(None, seqs, kv_heads, dh, block, context + (blocks + 1) * block, context, blocks, ring)
    if kind == "attention":
        heads, kv_heads, dh = rng.choice(HEADS)
        tokens = _log(rng, 1, 16)
        seqs = _log(rng, 1, 64)
        most = 12 * 16385 * 8 // (seqs * kv_heads)
        context = _log(rng, 1, min(131000, max(16, most)))
        window = rng.choice((0, 0, _log(rng, 16, 4096)))
        return _attention(None, seqs, tokens, heads, kv_heads, dh, context, rng.choice((32, 64, 128)),
                          rng.randrange(0, 200), 512, window, rng.randrange(0, 9) if window else 0,
                          rng.randrange(0, tokens), rng.random() < 0.7)
    vocab = _log(rng, 1000, 128003)
    seqs = _log(rng, 1, 48)
    return _verify(None, seqs, rng.randint(1, 8), vocab, rng.uniform(0.2, 1.0), rng.random() < 0.7,
                   rng.randrange(0, 3))


# --------------------------------------------------------------------------
# inputs


def _lengths(case):
    """Rows in each sequence's cache before the call: the first is the case's
    context, the others between a quarter of it and all."""
    rng = random.Random(case["context"] + 7 * case["seqs"])
    n = case["context"]
    if not case.get("ragged", True):
        return [n] * case["seqs"]
    return [n] + [rng.randint(n // 4, n) for _ in range(case["seqs"] - 1)]


def _counts(case):
    """Tokens of each sequence in the call."""
    rng = random.Random(case["short"] + 11 * case["seqs"])
    most = case["tokens"] if "tokens" in case else case["drafts"]
    return [most] + [most - rng.randint(0, min(case["short"], most)) for _ in range(case["seqs"] - 1)]


def _held(case):
    return [max(0, n - case["recent"]) // case["block"] * case["block"] for n in _lengths(case)]


def _reach(case):
    """Each sequence's (rows held in 8 bits, rows in bf16) that the call reads."""
    w = case["window"]
    found = []
    for n, t, h in zip(_lengths(case), _counts(case), _held(case)):
        low = max(0, n + 1 - w) if w else 0
        sinks = min(case["sinks"], low)
        eight = min(sinks, h) + max(0, h - low) if t else 0
        found.append((eight, (max(0, sinks - h) + n + t - max(low, h)) if t else 0))
    return found


def _whole(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _to_eight(x, block):
    """x [..., rows, dh] as (e4m3, scales [..., rows / block]): the power of
    two that brings a block's largest value to at most 448."""
    r = x.float().unflatten(-2, (-1, block))
    most = torch.where(r.isfinite(), r.abs(), 0.0).amax((-2, -1))
    part, e = torch.frexp(most)
    e = torch.where(part > 0.875, e - 8, e - 9).clamp(min=-64)
    scale = torch.where(most == 0, 1.0, torch.ldexp(torch.ones_like(most), e))
    y = r / scale[..., None, None]
    y = torch.where(r.isfinite(), y, float("nan"))
    return y.flatten(-3, -2).to(torch.float8_e4m3fn), scale


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, dtype=torch.float32, std=1.0):
        t = torch.empty(*shape, dtype=dtype, device="cuda").normal_(0.0, 1.0, generator=g)
        return t if std == 1.0 else t.mul_(std)

    s = dict(case)
    if case["op"] == "rope":
        B, T, H, Hkv, dh = (case[x] for x in ("seqs", "tokens", "heads", "kv_heads", "dh"))
        s["qkv"] = normal(B, T, (H + 2 * Hkv) * dh, std=1.5)
        s["lengths"], s["counts"] = _whole(_lengths(case)), _whole(_counts(case))
        s["k"] = normal(B, Hkv, case["ring"], dh, dtype=torch.bfloat16)
        s["v"] = normal(B, Hkv, case["ring"], dh, dtype=torch.bfloat16)
        s["q_gain"] = 1.0 + normal(dh, std=0.2) if case["norms"] else None
        s["k_gain"] = 1.0 + normal(dh, std=0.2) if case["norms"] else None
    elif case["op"] == "quantize":
        B, Hkv, dh, block = (case[x] for x in ("seqs", "kv_heads", "dh", "block"))
        rng = random.Random(case["context"] + 13 * case["blocks"])
        done = [n // block * block for n in _lengths(case)]
        # the first has all of its new blocks; most have a part of one more
        n = [case["blocks"]] + [rng.randint(0, case["blocks"]) for _ in range(B - 1)]
        s["held"] = _whole(done)
        s["lengths"] = _whole([min(case["max_seq"], d + m * block + (i + 1) % block)
                               for i, (d, m) in enumerate(zip(done, n))])
        # heads differ in size, as keys do
        size = torch.empty(Hkv, 1, 1, device="cuda").exponential_(generator=g).add_(0.1).bfloat16()
        s["k"] = normal(B, Hkv, case["ring"], dh, dtype=torch.bfloat16).mul_(size)
        s["v"] = normal(B, Hkv, case["ring"], dh, dtype=torch.bfloat16)
        for x in ("k", "v"):
            s[x + "8"] = torch.zeros(B, Hkv, case["max_seq"], dh, dtype=torch.uint8,
                                     device="cuda").view(torch.float8_e4m3fn)
            s[x + "_scale"] = torch.ones(B, Hkv, case["max_seq"] // block, device="cuda")
    elif case["op"] == "attention":
        B, T, H, Hkv, dh, block = (case[x] for x in ("seqs", "tokens", "heads", "kv_heads", "dh", "block"))
        held = _held(case)
        s["max_held"] = max(held)
        s["max_tail"] = max(n + t - h for n, t, h in zip(_lengths(case), _counts(case), held))
        rows = max(block, -(-case["context"] // block) * block)
        s["q"] = normal(B, T, H, dh, dtype=torch.bfloat16, std=1.5)
        s["k"] = normal(B, Hkv, case["ring"], dh, dtype=torch.bfloat16)
        s["v"] = normal(B, Hkv, case["ring"], dh, dtype=torch.bfloat16)
        s["lengths"], s["counts"], s["held"] = _whole(_lengths(case)), _whole(_counts(case)), _whole(held)
        for x in ("k", "v"):
            s[x + "8"] = normal(B, Hkv, rows, dh, dtype=torch.bfloat16, std=100.0).clamp_(
                -448.0, 448.0).to(torch.float8_e4m3fn)
            # as large as the bf16 rows, give or take a binade
            s[x + "_scale"] = torch.ldexp(torch.ones(B, Hkv, rows // block, device="cuda"), torch.randint(
                -8, -5, (B, Hkv, rows // block), generator=g, device="cuda"))
    else:
        B, d, V = case["seqs"], case["drafts"], case["vocab"]
        # the target's probabilities, and a draft's that shares a part of them
        z = normal(B, d + 1, V, std=2.0)
        s["p"] = torch.softmax(z, -1)
        z[:, :d] = z[:, :d] * case["agree"] + normal(B, d, V, std=2.0) * (1.0 - case["agree"])
        q = torch.softmax(z[:, :d], -1)
        if case["given"]:
            s["q"] = q
            s["ids"] = (q / torch.empty_like(q).exponential_(generator=g)).argmax(-1).int()
        else:
            s["q"] = None
            # greedy drafts, of which the target often thinks little
            s["ids"] = (s["p"][:, :d] * torch.empty_like(q).exponential_(generator=g).pow_(
                4.0 * (1.0 - case["agree"]))).argmax(-1).int()
        s["counts"] = _whole(_counts(case))
        s["accept_u"] = torch.rand(B, d, generator=g, device="cuda")
        s["sample_u"] = torch.rand(B, generator=g, device="cuda")
    return s


# --------------------------------------------------------------------------
# plain forms


def _plain_rope(s):
    B, T, H, Hkv, dh, R = (s[x] for x in ("seqs", "tokens", "heads", "kv_heads", "dh", "ring"))
    at = torch.arange(T, device="cuda")
    here = at[None] < s["counts"][:, None]
    row = s["lengths"][:, None] + at[None]
    inv = THETA ** (-torch.arange(0, dh, 2, device="cuda", dtype=torch.float64) / dh)
    angle = row[..., None].double() * inv                   # far positions: 64 bits
    c, d = torch.cos(angle).float()[:, :, None], torch.sin(angle).float()[:, :, None]
    q, k, v = s["qkv"].view(B, T, H + 2 * Hkv, dh).split((H, Hkv, Hkv), dim=2)

    def turned(x, gain):
        if gain is not None:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * gain
        a, b = x.chunk(2, dim=-1)
        return torch.cat((a * c - b * d, b * c + a * d), dim=-1)

    q = torch.where(here[..., None, None], turned(q, s["q_gain"]), 0.0).to(torch.bfloat16)
    # tokens that a sequence does not have leave the row of the last as it is
    seq = torch.arange(B, device="cuda")[:, None].expand(B, T)
    slot = (row % R).long()
    for name, x in (("k", turned(k, s["k_gain"])), ("v", v)):
        s[name][seq, :, slot] = torch.where(here[..., None, None], x.to(torch.bfloat16), s[name][seq, :, slot])
    return {"q": q, "k": s["k"], "v": s["v"]}


def _plain_quantize(s):
    B, Hkv, dh, block, R = (s[x] for x in ("seqs", "kv_heads", "dh", "block", "ring"))
    n = s["blocks"]
    stop = s["lengths"] // block * block
    at = s["held"][:, None] + torch.arange(n * block, device="cuda")[None]          # [B, rows]
    new = at < stop[:, None]
    row = at.long()
    seq = torch.arange(B, device="cuda")[:, None]
    for x in ("k", "v"):
        values = s[x].gather(2, (at % R).long()[:, None, :, None].expand(B, Hkv, n * block, dh))
        eight, scale = _to_eight(values, block)
        to = s[x + "8"].view(torch.uint8)
        # blocks that a sequence does not have yet stay as they are
        to[seq, :, row] = torch.where(new[..., None, None], eight.view(torch.uint8).transpose(1, 2), to[seq, :, row])
        where, fresh = row[:, ::block] // block, new[:, ::block, None]
        s[x + "_scale"][seq, :, where] = torch.where(fresh, scale.transpose(1, 2), s[x + "_scale"][seq, :, where])
    held = torch.maximum(s["held"], stop).int()
    return {"k8": s["k8"], "v8": s["v8"], "k_scale": s["k_scale"], "v_scale": s["v_scale"], "held": held}


def _plain_attention(s):
    B, T, H, Hkv, dh, block, R = (s[x] for x in ("seqs", "tokens", "heads", "kv_heads", "dh", "block", "ring"))
    G, w, sinks = H // Hkv, s["window"], s["sinks"]
    at = torch.arange(T, device="cuda")
    pos = s["lengths"][:, None] + at[None]                                          # [B, T]
    here = at[None] < s["counts"][:, None]
    low = (s["lengths"] + 1 - w).clamp(min=0) if w else torch.zeros_like(s["lengths"])
    many = s["max_held"]
    if w and many > sinks + w + T:
        # the first rows, then those from the first window on
        first = torch.arange(sinks, device="cuda")[None].expand(B, sinks)
        more = torch.maximum(low, torch.tensor(sinks, device="cuda"))[:, None] + torch.arange(
            w + T, device="cuda")[None]
        j8 = torch.cat((first, more), 1)
        row = j8.clamp(max=many - 1).long()
        pick = row[:, None, :, None].expand(B, Hkv, j8.shape[1], dh)
        k8, v8 = (s[x].view(torch.uint8).gather(2, pick).view(torch.float8_e4m3fn) for x in ("k8", "v8"))
        ks, vs = (s[x].gather(2, (row // block)[:, None].expand(B, Hkv, j8.shape[1])) for x in ("k_scale", "v_scale"))
    else:
        j8 = torch.arange(many, device="cuda")[None].expand(B, many)
        k8, v8 = s["k8"][:, :, :many], s["v8"][:, :, :many]
        ks, vs = (s[x][:, :, :many // block].repeat_interleave(block, 2) for x in ("k_scale", "v_scale"))
    jt = s["held"][:, None] + torch.arange(s["max_tail"], device="cuda")[None]
    slot = (jt % R).long()[:, None, :, None].expand(B, Hkv, jt.shape[1], dh)
    j = torch.cat((j8, jt), 1)[:, None]                                             # [B, 1, N]
    eight = torch.arange(j.shape[2], device="cuda") < j8.shape[1]
    seen = (j <= pos[..., None]) & (~eight | (j < s["held"][:, None, None])) & here[..., None]
    if w:
        seen &= (j < sinks) | (j > pos[..., None] - w)
    k = torch.cat((k8.float() * ks[..., None], s["k"].gather(2, slot).float()), 2)
    q = s["q"].view(B, T, Hkv, G, dh).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * T, dh).float()
    score = torch.matmul(q, k.transpose(2, 3)).view(B, Hkv, G, T, -1)
    score.mul_(1.0 / math.sqrt(dh)).masked_fill_(~seen[:, None, None], float("-inf"))
    most = score.amax(-1, keepdim=True)
    score.sub_(torch.where(most == float("-inf"), 0.0, most)).exp_()
    total = score.sum(-1, keepdim=True)
    score.div_(torch.where(total == 0, 1.0, total))
    v = torch.cat((v8.float() * vs[..., None], s["v"].gather(2, slot).float()), 2)
    out = torch.matmul(score.view(B, Hkv, G * T, -1), v).view(B, Hkv, G, T, dh)
    return out.permute(0, 3, 1, 2, 4).reshape(B, T, H, dh).to(torch.bfloat16)


def _plain_verify(s):
    B, d, V = s["seqs"], s["drafts"], s["vocab"]
    at = torch.arange(d, device="cuda")[None]
    y = s["ids"].long()[..., None]
    py = s["p"][:, :d].gather(2, y)[..., 0].double()
    qy = s["q"].gather(2, y)[..., 0].double() if s["given"] else torch.ones_like(py)
    # the product of two 32-bit values is exact in 64
    good = (s["accept_u"].double() * qy < py) & (at < s["counts"][:, None])
    taken = good.int().cumprod(1).sum(1)                                            # [B]
    p = s["p"].gather(1, taken[:, None, None].expand(B, 1, V))[:, 0].double()
    short = (taken < s["counts"])[:, None]
    last = taken.clamp(max=d - 1)[:, None]
    if s["given"]:
        q = s["q"].gather(1, last[..., None].expand(B, 1, V))[:, 0].double()
    else:
        q = torch.zeros_like(p).scatter_(1, s["ids"].long().gather(1, last), float("inf"))
    rest = torch.where(short, (p - q).clamp(min=0.0), p)
    rest = torch.where(rest.sum(1, keepdim=True) > 0, rest, p)
    part = rest.cumsum(1)                                                           # 64 bits: values next to a border
    token = (part > s["sample_u"].double()[:, None] * part[:, -1:]).int().argmax(1).int()
    tokens = torch.cat((s["ids"], s["ids"][:, :1]), 1)
    at = torch.arange(d + 1, device="cuda")[None]
    tokens = torch.where(at < taken[:, None], tokens, torch.where(at == taken[:, None], token[:, None], -1))
    return {"tokens": tokens.int(), "n": (taken + 1).int()}


PLAIN = {"rope": _plain_rope, "quantize": _plain_quantize, "attention": _plain_attention,
         "verify": _plain_verify}


def _own(s):
    from self_speculative_decoding_gb300 import ops
    if s["op"] == "rope":
        q = ops.rope_append(s["qkv"], s["lengths"], s["k"], s["v"], s["heads"], s["kv_heads"], s["dh"],
                            THETA, q_gain=s["q_gain"], k_gain=s["k_gain"], eps=EPS, counts=s["counts"])
        return {"q": q, "k": s["k"], "v": s["v"]}
    if s["op"] == "quantize":
        held = ops.cache_quantize(s["k"], s["v"], s["held"], s["lengths"], s["k8"], s["v8"],
                                  s["k_scale"], s["v_scale"])
        return {"k8": s["k8"], "v8": s["v8"], "k_scale": s["k_scale"], "v_scale": s["v_scale"],
                "held": held}
    if s["op"] == "attention":
        return ops.cache_attention(s["q"], s["k"], s["v"], s["lengths"], k8=s["k8"], v8=s["v8"],
                                   k_scale=s["k_scale"], v_scale=s["v_scale"], held=s["held"],
                                   counts=s["counts"], window=s["window"], sinks=s["sinks"])
    tokens, n = ops.verify_drafts(s["p"], s["ids"], s["accept_u"], s["sample_u"], q=s["q"],
                                  counts=s["counts"])
    return {"tokens": tokens, "n": n}


def run(state):
    if own:
        return _own(state)
    return PLAIN[state["op"]](state)


# --------------------------------------------------------------------------
# what a call cannot do without


def work(case):
    if case["op"] == "rope":
        H, Hkv, dh = case["heads"], case["kv_heads"], case["dh"]
        n = sum(_counts(case))
        return {"bytes": n * (H + 2 * Hkv) * dh * 6 + 8 * case["seqs"], "flops": 10 * n * (H + Hkv) * dh}
    if case["op"] == "quantize":
        rng = random.Random(case["context"] + 13 * case["blocks"])
        n = case["blocks"] + sum(rng.randint(0, case["blocks"]) for _ in range(case["seqs"] - 1))
        e = n * case["kv_heads"] * case["block"] * case["dh"] * 2
        return {"bytes": 3 * e + n * case["kv_heads"] * 8 + 12 * case["seqs"], "flops": 2 * e}
    if case["op"] == "attention":
        H, Hkv, dh = case["heads"], case["kv_heads"], case["dh"]
        reach, counts = _reach(case), _counts(case)
        nbytes = sum(e * Hkv * (2 * dh + 8 / case["block"]) + b * Hkv * 4 * dh for e, b in reach)
        nbytes += sum(counts) * H * dh * 2 + case["seqs"] * case["tokens"] * H * dh * 2
        return {"bytes": int(nbytes), "flops": sum(4 * H * dh * t * (e + b) for (e, b), t in zip(reach, counts))}
    rows = 2 if case["given"] else 1
    return {"bytes": case["seqs"] * (rows * case["vocab"] * 4 + case["drafts"] * 16), "flops": case["seqs"] * case["vocab"] * 3}


# --------------------------------------------------------------------------
# definitions in 64 bits


def _exact_rope(s):
    B, T, H, Hkv, dh, R = (s[x] for x in ("seqs", "tokens", "heads", "kv_heads", "dh", "ring"))
    half = dh // 2
    x = s["qkv"].double().reshape(B, T, H + 2 * Hkv, dh)
    power = torch.tensor([THETA ** (-2.0 * i / dh) for i in range(half)], dtype=torch.float64, device="cuda")
    out = torch.zeros(B, T, H, dh, dtype=torch.float64, device="cuda")
    k, v = s["k"].double(), s["v"].double()
    for b, (n, t) in enumerate(zip(_lengths(s), _counts(s))):
        if not t:
            continue
        p = torch.arange(n, n + t, dtype=torch.float64, device="cuda")
        turn = torch.polar(torch.ones(t, half, dtype=torch.float64, device="cuda"), p[:, None] * power[None])
        heads = x[b, :t, :H + Hkv].clone()
        if s["norms"]:
            heads /= (heads.pow(2).sum(-1, keepdim=True) / dh + EPS).sqrt()
            heads[:, :H] *= s["q_gain"].double()
            heads[:, H:] *= s["k_gain"].double()
        z = torch.complex(heads[..., :half].contiguous(), heads[..., half:].contiguous()) * turn[:, None]
        heads = torch.cat((z.real, z.imag), -1)
        out[b, :t] = heads[:, :H]
        slots = torch.tensor([(n + i) % R for i in range(t)], device="cuda")
        k[b, :, slots] = heads[:, H:].transpose(0, 1)
        v[b, :, slots] = x[b, :t, H + Hkv:].transpose(0, 1)
    return {"q": out, "k": k, "v": v}


def _exact_quantize(s):
    block, R = s["block"], s["ring"]
    held, length = s["held"].tolist(), s["lengths"].tolist()
    # every e4m3 value that is not negative, in order: its place is its code
    steps = [m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10) for e in range(16) for m in range(8)][:-1]
    steps = torch.tensor(steps, dtype=torch.float64, device="cuda")
    r = {"held": _whole([max(a, b // block * block) for a, b in zip(held, length)])}
    for x in ("k", "v"):
        eight, scales = s[x + "8"].double(), s[x + "_scale"].double()
        for b, (a, stop) in enumerate(zip(held, length)):
            for c in range(a // block, stop // block):
                rows = s[x][b, :, [j % R for j in range(c * block, c * block + block)]].double()
                most = rows.abs().amax((1, 2))
                scale = torch.tensor([2.0 ** max(-64, math.ceil(math.log2(m / 448.0))) if m else 1.0
                                      for m in most.tolist()], dtype=torch.float64, device="cuda")
                y = rows / scale[:, None, None]
                up = torch.searchsorted(steps, y.abs().contiguous()).clamp(max=126)
                low = (up - 1).clamp(min=0)
                near, far = steps[up] - y.abs(), y.abs() - steps[low]
                code = torch.where((near < far) | ((near == far) & (up % 2 == 0)), up, low)
                eight[b, :, c * block:c * block + block] = steps[code] * y.sign()
                scales[b, :, c] = scale
        r[x + "8"], r[x + "_scale"] = eight, scales
    return r


def _exact_attention(s):
    T, H, Hkv, dh, R = (s[x] for x in ("tokens", "heads", "kv_heads", "dh", "ring"))
    G, block, w = H // Hkv, s["block"], s["window"]
    out = torch.zeros(s["seqs"], T, H, dh, dtype=torch.float64, device="cuda")
    for b, (n, t, held) in enumerate(zip(_lengths(s), _counts(s), _held(s))):
        if not t:
            continue
        j = torch.arange(n + t, device="cuda")
        p = torch.arange(n, n + t, device="cuda")[:, None]
        hidden = j[None] > p
        if w:
            hidden |= (j[None] <= p - w) & (j[None] >= s["sinks"])
        slots = torch.arange(held, n + t, device="cuda") % R
        for h in range(Hkv):
            def rows(x):
                old = s[x + "8"][b, h, :held].double().reshape(-1, block, dh)
                old = old * s[x + "_scale"][b, h, :held // block].double()[:, None, None]
                return torch.cat((old.reshape(-1, dh), s[x][b, h, slots].double()))

            a = torch.einsum("tgd,jd->gtj", s["q"][b, :t, h * G:h * G + G].double(), rows("k")) / math.sqrt(dh)
            a.masked_fill_(hidden, -math.inf)
            a = (a - torch.logsumexp(a, -1, keepdim=True)).exp()
            out[b, :t, h * G:h * G + G] = torch.einsum("gtj,jd->tgd", a, rows("v"))
    return out


def _exact_verify(s):
    tokens = torch.full((s["seqs"], s["drafts"] + 1), -1, dtype=torch.int32)
    count = []
    u, U, drafts = s["accept_u"].tolist(), s["sample_u"].tolist(), s["ids"].tolist()
    for b, most in enumerate(_counts(s)):
        n = 0
        while n < most:
            y = drafts[b][n]
            if not u[b][n] * (s["q"][b, n, y].item() if s["given"] else 1.0) < s["p"][b, n, y].item():
                break
            tokens[b, n] = y
            n += 1
        r = s["p"][b, n].double()
        if n < most:
            other = r.clone()
            if s["given"]:
                other = (r - s["q"][b, n].double()).clamp(min=0.0)
            else:
                other[drafts[b][n]] = 0.0
            r = other if float(other.sum()) > 0 else r
        part = torch.cumsum(r, 0)
        tokens[b, n] = int(torch.searchsorted(part, part[-1:] * U[b], right=True))
        count.append(n + 1)
    return {"tokens": tokens.cuda(), "n": _whole(count)}


def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "quantize": _exact_quantize, "attention": _exact_attention,
            "verify": _exact_verify}[case["op"]](s)
