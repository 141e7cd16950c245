"""Timed cases of the tree-decoding operators.

Four operators of a decoding round that drafts a tree of tokens instead of a
chain: attention of the tree's nodes over the cache, eviction from a cache by
accumulated attention weight, the beam selection that picks a tree level (or
the next beams) from the logits, and the reordering of the beams' caches.

``listed`` and ``draw`` give cases, ``prepare`` the tensors that a program has
in hand before the call, ``run`` one call: the plain torch form, or the
library's kernels where ``own`` is true.  ``exact`` is the definition in 64
bits and ``work`` the bytes and operations that a call cannot do without.
"""

import math
import random

import numpy as np
import torch

own = False

THETA = 1.0e4


# --------------------------------------------------------------------------
# cases


def _tree(name, heads, kv_heads, dh, context, nodes, weights, absent=0, width=4, spare=0, skipped=0):
    c = {"op": "tree", "heads": heads, "kv_heads": kv_heads, "dh": dh, "context": context,
         "nodes": nodes, "weights": weights, "absent": absent, "width": width,
         "max_seq": context + nodes + spare, "pos0": context + skipped}
    return dict(c, name=name) if name else c


def _evict(name, kv_heads, dh, bits, rows, keep, sinks, recent, spare=0):
    c = {"op": "evict", "kv_heads": kv_heads, "dh": dh, "bits": bits, "rows": rows, "keep": keep,
         "sinks": sinks, "recent": recent, "max_seq": rows + spare, "max_out": keep + spare}
    return dict(c, name=name) if name else c


def _select(name, beams, vocab, width, finished=0, spread=2.0):
    c = {"op": "select", "beams": beams, "vocab": vocab, "width": width, "finished": finished,
         "spread": spread}
    return dict(c, name=name) if name else c


def _reorder(name, beams, width, layers, kv_heads, dh, bits, max_seq, start, stop):
    c = {"op": "reorder", "beams": beams, "width": width, "layers": layers, "kv_heads": kv_heads,
         "dh": dh, "bits": bits, "max_seq": max_seq, "start": start, "stop": stop}
    return dict(c, name=name) if name else c


def listed():
    return [
        # the tiny model's verify: a handful of drafted tokens behind a short
        # prompt, where the call's latency is all there is
        _tree("tree-tiny", 4, 4, 64, 83, 5, False, spare=40),
        # a single token behind a long context with grouped heads: the plain
        # decode step, with the weights that the eviction goes by
        _tree("tree-one-token", 64, 8, 128, 16385, 1, True, spare=62),
        # one head's cache per query head, a tree of 58 nodes padded to 61
        # rows, the weights accumulated
        _tree("tree-mha", 40, 40, 128, 2047, 61, True, absent=3, spare=1988),
        # grouped heads, 64 nodes, a cache that has been evicted from (the
        # tokens' positions run ahead of the cache's rows)
        _tree("tree-gqa-weights", 64, 8, 128, 32768, 64, True, spare=448, skipped=9000),
        # the largest tree behind the longest context
        _tree("tree-gqa-long", 64, 8, 128, 131000, 256, False, width=16, spare=72),
        # the tiny fp32 model's cache, cut to 64 rows
        _evict("evict-tiny", 4, 64, 32, 121, 64, 4, 16, spare=7),
        # a cache of 4095 rows halved, one head per query head
        _evict("evict-mha", 40, 128, 16, 4095, 2048, 4, 256, spare=1),
        # the longest cache, an eighth of it kept
        _evict("evict-long", 8, 128, 16, 131072, 16384, 4, 1024),
        # one level of a small tree over the tiny vocabulary
        _select("select-tiny", 4, 1024, 4),
        # many beams over a large vocabulary of odd size, some of them ended
        _select("select-wide", 48, 128003, 48, finished=3),
        # the tiny model's beams, a few tokens behind their common prompt
        _reorder("reorder-tiny", 4, 4, 4, 4, 64, 32, 128, 16, 29),
        # eight beams of a 32-layer model, a thousand tokens behind the prompt
        _reorder("reorder-deep", 8, 8, 32, 8, 128, 16, 2048, 512, 1537),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(("tree", "tree", "evict", "select", "reorder"))
    if kind == "tree":
        heads, kv_heads, dh = rng.choice(((4, 4, 64), (8, 2, 64), (32, 32, 128), (40, 40, 128),
                                          (64, 8, 128), (12, 4, 128)))
        nodes = _log(rng, 1, 256)
        most = 64 * 256 * 131000 // (heads * nodes)
        context = _log(rng, 1, min(131000, max(16, most)))
        context = min(context, 131000 * 8 // kv_heads)
        absent = rng.randrange(0, nodes // 4 + 1)
        return _tree(None, heads, kv_heads, dh, context, nodes, rng.random() < 0.5, absent,
                     rng.randint(1, 16), rng.randrange(0, 300), rng.choice((0, rng.randrange(5000))))
    if kind == "evict":
        kv_heads, dh = rng.choice(((4, 64), (8, 128), (32, 128), (40, 128)))
        rows = _log(rng, 64, 131072 * 8 // max(8, kv_heads))
        keep = max(1, min(rows, int(rows * rng.uniform(0.05, 0.5))))
        sinks = min(keep, rng.randrange(0, 9))
        recent = rng.randrange(0, (keep - sinks) // 2 + 1)
        return _evict(None, kv_heads, dh, rng.choice((16, 16, 32)) if rows <= 65536 else 16, rows,
                      keep, sinks, recent, rng.randrange(0, 200))
    if kind == "select":
        beams = _log(rng, 1, 48)
        vocab = _log(rng, 1000, 128003)
        return _select(None, beams, vocab, _log(rng, 1, 48), rng.randrange(0, beams // 4 + 1),
                       rng.choice((1.0, 2.0, 4.0)))
    beams, width = rng.randint(1, 8), rng.randint(1, 8)
    layers = _log(rng, 1, 32)
    kv_heads, dh = rng.choice(((4, 64), (8, 128)))
    max_seq = _log(rng, 64, 2048)
    start = rng.randrange(0, max_seq // 2)
    stop = start + rng.randrange(1, max_seq // 2)
    return _reorder(None, beams, width, layers, kv_heads, dh, 16, max_seq, start, stop)


# --------------------------------------------------------------------------
# inputs


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rng = random.Random(seed)

    def normal(*shape, std=1.0, dtype=torch.float32):
        t = torch.empty(*shape, dtype=dtype, device="cuda").normal_(0.0, 1.0, generator=g)
        return t if std == 1.0 else t.mul_(std)

    def expo(*shape):
        return torch.empty(*shape, dtype=torch.float32, device="cuda").exponential_(generator=g)

    s = dict(case)
    if case["op"] == "tree":
        H, Hkv, dh, T = case["heads"], case["kv_heads"], case["dh"], case["nodes"]
        qkv = normal(T, (H + 2 * Hkv) * dh)
        qkv[:, : H * dh] *= 1.5           # scores spread a little over a unit
        live = T - case["absent"]
        # node 0 is the pending token; the others hang below one of the last
        # `width` nodes before them; the padding rows at the end name no parent
        parents = [-1] + [i - 1 - rng.randrange(min(i, case["width"])) for i in range(1, live)]
        parents += [-2] * (T - live)
        s["qkv"] = qkv
        s["parents"] = torch.tensor(parents[:T], dtype=torch.int32, device="cuda")
        s["k"] = normal(Hkv, case["max_seq"], dh, dtype=torch.bfloat16)
        s["v"] = normal(Hkv, case["max_seq"], dh, dtype=torch.bfloat16)
        if case["weights"]:
            # what earlier calls left: a few rows hold most of it
            s["weights"] = expo(Hkv, case["max_seq"]).pow_(3)
            s["weights_out"] = torch.zeros_like(s["weights"])
    elif case["op"] == "evict":
        dt = torch.bfloat16 if case["bits"] == 16 else torch.float32
        Hkv, dh = case["kv_heads"], case["dh"]
        s["k"] = normal(Hkv, case["max_seq"], dh, dtype=dt)
        s["v"] = normal(Hkv, case["max_seq"], dh, dtype=dt)
        s["weights"] = expo(Hkv, case["max_seq"]).pow_(3)
        s["k_out"] = torch.zeros(Hkv, case["max_out"], dh, dtype=dt, device="cuda")
        s["v_out"] = torch.zeros_like(s["k_out"])
        s["weights_out"] = torch.zeros(Hkv, case["max_out"], device="cuda")
    elif case["op"] == "select":
        B, V = case["beams"], case["vocab"]
        s["logits"] = normal(B, V, std=case["spread"])
        s["lse"] = torch.logsumexp(s["logits"].double(), 1).float()  # as the LM head's row summary holds it
        s["scores"] = expo(B).mul_(-4.0)
        s["end_id"] = 2
        done = [1] * case["finished"] + [0] * (B - case["finished"])
        rng.shuffle(done)
        s["done"] = torch.tensor(done, dtype=torch.int32, device="cuda")
    else:
        dt = torch.bfloat16 if case["bits"] == 16 else torch.float32
        shape = (case["layers"], case["kv_heads"], case["max_seq"], case["dh"])
        s["k"] = normal(case["beams"], *shape, dtype=dt)
        s["v"] = normal(case["beams"], *shape, dtype=dt)
        s["k_out"] = torch.zeros(case["width"], *shape, dtype=dt, device="cuda")
        s["v_out"] = torch.zeros_like(s["k_out"])
        s["parents"] = torch.tensor([rng.randrange(case["beams"]) for _ in range(case["width"])],
                                    dtype=torch.int32, device="cuda")
    return s


# --------------------------------------------------------------------------
# plain forms


def _visible(parents):
    """(visible [T, T], depth [T]): node i sees its ancestors and itself; a
    row whose chain does not end in a parent of -1 is absent and sees nothing."""
    T = parents.shape[0]
    at = torch.arange(T, device=parents.device)
    edge = (parents[:, None] == at[None, :]) & (at[None, :] < at[:, None])
    eye = torch.eye(T, device=parents.device)
    # the sum of all powers of the strictly lower triangular edge matrix
    reach = torch.linalg.solve_triangular(eye - edge.float(), eye, upper=False, unitriangular=True) > 0.5
    present = (reach & (parents == -1)[None, :]).any(1)
    visible = reach & present[:, None]
    return visible, visible.sum(1) - 1, present


def _rotate(x, angle):
    """Rotate-half RoPE of x [T, heads, dh] by angle [T, dh / 2]."""
    a, b = x.chunk(2, dim=-1)
    c, s = torch.cos(angle)[:, None].to(x.dtype), torch.sin(angle)[:, None].to(x.dtype)
    return torch.cat((a * c - b * s, b * c + a * s), dim=-1)


def _plain_tree(s):
    H, Hkv, dh, n, T = s["heads"], s["kv_heads"], s["dh"], s["context"], s["nodes"]
    G, N = H // Hkv, s["context"] + s["nodes"]
    visible, depth, present = _visible(s["parents"])
    inv = THETA ** (-torch.arange(0, dh, 2, device="cuda", dtype=torch.float64) / dh)
    angle = (s["pos0"] + depth).double()[:, None] * inv  # far positions: 64 bits
    q, k, v = s["qkv"].view(T, H + 2 * Hkv, dh).split((H, Hkv, Hkv), dim=1)
    q, k = _rotate(q, angle), _rotate(k, angle)
    here = present[:, None, None]
    s["k"][:, n:N] = torch.where(here, k, 0.0).transpose(0, 1).to(torch.bfloat16)
    s["v"][:, n:N] = torch.where(here, v, 0.0).transpose(0, 1).to(torch.bfloat16)
    seen = torch.cat((present[:, None].expand(T, n), visible), dim=1)        # [T, N]
    q = q.view(T, Hkv, G, dh).permute(1, 2, 0, 3).reshape(Hkv, G * T, dh)
    score = torch.matmul(q, s["k"][:, :N].float().transpose(1, 2)).view(Hkv, G, T, N)
    score.mul_(1.0 / math.sqrt(dh)).masked_fill_(~seen, float("-inf"))
    most = score.amax(-1, keepdim=True)
    score.sub_(torch.where(most == float("-inf"), 0.0, most)).exp_()
    total = score.sum(-1, keepdim=True)
    score.div_(torch.where(total == 0, 1.0, total))
    out = torch.matmul(score.view(Hkv, G * T, N), s["v"][:, :N].float())
    out = out.view(Hkv, G, T, dh).permute(2, 0, 1, 3).reshape(T, H * dh).to(torch.bfloat16)
    r = {"out": out, "k": s["k"], "v": s["v"]}
    if s.get("weights") is not None and s["op"] == "tree" and "weights_out" in s:
        mass = score.sum((1, 2))
        s["weights_out"][:, :n] = s["weights"][:, :n] + mass[:, :n]
        s["weights_out"][:, n:N] = mass[:, n:]
        r["weights"] = s["weights_out"]
    return r


def _plain_evict(s):
    n, keep, sinks, recent = s["rows"], s["keep"], s["sinks"], s["recent"]
    Hkv, dh = s["kv_heads"], s["dh"]
    w = s["weights"][:, sinks:n - recent]
    w = torch.where(torch.isnan(w), float("-inf"), w)
    # ties go to the lowest row: a stable sort
    middle = w.sort(dim=1, descending=True, stable=True).indices[:, :keep - sinks - recent] + sinks
    middle = middle.sort(dim=1).values
    first = torch.arange(sinks, device="cuda").expand(Hkv, sinks)
    last = torch.arange(n - recent, n, device="cuda").expand(Hkv, recent)
    kept = torch.cat((first, middle, last), dim=1)
    rows = kept[:, :, None].expand(Hkv, keep, dh)
    s["k_out"][:, :keep] = s["k"].gather(1, rows)
    s["v_out"][:, :keep] = s["v"].gather(1, rows)
    s["weights_out"][:, :keep] = s["weights"].gather(1, kept)
    return {"k": s["k_out"], "v": s["v_out"], "weights": s["weights_out"], "kept": kept.to(torch.int32)}


def _plain_select(s):
    B, V, W = s["beams"], s["vocab"], s["width"]
    take = min(W, V)
    done = s["done"] != 0
    z = torch.where(torch.isnan(s["logits"]), float("-inf"), s["logits"])
    z, token = z.sort(dim=1, descending=True, stable=True)
    z, token = z[:, :take], token[:, :take]
    # the sums of 32-bit values in 64 bits: beams are compared without rounding
    score = s["scores"].double()[:, None] + (z.double() - s["lse"].double()[:, None])
    # an ended beam stands for itself: one candidate, its own score
    lone = torch.full_like(score, float("-inf"))
    lone[:, 0] = s["scores"].double()
    score = torch.where(done[:, None], lone, score)
    token = torch.where(done[:, None], s["end_id"], token)
    score = torch.where(torch.isnan(score), float("-inf"), score).view(-1)
    short = max(0, W - B * take)
    score = torch.cat((score, score.new_full((short,), float("-inf"))))
    token = torch.cat((token.reshape(-1), token.new_zeros(short)))
    best, at = score.sort(descending=True, stable=True)
    best, at = best[:W], at[:W]
    none = best == float("-inf")
    tokens = torch.where(none, -1, token[at])
    parents = torch.where(none, -1, at // take)
    ended = (tokens == s["end_id"]) | none
    return {"tokens": tokens.to(torch.int32), "parents": parents.to(torch.int32),
            "scores": best.float(), "done": ended.to(torch.int32)}


def _plain_reorder(s):
    a, b = s["start"], s["stop"]
    p = s["parents"].long()
    good = ((p >= 0) & (p < s["beams"]))[:, None, None, None, None]
    p = p.clamp(0, s["beams"] - 1)
    s["k_out"][:, :, :, a:b] = torch.where(good, s["k"][:, :, :, a:b][p], s["k_out"][:, :, :, a:b])
    s["v_out"][:, :, :, a:b] = torch.where(good, s["v"][:, :, :, a:b][p], s["v_out"][:, :, :, a:b])
    return {"k": s["k_out"], "v": s["v_out"]}


PLAIN = {"tree": _plain_tree, "evict": _plain_evict, "select": _plain_select, "reorder": _plain_reorder}


def _own(s):
    from self_speculative_decoding_gb300 import ops
    if s["op"] == "tree":
        out = ops.tree_attention(s["qkv"], s["parents"], s["k"], s["v"], s["context"], s["pos0"],
                                 s["heads"], s["kv_heads"], s["dh"], THETA,
                                 weights=s.get("weights") if "weights_out" in s else None,
                                 weights_out=s.get("weights_out"))
        r = {"out": out, "k": s["k"], "v": s["v"]}
        if "weights_out" in s:
            r["weights"] = s["weights_out"]
        return r
    if s["op"] == "evict":
        kept = ops.cache_evict(s["k"], s["v"], s["weights"], s["rows"], s["keep"], s["k_out"],
                               s["v_out"], s["weights_out"], sinks=s["sinks"], recent=s["recent"])
        return {"k": s["k_out"], "v": s["v_out"], "weights": s["weights_out"], "kept": kept}
    if s["op"] == "select":
        tokens, parents, scores, done = ops.beam_select(s["logits"], s["scores"], s["width"],
                                                        lse=s["lse"], done=s["done"],
                                                        end_id=s["end_id"])
        return {"tokens": tokens, "parents": parents, "scores": scores, "done": done}
    ops.beam_reorder(s["k"], s["v"], s["parents"], s["start"], s["stop"], s["k_out"], s["v_out"])
    return {"k": s["k_out"], "v": s["v_out"]}


def run(state):
    if own:
        return _own(state)
    return PLAIN[state["op"]](state)


# --------------------------------------------------------------------------
# what a call cannot do without


def work(case):
    if case["op"] == "tree":
        H, Hkv, dh, n, T = case["heads"], case["kv_heads"], case["dh"], case["context"], case["nodes"]
        live = T - case["absent"]
        nbytes = n * Hkv * dh * 2 * 2 + T * Hkv * dh * 2 * 2       # the cache read, the new rows written
        nbytes += T * (H + 2 * Hkv) * dh * 4 + T * 4 + T * H * dh * 2
        if case["weights"]:
            nbytes += Hkv * n * 4 + Hkv * (n + T) * 4
        return {"bytes": nbytes, "flops": 4 * H * dh * live * (n + 1)}
    if case["op"] == "evict":
        Hkv, dh, e = case["kv_heads"], case["dh"], case["bits"] // 8
        nbytes = Hkv * case["rows"] * 4 + Hkv * case["keep"] * (2 * 2 * dh * e + 4 + 4)
        return {"bytes": nbytes, "flops": Hkv * case["rows"]}
    if case["op"] == "select":
        B, V, W = case["beams"], case["vocab"], case["width"]
        return {"bytes": (B - case["finished"]) * V * 4 + B * 12 + W * 16,
                "flops": (B - case["finished"]) * V}
    e = case["bits"] // 8
    rows = case["width"] * case["layers"] * case["kv_heads"] * (case["stop"] - case["start"])
    # a source row is read once however many beams take it: so many of them are taken on average
    taken = case["beams"] * (1.0 - (1.0 - 1.0 / case["beams"]) ** case["width"]) / case["width"]
    return {"bytes": int(2 * rows * case["dh"] * e * (1.0 + taken)), "flops": 0}


# --------------------------------------------------------------------------
# definitions in 64 bits


def _exact_tree(s):
    H, Hkv, dh, n, T = s["heads"], s["kv_heads"], s["dh"], s["context"], s["nodes"]
    G, half = H // Hkv, dh // 2
    parents = s["parents"].tolist()
    paths = []
    for i, p in enumerate(parents):
        above = [] if p == -1 else paths[p] if 0 <= p < i else None
        paths.append(None if above is None else above + [i])
    qkv = s["qkv"].double().reshape(T, H + 2 * Hkv, dh)
    turn = [[(s["pos0"] + len(p) - 1 if p else 0) * THETA ** (-2.0 * i / dh) for i in range(half)] for p in paths]
    turn = torch.polar(torch.ones(T, half, dtype=torch.float64), torch.tensor(turn, dtype=torch.float64)).cuda()
    z = torch.complex(qkv[..., :half], qkv[..., half:])[:, :H + Hkv] * turn[:, None]
    rot = torch.cat((z.real, z.imag), -1)
    live = [i for i, p in enumerate(paths) if p]
    k_all, v_all = s["k"].double(), s["v"].double()
    k_all[:, n:n + T] = 0.0
    v_all[:, n:n + T] = 0.0
    for i in live:
        k_all[:, n + i] = rot[i, H:].bfloat16().double()    # the cache holds bf16, and attention reads the cache
        v_all[:, n + i] = qkv[i, H + Hkv:].bfloat16().double()
    hidden = torch.ones(T, T, dtype=torch.bool)
    for i in live:
        hidden[i, paths[i]] = False
    hidden = hidden.cuda()
    out = torch.zeros(T, H, dh, dtype=torch.float64, device="cuda")
    mass = torch.zeros(Hkv, n + T, dtype=torch.float64, device="cuda")
    rows = torch.tensor(live, device="cuda")
    for h in range(H):
        kv = h // G
        a = rot[rows, h] @ k_all[kv, :n + T].T / math.sqrt(dh)
        a[:, n:].masked_fill_(hidden[rows], -math.inf)
        a -= torch.logsumexp(a, 1, keepdim=True)
        a.exp_()
        out[rows, h] = a @ v_all[kv, :n + T]
        mass[kv] += a.sum(0)
    # the rows as they were before they went into the cache
    k_all[:, n + rows], v_all[:, n + rows] = rot[rows, H:].transpose(0, 1), qkv[rows, H + Hkv:].transpose(0, 1)
    r = {"out": out.reshape(T, H * dh), "k": k_all, "v": v_all}
    if s["weights_out"] is not None:
        w = torch.zeros(Hkv, s["max_seq"], dtype=torch.float64, device="cuda")
        w[:, :n] = s["weights"][:, :n].double()
        w[:, :n + T] += mass
        r["weights"] = w
    return r


def _exact_evict(s):
    n, keep, sinks, recent = s["rows"], s["keep"], s["sinks"], s["recent"]
    w = s["weights"].cpu().numpy().astype(np.float64)[:, :n]
    kept = []
    for row in w:
        place = np.arange(n)
        rank = np.zeros(n)
        rank[:sinks] = rank[n - recent:] = -1
        value = np.where(np.isnan(row), -np.inf, row)
        kept.append(np.sort(np.lexsort((place, -value, rank))[:keep]))
    kept = torch.from_numpy(np.stack(kept)).cuda()
    k, v, wo = (torch.zeros_like(s[x], dtype=torch.float64) for x in ("k_out", "v_out", "weights_out"))
    for h in range(s["kv_heads"]):
        k[h, :keep], v[h, :keep] = s["k"][h, kept[h]].double(), s["v"][h, kept[h]].double()
        wo[h, :keep] = s["weights"][h, kept[h]].double()
    return {"k": k, "v": v, "weights": wo, "kept": kept.to(torch.int32)}


def _exact_select(s):
    B, W = s["beams"], s["width"]
    z, lse = s["logits"].cpu().numpy().astype(np.float64), s["lse"].cpu().numpy().astype(np.float64)
    base, done = s["scores"].cpu().numpy().astype(np.float64), s["done"].cpu().numpy()
    found = []
    for b in range(B):
        if done[b]:
            found.append((-base[b], b, 0, s["end_id"]))
            continue
        value = base[b] + (z[b] - lse[b])
        first = np.lexsort((np.arange(z.shape[1]), -z[b]))[:W]
        found += [(-value[t], b, r, int(t)) for r, t in enumerate(first)]
    found = sorted(found)[:W]
    lack = W - len(found)
    tokens = [f[3] for f in found] + [-1] * lack
    whole = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    return {"tokens": whole(tokens), "parents": whole([f[1] for f in found] + [-1] * lack),
            "scores": torch.tensor([-f[0] for f in found] + [-math.inf] * lack, dtype=torch.float64, device="cuda"),
            "done": whole([int(t == s["end_id"] or t < 0) for t in tokens])}


def _exact_reorder(s):
    k, v = torch.zeros_like(s["k_out"]), torch.zeros_like(s["v_out"])
    for w, p in enumerate(s["parents"].tolist()):
        k[w, :, :, s["start"]:s["stop"]] = s["k"][p, :, :, s["start"]:s["stop"]]
        v[w, :, :, s["start"]:s["stop"]] = s["v"][p, :, :, s["start"]:s["stop"]]
    return {"k": k, "v": v}


def exact(case, seed):
    s = prepare(case, seed)
    s.setdefault("weights_out", None)
    return {"tree": _exact_tree, "evict": _exact_evict, "select": _exact_select, "reorder": _exact_reorder}[case["op"]](s)
