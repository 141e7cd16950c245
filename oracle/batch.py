"""fp64 references of the calls of several sequences over 8-bit caches: head
norms with rotation, e4m3 blocks, attention over rows and verification of
drafts.  Written from the formulas, apart from the CUDA path."""

from __future__ import annotations

import math

import numpy as np


def head_norm(x, gain, eps):
    """x [..., dh] / sqrt(mean x^2 + eps) * gain; gain None: x."""
    if gain is None:
        return x
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * gain


def rotate(x, pos, theta):
    """Rotate-half RoPE of x [..., dh] to position pos."""
    half = x.shape[-1] // 2
    angle = pos * theta ** (-np.arange(half) / half)
    a, b = x[..., :half], x[..., half:]
    c, s = np.cos(angle), np.sin(angle)
    return np.concatenate((a * c - b * s, b * c + a * s), -1)


def e4m3_values():
    """The values of codes 0..126 (the largest, 448), in order."""
    return np.array([m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
                     for e in range(16) for m in range(8)][:-1])


def to_e4m3(y):
    """Codes (uint8) of y: nearest, ties to the even code; NaN and infinity 0x7f."""
    steps = e4m3_values()
    with np.errstate(invalid="ignore"):
        mag = np.abs(y)
        up = np.minimum(np.searchsorted(steps, np.where(np.isfinite(mag), mag, 0.0)), 126)
        low = np.maximum(up - 1, 0)
        near, far = steps[up] - mag, mag - steps[low]
        code = np.where((near < far) | ((near == far) & (up % 2 == 0)), up, low)
    return np.where(np.isfinite(y), code, 0x7F).astype(np.uint8) | (np.signbit(y) & np.isfinite(y)).astype(np.uint8) * 0x80


def from_e4m3(code):
    steps = np.append(e4m3_values(), np.nan)
    return np.where(code & 0x80, -1.0, 1.0) * steps[code & 0x7F]


def block_scale(rows):
    """The smallest power of two (2^-64 at least) that brings the largest finite
    magnitude to at most 448; 1 for zeros."""
    most = np.abs(rows[np.isfinite(rows)]).max(initial=0.0)
    if most == 0:
        return 1.0
    e = -64
    while most > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def seen_rows(pos, window=0, sinks=0):
    """The rows that a token in row pos sees."""
    j = np.arange(pos + 1)
    return j if not window else j[(j < sinks) | (j > pos - window)]


def attend(q, K, V, rows, scale):
    """softmax(scale q K^T) V over `rows`, and sum p |v|."""
    s = scale * (K[rows] @ q)
    p = np.exp(s - s.max())
    p /= p.sum()
    return p @ V[rows], p @ np.abs(V[rows])


def verify(p, q, drafts, accept_u, sample_u):
    """One sequence: p [c + 1, V], q [c, V] or None, drafts [c] -> the tokens."""
    out, V = [], p.shape[1]
    r = p[len(drafts)]
    for j, y in enumerate(drafts):
        if 0 <= y < V and accept_u[j] * (1.0 if q is None else q[j, y]) < p[j, y]:
            out.append(int(y))
            continue
        rest = p[j].copy()
        if q is not None:
            rest = p[j] - q[j]
        elif 0 <= y < V:
            rest[y] = 0.0
        rest = np.where(rest > 0, rest, 0.0)
        r = rest if rest.sum() > 0 else p[j]
        break
    r = np.where(r > 0, r, 0.0)
    total = math.fsum(r)
    if not 0 < total < math.inf:
        return out
    past = np.nonzero(np.cumsum(r) > sample_u * total)[0]
    return out + [int(past[0]) if len(past) else int(np.nonzero(r)[0][-1])]
