"""Plain 64-bit forms of the new-token operators (head norms with rotary positions, attention with capped,
biased and masked scores) and the error bounds that the kernels' arithmetic allows.

Bounds.  u = 2^-24 is half an fp32 step.  A score is a sum of 128 exact products in fp32, in any order
and perhaps truncated: off by at most 130 * 2u * sum|q_c k_c| * scale.  tanhf adds 4u * cap, the bias 2u
per term of the score's size.  A weight exp(s - m) is then off by a factor within e^(+-2 eps) and 2^-20
for the exponential, a sum of n of them by n * 2u; splitting the weight into two halves leaves 2^-21.
Rounding a weight once to fp16 adds 2^-11 (and 2^-25 * 2^9 absolute below the normal range, the weights
being at least 2^-9 of their scaled size).  An fp16 output adds 2^-11 of itself and 2^-25."""
import math

import numpy as np
import torch

D = 128
U = 2.0 ** -24


def visible(T, pos, prefix=0, doc=0, window=0, n_sink=0):
    """Truth per cached token for the query at position pos (its document from doc on)."""
    j = np.arange(T)
    hi = min(max(pos + 1, prefix), T)
    seen = (j >= doc) & (j < hi)
    if window:
        seen &= (j > pos - window) | (j < doc + n_sink)
    return seen


def attend(q, K, V, seen, pos, scale=0.0, softcap=0.0, slope=0.0, fp16=False):
    """(out, lse, bound on out, bound on lse) of one query row q [d] over K, V [T][d] (float64 arrays)."""
    scale = scale or 1.0 / math.sqrt(D)
    j = np.nonzero(seen)[0]
    if len(j) == 0:
        return np.zeros(D), -math.inf, np.zeros(D), 0.0
    k, v = K[j], V[j]
    s = scale * (k @ q)
    eps = 130 * 2 * U * scale * np.max(np.abs(k) @ np.abs(q))
    if softcap:
        s = softcap * np.tanh(s / softcap)
        eps += 4 * U * softcap
    if slope:
        s = s - slope * np.abs(pos - j)
    eps += 4 * U * max(1.0, np.max(np.abs(s)))
    m = np.max(s)
    p = np.exp(s - m)
    l = p.sum()
    out = (p / l) @ v
    size = (p / l) @ np.abs(v)
    rel = 2 * eps + (len(j) + 64) * 2 * U + 2.0 ** -19
    bound = rel * size
    if fp16:
        bound = bound + 2.0 ** -11 * size + 2.0 ** -16 * np.abs(v).sum(0) / l + 2.0 ** -11 * (np.abs(out) + bound) + 2.0 ** -25
    lse = m + math.log(l)
    return out, lse, bound + 2 * U * np.abs(out), eps + (len(j) + 8) * 2 * U + 4 * U * max(1.0, abs(lse))


def frequencies(rot, base, scaling="plain", factor=1.0, original=0, low=1.0, high=4.0):
    """(radians per position of every pair, mscale)."""
    if scaling == "ntk":
        base = base * factor ** (rot / (rot - 2))
    f = np.array([base ** (-2.0 * i / rot) for i in range(rot // 2)])
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "yarn":
        at = lambda turns: rot * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(math.floor(at(low)), 0), min(math.ceil(at(high)), rot - 1)
        t = np.clip((np.arange(rot // 2) - lo) / max(hi - lo, 1e-3), 0, 1)
        return f * (1 - t) + f / factor * t, 0.1 * math.log(factor) + 1
    if scaling == "knees":
        s = np.clip((original * f / (2 * math.pi) - low) / (high - low), 0, 1)
        return f * s + f / factor * (1 - s), 1.0
    return f, 1.0


def norm_rope(x, pos, f, mscale, rot, interleaved, weight=None, eps=1e-6):
    """x [n][heads][d] float64 -> (z, bound on its fp16 rounding and fp32 arithmetic)."""
    y = x
    if weight is not None:
        y = x * weight / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    z, size = y.copy(), np.abs(y)
    if rot:
        a = pos[:, None] * f
        c, s = (mscale * np.cos(a))[:, None], (mscale * np.sin(a))[:, None]
        ia, ib = (np.arange(0, rot, 2), np.arange(1, rot, 2)) if interleaved else \
            (np.arange(rot // 2), np.arange(rot // 2) + rot // 2)
        u, v = y[..., ia], y[..., ib]
        z[..., ia], z[..., ib] = u * c - v * s, v * c + u * s
        both = mscale * (np.abs(u) + np.abs(v))
        size[..., ia], size[..., ib] = both, both
    # the norm (a sum of 128 squares, a root, two products), the angle (2^-24 turns = 2 pi u) and the
    # rotation: under 200 roundings of the pair's size
    return z, 200 * U * size + 2.0 ** -11 * np.abs(z) * (1 + 2.0 ** -10) + 2.0 ** -25


def as64(t):
    return t.detach().to("cpu").to(torch.float64).numpy()
