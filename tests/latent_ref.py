"""Plain 64-bit forms of the appends, of tree attention and of the latent layers' attention, with the bounds that the
kernels' arithmetic allows.

Bounds.  u = 2^-24 is half an fp32 step.  A score is a sum of d exact products in fp32, in any order and perhaps
truncated: off by at most (d + 2) * 2u * sum|q_c k_c| * scale, and by 4u of its size behind that.  A weight is then off by
a factor within e^(+-2 eps) and 2^-20 for the exponential, a sum of n of them by n * 2u.  Rounding a weight once to
fp16 adds 2^-11 of it (and 2^-32 of the row's largest, taken here as 2^-31 of each value).  An fp16 output adds
2^-11 of itself and 2^-25."""
import math

import numpy as np

U = 2.0 ** -24


def paths(parents):
    """Ancestors of every node, itself last."""
    out = []
    for i, p in enumerate(parents):
        assert -1 <= p < i
        out.append((out[p] if p >= 0 else []) + [i])
    return out


def key_positions(T, parents):
    """Position of every token of a sequence whose last len(parents) ones are nodes of trees."""
    n = len(parents)
    return np.concatenate([np.arange(T - n), [T - n + len(p) - 1 for p in paths(parents)]]).astype(np.int64)


def tree_seen(T, parents, i, doc=0, window=0, n_sink=0):
    """Truth per token: what node i sees."""
    n = len(parents)
    pos = key_positions(T, parents)
    seen = np.zeros(T, bool)
    seen[:T - n] = True
    seen[[T - n + k for k in paths(parents)[i]]] = True
    here = pos[T - n + i]
    seen &= pos >= doc
    if window:
        seen &= (pos > here - window) | (pos < doc + n_sink)
    return seen


def attend(q, K, V, seen, scale, softcap=0.0, bias=None):
    """(out, lse, bound on out, bound on lse) of one query row over K [T][d], V [T][dv] (float64); bias: added per token."""
    j = np.nonzero(seen)[0]
    if len(j) == 0:
        return np.zeros(V.shape[1]), -math.inf, np.zeros(V.shape[1]), 0.0
    k, v = K[j], V[j]
    s = scale * (k @ q)
    eps = (len(q) + 2) * 2 * U * scale * np.max(np.abs(k) @ np.abs(q))
    if softcap:
        s = softcap * np.tanh(s / softcap)
        eps += 4 * U * softcap
    if bias is not None:
        s = s + bias[j]
    eps += 4 * U * max(1.0, np.max(np.abs(s)))
    m = np.max(s)
    p = np.exp(s - m)
    l = p.sum()
    out = (p / l) @ v
    size = (p / l) @ np.abs(v)
    bound = (2 * eps + (len(j) + 64) * 2 * U + 2.0 ** -19) * size
    bound = bound + 2.0 ** -11 * size + 2.0 ** -31 * np.abs(v).sum(0) / l + 2.0 ** -11 * (np.abs(out) + bound) + 2.0 ** -25
    lse = m + math.log(l)
    return out, lse, bound + 2 * U * np.abs(out), eps + (len(j) + 8) * 2 * U + 4 * U * max(1.0, abs(lse))


def e4m3(x):
    """Nearest E4M3 value (ties to even), finite values saturating at +-448, and half its step."""
    x = np.clip(np.asarray(x, dtype=np.float64), -448.0, 448.0)
    e = np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -6)))
    step = 2.0 ** (e - 3)
    return np.clip(np.round(x / step) * step, -448.0, 448.0), step / 2


def e4m3_value(code):
    """The values of E4M3 bytes."""
    c = np.asarray(code).astype(np.int64)
    e, f = (c >> 3) & 15, c & 7
    v = np.where(e > 0, (1 + f / 8.0) * 2.0 ** (e - 7.0), f / 8.0 * 2.0 ** -6)
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c & 128, -v, v)
