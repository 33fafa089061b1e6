"""GPU tests of tree attention and of the latent layers' attention with scores far beyond 2^24, where neighbouring fp32
values are more than a step of the exponent apart."""
import math

import numpy as np
import pytest
import torch

import latent_ref as LR
import new_token_ref as R
from compressed_kv_cache_quant_gb300 import kvq
from gpu_helpers import paged_batch, require_gpu, ws
from test_gpu_tree import tree_of

pytestmark = pytest.mark.gpu
D, LAT, ROT, ROW = 128, 512, 64, 576


def rnd(shape, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed))


def far(K_shape, q_shape, sign, seed):
    """fp16 keys and queries: scores of both signs, or all of them negative."""
    if sign == "both":
        return (rnd(K_shape, seed) * 20000).clamp(-60000, 60000).half(), (rnd(q_shape, seed + 1) * 20000).clamp(-60000, 60000).half()
    return ((rnd(K_shape, seed) * 0.3 + 1) * 20000).clamp(-60000, 60000).half(), torch.full(q_shape, -20000.0).half()


def largest_takes_all(q, K, V, seen, scale, out, lse):
    """The row's largest score takes all the weight, so that its value comes out to the last bit; False where two of them lie
    too close to tell."""
    k = K[seen]
    s = scale * (k @ q)
    eps = (len(q) + 2) * 2 * R.U * scale * np.max(np.abs(k) @ np.abs(q))
    at = int(np.argmax(s))
    others = np.delete(s, at)
    if len(others) and s[at] - others.max() < 4 * eps:
        return False
    assert bool((R.as64(out) == V[seen][at]).all())
    assert abs(float(lse) - s[at]) <= 2 * eps + 1e-6 * abs(s[at])
    return True


@pytest.mark.parametrize("sign", ["both", "negative"])
@pytest.mark.parametrize("hq,hkv,lens,news", [
    (8, 2, [150, 700], [130, 70]),     # nodes in two tiles, behind little and behind some context
    (2, 1, [300], [256]),
    (8, 1, [9001], [30]),              # parts joined
])
def test_trees_of_far_scores(hq, hkv, lens, news, sign):
    require_gpu()
    B, n, g = len(lens), sum(news), np.random.default_rng(sum(lens))
    pool = sum(-(-t // 16) for t in lens) + 2
    batch, _ = paged_batch(lens, kvq.Allocator(pool, seed=9))
    cache = kvq.LayerCache(hq, hkv, 16, pool, B)
    KV = []
    for b, t in enumerate(lens):
        K, q = far((t, hkv, D), (n, hq, D), sign, 10 + b)
        KV.append((K, rnd((t, hkv, D), 30 + b).half()))
        kvq.kv_quant_pack(cache, batch, b, 0, t, K.cuda(), KV[b][1].cuda())
    trees = [tree_of("random", m, g) for m in news]
    q, out = q.cuda(), torch.empty((n, hq, D), dtype=torch.float16, device="cuda")
    lse = torch.empty((n, hq), device="cuda")
    starts = torch.tensor(np.concatenate([[0], np.cumsum(news)]), dtype=torch.int32, device="cuda")
    par = torch.tensor([p for t in trees for p in t], dtype=torch.int32, device="cuda")
    w = ws(kvq.kv_tree_attn_ws(cache, batch, n, max(news)))
    kvq.kv_tree_attn(cache, batch, q, par, starts, max(news), out, w, lse=lse)
    kvq.kvq_check(w)
    row = told = 0
    for b, (t, m) in enumerate(zip(lens, news)):
        K, V = R.as64(KV[b][0]), R.as64(KV[b][1])
        for i in range(m):
            for h in range(hq):
                kh = h // (hq // hkv)
                told += largest_takes_all(R.as64(q[row, h]), K[:, kh], V[:, kh], LR.tree_seen(t, trees[b], i), 1 / math.sqrt(D), out[row, h],
                                          lse[row, h])
            row += 1
    assert told > n * hq // 4


@pytest.mark.parametrize("sign", ["both", "negative"])
def test_expanded_far_scores(sign):
    """More groups of queries than SMs, of one and of two tiles, several per CTA."""
    require_gpu()
    lens, H = [700, 129, 1000, 31, 256], 40
    m, starts = sum(lens), np.concatenate([[0], np.cumsum(lens)])
    at = torch.tensor(starts, dtype=torch.int32, device="cuda")
    K, q = far((m, H, D + ROT), (m, H, D + ROT), sign, 50)
    K[:, :, D:] = K[:, :1, D:]   # (shared by the heads)
    V = rnd((m, H, D), 60).half()
    kn, kr = K[..., :D].contiguous().cuda(), K[:, 0, D:].contiguous().cuda()
    out, lse = torch.empty((m, H, D), dtype=torch.float16, device="cuda"), torch.empty((m, H), device="cuda")
    w = ws(kvq.kv_latent_expanded_attn_ws(len(lens), H, m, max(lens), max(lens)))
    kvq.kv_latent_expanded_attn(q.cuda(), kn, kr, V.cuda(), at, at, max(lens), max(lens), out, w, lse=lse)
    kvq.kvq_check(w)
    told = rows = 0
    for b, t in enumerate(lens):
        here = slice(int(starts[b]), int(starts[b]) + t)
        for h in (0, 17, H - 1):
            k, v = R.as64(K[here, h]), R.as64(V[here, h])
            for i in range(0, t, 37):
                rows += 1
                told += largest_takes_all(R.as64(q[here][i, h]), k, v, np.arange(t) <= i, 1 / math.sqrt(192), out[here][i, h], lse[here][i, h])
    assert told > rows // 4


@pytest.mark.parametrize("sign", ["both", "negative"])
@pytest.mark.parametrize("heads,lens,news", [(4, [333, 60], [2, 1]), (16, [5000], [1]), (64, [700, 90], [3, 5]), (128, [3001], [1])])
def test_absorbed_far_scores(heads, lens, news, sign):
    require_gpu()
    n = sum(news)
    pool = sum(-(-t // 16) for t in lens) + 2
    batch, bt = paged_batch(lens, kvq.Allocator(pool, seed=9))
    cache = kvq.LatentCache(pool)
    rows = []
    for b, t in enumerate(lens):
        K, q = far((t, ROW), (n, heads, ROW), sign, 70 + b)
        rows.append(K)
        for p in range(-(-t // 16)):
            part = K[16 * p:16 * p + 16].cuda()
            cache.rows[bt[b, p], :len(part)] = part
    q, out = q.cuda(), torch.empty((n, heads, LAT), dtype=torch.float16, device="cuda")
    lse = torch.empty((n, heads), device="cuda")
    starts = torch.tensor(np.concatenate([[0], np.cumsum(news)]), dtype=torch.int32, device="cuda")
    w = ws(kvq.kv_latent_attn_ws(batch, heads, n, max(news)))
    kvq.kv_latent_attn(cache, batch, q, starts, max(news), out, w, lse=lse)
    kvq.kvq_check(w)
    row = told = 0
    for b, (t, m) in enumerate(zip(lens, news)):
        K = R.as64(rows[b])
        for i in range(m):
            for h in range(heads):
                told += largest_takes_all(R.as64(q[row, h]), K, K[:, :LAT], np.arange(t) <= t - m + i, 1 / math.sqrt(192), out[row, h], lse[row, h])
            row += 1
    assert told > n * heads // 4


@pytest.mark.parametrize("op,heads,lens,news", [
    ("absorbed", 16, [40, 700], [1, 2]), ("absorbed", 8, [20001], [1]), ("absorbed", 64, [130, 700], [3, 2]), ("absorbed", 128, [9001], [1]),
    ("expanded", 3, [40, 700], [40, 300]), ("expanded", 2, [9001], [3]), ("tree", 8, [150, 700], [130, 9]), ("tree", 8, [9001], [30]),
])
def test_nan_in_a_query(op, heads, lens, news):
    """NaN in one head of one query gives NaN in that row, and changes no bit of any other."""
    require_gpu()
    B, n, m = len(lens), sum(news), sum(lens)
    pool = sum(-(-t // 16) for t in lens) + 2
    batch, _ = paged_batch(lens, kvq.Allocator(pool, seed=9))
    starts = torch.tensor(np.concatenate([[0], np.cumsum(news)]), dtype=torch.int32, device="cuda")
    if op == "absorbed":
        dq, dv, cache = ROW, LAT, kvq.LatentCache(pool)
        cache.rows.copy_(rnd(cache.rows.shape, 1))
        w = ws(kvq.kv_latent_attn_ws(batch, heads, n, max(news)))
        call = lambda q, out, lse: kvq.kv_latent_attn(cache, batch, q, starts, max(news), out, w, lse=lse)  # noqa: E731
    elif op == "tree":
        dq, dv, cache = D, D, kvq.LayerCache(heads, 2, 16, pool, B)
        cache.k16.copy_(rnd(cache.k16.shape, 1))
        cache.v16.copy_(rnd(cache.v16.shape, 2))
        par = torch.tensor([(i - 1) // 2 if i else -1 for k in news for i in range(k)], dtype=torch.int32, device="cuda")
        w = ws(kvq.kv_tree_attn_ws(cache, batch, n, max(news)))
        call = lambda q, out, lse: kvq.kv_tree_attn(cache, batch, q, par, starts, max(news), out, w, lse=lse)  # noqa: E731
    else:
        dq, dv = D + ROT, D
        kv, kr = rnd((m, heads, 2 * D), 1).half().cuda(), rnd((m, ROT), 2).half().cuda()
        at = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
        w = ws(kvq.kv_latent_expanded_attn_ws(B, heads, n, max(news), max(lens)))
        call = lambda q, out, lse: kvq.kv_latent_expanded_attn(q, kv[..., :D], kr, kv[..., D:], starts, at, max(news), max(lens), out, w, lse=lse)  # noqa: E731
    q = rnd((n, heads, dq), 5).half().cuda()
    got = []
    for bad in (False, True):
        if bad:
            q[n - 1, 1, 5] = math.nan
        out, lse = torch.empty((n, heads, dv), dtype=torch.float16, device="cuda"), torch.empty((n, heads), device="cuda")
        call(q, out, lse)
        got.append((out, lse))
    kvq.kvq_check(w)
    hit = torch.zeros((n, heads), dtype=torch.bool, device="cuda")
    hit[n - 1, 1] = True
    (clean, clean_lse), (out, lse) = got
    assert bool(out[hit].isnan().all()) and bool(lse[hit].isnan().all())
    assert torch.equal(out[~hit], clean[~hit]) and torch.equal(lse[~hit], clean_lse[~hit]) and not bool(clean.isnan().any())
    assert not bool(w.t.any())   # left zeroed, NaN included
