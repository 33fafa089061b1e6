"""GPU parity of kv_tree_attn against the plain 64-bit form: chains, stars and random trees, at every place of a page
and tile, under caps, slopes, windows, sinks and documents."""
import math

import numpy as np
import pytest
import torch

import latent_ref as LR
import new_token_ref as R
from compressed_kv_cache_quant_gb300 import _abi, kvq, synth
from gpu_helpers import paged_batch, require_gpu, ws

pytestmark = pytest.mark.gpu
D = 128


def rnd(shape, *ids, dtype=torch.float16, scale=1.0):
    return synth.normal(shape, synth.mix(synth.BASE_SEED, 9200, *ids), scale=scale, dtype=dtype)


def tree_of(kind, n, g):
    if kind == "chain":
        return list(range(-1, n - 1))
    if kind == "star":
        return [-1] * n
    if kind == "binary":
        return [(i - 1) // 2 if i else -1 for i in range(n)]
    return [-1 if i == 0 or g.random() < 0.1 else int(g.integers(max(0, i - 9), i)) for i in range(n)]


MODS = {
    "plain": {},
    "cap": dict(softcap=20.0),
    "bias": dict(bias=True),
    "cap_bias_scale": dict(softcap=5.0, bias=True, scale=0.2),
    "window": dict(window=37),
    "window_small": dict(window=3),
    "window_one_sink": dict(window=1, n_sink=5),
    "window_many_sinks": dict(window=2, n_sink=10 ** 6),
    "docs": dict(docs=True),
    "docs_window_sink_bias": dict(docs=True, window=4, n_sink=2, bias=True),
}


def check(lens, news, hq, hkv, kind, mod, seed=0, sample=None):
    require_gpu()
    g = np.random.default_rng(seed + 17 * len(lens) + sum(news))
    spec = dict(MODS[mod])
    B, rows = len(lens), sum(news)
    pool = sum(-(-t // 16) for t in lens) + 2 + B
    batch, bt = paged_batch([max(t, 1) for t in lens], kvq.Allocator(pool, seed=9), lengths=lens)
    cache = kvq.LayerCache(hq, hkv, 16, pool, B)
    cache.k16.fill_(float("nan"))   # whatever no sequence holds
    cache.v16.fill_(float("nan"))
    KV = [synth.kv_rows(t, hkv, synth.mix(seed, 50 + b)) for b, t in enumerate(lens)]
    for b, t in enumerate(lens):
        if t:
            kvq.kv_quant_pack(cache, batch, b, 0, t, KV[b][0].cuda(), KV[b][1].cuda())
    trees = [tree_of(kind, n, g) for n in news]
    q = rnd((rows + 2, hq, D), seed, rows).cuda()
    slopes = torch.tensor([2.0 ** (-8 * (h + 1) / hq) for h in range(hq)]) if spec.pop("bias", False) else None
    doc = None
    if spec.pop("docs", False):   # some begin among the nodes, some behind their query
        doc = np.array([int(g.integers(0, t + 2)) if i % 3 else max(0, t - n + i % 5 - 1) for t, n in zip(lens, news)
                        for i in range(n)] + [0, 0], dtype=np.int32)
    m = kvq.AttnMod(slopes=None if slopes is None else slopes.cuda(), doc_start=None if doc is None else torch.tensor(doc).cuda(),
                    **spec)
    out = torch.full((rows + 2, hq, D), -7.0, dtype=torch.float16, device="cuda")
    lse = torch.full((rows + 2, hq), -7.0, device="cuda")
    starts = torch.tensor(np.concatenate([[0], np.cumsum(news)]), dtype=torch.int32, device="cuda")
    par = torch.tensor([p for t in trees for p in t] + [5, 5], dtype=torch.int32, device="cuda")
    w = ws(kvq.kv_tree_attn_ws(cache, batch, rows + 2, max(news)))
    kvq.kv_tree_attn(cache, batch, q, par, starts, max(news), out, w, mod=m, lse=lse)
    kvq.kvq_check(w)
    first = (out.clone(), lse.clone())
    kvq.kv_tree_attn(cache, batch, q, par, starts, max(news), out, w, mod=m, lse=lse)
    assert torch.equal(first[0], out) and torch.equal(first[1], lse)
    assert not bool(w.t.any())   # left zeroed
    assert bool((out[rows:] == -7).all()) and bool((lse[rows:] == -7).all())
    row = 0
    for b, (t, n) in enumerate(zip(lens, news)):
        K, V = R.as64(KV[b][0]), R.as64(KV[b][1])
        pos = LR.key_positions(t, trees[b])
        for i in range(n):
            if sample is None or row in sample:
                seen = LR.tree_seen(t, trees[b], i, 0 if doc is None else int(doc[row]), spec.get("window", 0), spec.get("n_sink", 0))
                for h in range(hq):
                    kh = h // (hq // hkv)
                    bias = None if slopes is None else -float(slopes[h]) * np.abs(pos[t - n + i] - pos)
                    o, z, bo, bz = LR.attend(R.as64(q[row, h]), K[:, kh], V[:, kh], seen, spec.get("scale", 1 / math.sqrt(D)),
                                             spec.get("softcap", 0.0), bias)
                    assert np.all(np.abs(R.as64(out[row, h]) - o) <= bo), (b, i, h)
                    mine = float(lse[row, h])
                    assert mine == z if math.isinf(z) else abs(mine - z) <= bz, (b, i, h, mine, z)
            row += 1


@pytest.mark.parametrize("mod", list(MODS))
def test_score_forms(mod):
    check([150, 40, 257], [20, 9, 33], 4, 2, "random", mod, seed=1)


@pytest.mark.parametrize("kind", ["chain", "star", "binary", "random"])
@pytest.mark.parametrize("lens,news,hq,hkv", [
    ([1], [1], 1, 1),
    ([25], [25], 8, 1),                      # nothing but the tree
    ([130, 128, 129, 17], [3, 64, 1, 16], 8, 2),
    ([300], [256], 2, 1),                    # the most nodes
    ([513, 0, 64], [65, 0, 31], 2, 2),
])
def test_shapes(lens, news, hq, hkv, kind):
    check(lens, news, hq, hkv, kind, "plain", seed=2)


@pytest.mark.parametrize("mod", ["plain", "cap_bias_scale", "window"])
def test_long_split_contexts(mod):
    """Parts of the cache joined; sampled rows."""
    check([9001, 4096], [64, 7], 8, 2, "random", mod, seed=3, sample={0, 31, 63, 64, 70})


@pytest.mark.parametrize("mod", ["plain", "bias", "window", "window_one_sink", "docs_window_sink_bias"])
def test_many_parts(mod):
    """One or two row groups and long contexts: dozens of parts, of which a window or a document leaves few."""
    check([9001], [30], 8, 1, "random", mod, seed=4, sample={0, 13, 29})
    check([20000, 77], [8, 2], 8, 1, "binary", mod, seed=5, sample={7, 9})


def test_chain_is_kv_chunk_attn():
    """A chain is the causal run: the same bits, where both take the cache whole."""
    require_gpu()
    batch, _ = paged_batch([250], kvq.Allocator(70, seed=2))
    cache = kvq.LayerCache(8, 2, 16, 70, 1)
    kv = synth.kv_rows(250, 2, 77)
    kvq.kv_quant_pack(cache, batch, 0, 0, 250, kv[0].cuda(), kv[1].cuda())
    q = rnd((50, 8, D), 8).cuda()
    starts = torch.tensor([0, 50], dtype=torch.int32, device="cuda")
    a, b = torch.empty_like(q), torch.empty_like(q)
    w = ws(kvq.kv_tree_attn_ws(cache, batch, 50, 50))
    par = torch.arange(-1, 49, dtype=torch.int32, device="cuda")
    for mod in (None, kvq.AttnMod(window=30, n_sink=2)):
        kvq.kv_chunk_attn(cache, batch, q, starts, 50, a, w, mod=mod)
        kvq.kv_tree_attn(cache, batch, q, par, starts, 50, b, w, mod=mod)
        assert torch.equal(a, b)


def test_bad_parents_are_flagged():
    """An entry that is no earlier node counts as a root."""
    require_gpu()
    batch, _ = paged_batch([40], kvq.Allocator(8))
    cache = kvq.LayerCache(2, 1, 16, 8, 1)
    kv = synth.kv_rows(40, 1, 78)
    kvq.kv_quant_pack(cache, batch, 0, 0, 40, kv[0].cuda(), kv[1].cuda())
    q = rnd((4, 2, D), 9).cuda()
    starts = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    w = ws(kvq.kv_tree_attn_ws(cache, batch, 4, 4))
    got = []
    for par in ([-1, 1, 7, -9], [-1, -1, -1, -1]):
        out = torch.empty_like(q)
        kvq.kv_tree_attn(cache, batch, q, torch.tensor(par, dtype=torch.int32, device="cuda"), starts, 4, out, w)
        if par[1] == 1:
            with pytest.raises(kvq.KvqError) as e:
                kvq.kvq_check(w)
            assert e.value.code == _abi.KVQ_ERR_DEVICE_CHECK
        else:
            kvq.kvq_check(w)
        got.append(out)
    assert torch.equal(*got)
