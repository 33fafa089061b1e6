"""GPU parity of the latent layers' attention, absorbed and expanded, against the plain 64-bit form."""
import math

import numpy as np
import pytest
import torch

import latent_ref as LR
import new_token_ref as R
from compressed_kv_cache_quant_gb300 import kvq, synth
from gpu_helpers import paged_batch, require_gpu, ws
from test_gpu_tree import tree_of

pytestmark = pytest.mark.gpu
D, LAT, ROT, ROW = 128, 512, 64, 576
SCALE = 1 / math.sqrt(192)


def rnd(shape, *ids, dtype=torch.float16, scale=1.0):
    return synth.normal(shape, synth.mix(synth.BASE_SEED, 9300, *ids), scale=scale, dtype=dtype)


def absorbed(lens, news, heads, kind=None, seed=0, scale=0.0, sample=None, q_scale=1.0):
    require_gpu()
    g = np.random.default_rng(seed + sum(news))
    B, rows = len(lens), sum(news)
    pool = sum(-(-t // 16) for t in lens) + 2 + B
    batch, bt = paged_batch([max(t, 1) for t in lens], kvq.Allocator(pool, seed=9), lengths=lens)
    cache = kvq.LatentCache(pool)
    cache.rows.fill_(float("nan"))   # whatever no sequence holds
    lat = [rnd((t, ROW), seed, 50 + b) for b, t in enumerate(lens)]
    for b, t in enumerate(lens):
        for p in range(-(-t // 16)):
            part = lat[b][16 * p:16 * p + 16].cuda()
            cache.rows[bt[b, p], :len(part)] = part
    q = rnd((rows + 2, heads, ROW), seed, rows, scale=q_scale).cuda()
    trees = [tree_of(kind or "chain", n, g) for n in news]
    par = torch.tensor([p for t in trees for p in t] + [5, 5], dtype=torch.int32, device="cuda") if kind else None
    out = torch.full((rows + 2, heads, LAT), -7.0, dtype=torch.float16, device="cuda")
    lse = torch.full((rows + 2, heads), -7.0, device="cuda")
    starts = torch.tensor(np.concatenate([[0], np.cumsum(news)]), dtype=torch.int32, device="cuda")
    w = ws(kvq.kv_latent_attn_ws(batch, heads, rows + 2, max(news)))
    call = lambda: kvq.kv_latent_attn(cache, batch, q, starts, max(news), out, w, scale=scale, parents=par, lse=lse)  # noqa: E731
    call()
    kvq.kvq_check(w)
    first = (out.clone(), lse.clone())
    call()
    assert torch.equal(first[0], out) and torch.equal(first[1], lse)
    assert not bool(w.t.any())   # left zeroed
    assert bool((out[rows:] == -7).all()) and bool((lse[rows:] == -7).all())
    row = 0
    for b, (t, n) in enumerate(zip(lens, news)):
        K = R.as64(lat[b])
        for i in range(n):
            if sample is None or row in sample:
                seen = LR.tree_seen(t, trees[b], i)
                for h in range(heads):
                    o, z, bo, bz = LR.attend(R.as64(q[row, h]), K, K[:, :LAT], seen, scale or SCALE)
                    assert np.all(np.abs(R.as64(out[row, h]) - o) <= bo), (b, i, h)
                    assert abs(float(lse[row, h]) - z) <= bz, (b, i, h)
            row += 1


@pytest.mark.parametrize("lens,news,heads", [
    ([1], [1], 1),
    ([1, 2, 15, 16, 17], [1, 1, 1, 1, 1], 16),
    ([63, 64, 65, 0, 129], [1, 1, 1, 0, 1], 8),
    ([200, 77], [3, 5], 12),
    ([300], [1], 128),
    ([90, 131], [4, 2], 64),
    ([65], [65], 3),
    ([140], [2], 130),
    ([129, 64], [5, 1], 20),
])
def test_absorbed(lens, news, heads):
    absorbed(lens, news, heads, seed=1)


@pytest.mark.parametrize("kind", ["star", "random"])
@pytest.mark.parametrize("lens,news,heads", [([25], [25], 8), ([130, 33], [7, 20], 16), ([300], [256], 1), ([70], [5], 128)])
def test_absorbed_trees(lens, news, heads, kind):
    absorbed(lens, news, heads, kind, seed=2)


def test_absorbed_long_and_ragged():
    """Parts of the cache joined: sampled rows."""
    absorbed([9001, 130, 1, 4096], [1, 1, 1, 1], 16, seed=3)
    absorbed([5000, 2049], [5, 2], 32, seed=4, sample={0, 4, 6})
    absorbed([4097, 800], [2, 1], 128, seed=5, sample={1, 2})


@pytest.mark.parametrize("lens,news,heads", [
    ([288, 1, 287], [1, 1, 1], 16),        # six steps of 48 tokens: not cut; one token more: cut
    ([289, 1, 287], [1, 1, 1], 16),
    ([384, 5, 129], [2, 2, 1], 64),        # six steps of 64 for more than 32 rows
    ([385, 5, 129], [2, 2, 1], 64),
    ([96] * 200, [1] * 200, 1),            # more row groups than SMs
    ([200, 0, 150], [1, 0, 2], 16),
])
def test_absorbed_short(lens, news, heads):
    absorbed(lens, news, heads, seed=7)


def test_absorbed_short_tree():
    absorbed([130, 288, 60], [25, 7, 1], 2, "random", seed=8)


def test_absorbed_joins():
    """Parts joined by a cluster per row and by a warp per row, up to 256 rows of row groups and beyond."""
    absorbed([1119, 900, 182, 600, 700, 333, 800, 1000, 450], [1] * 9, 12, seed=9, sample={0, 2, 8})
    absorbed([700] * 14, [1] * 14, 16, seed=10, sample={0, 13})
    absorbed([3000, 2000], [1, 1], 128, seed=11, sample={0, 1})
    absorbed([1500] * 17, [1] * 17, 16, seed=12, sample={0, 16})


def test_absorbed_scores_of_every_size():
    """Flat, sharp and far scores."""
    for s, scale in ((0.01, 0.0), (8.0, 0.0), (30.0, 0.5), (1.0, 1e-6)):
        absorbed([333], [2], 4, seed=6, q_scale=s, scale=scale)


def expanded(lens, news, heads, seed=0, gap=0, scale=0.0, sample=None):
    """gap: rows between the sequences' keys that belong to none."""
    require_gpu()
    B, rows = len(lens), sum(news)
    k_starts = np.concatenate([[gap], gap + np.cumsum(lens)]).astype(np.int32)
    m = int(k_starts[-1]) + gap
    kv = rnd((m, heads, 2 * D + 8), seed, m).cuda()
    lat = rnd((m, ROW), seed, m, 1).cuda()
    kn, v, kr = kv[..., :D], kv[..., D:2 * D], lat[:, LAT:]
    if gap:
        for x in (kv, lat):
            x[:gap] = float("nan")
            x[m - gap:] = float("nan")
    q = rnd((rows + 2, heads, D + ROT), seed, rows, 2).cuda()
    out = torch.full((rows + 2, heads, D), -7.0, dtype=torch.float16, device="cuda")
    lse = torch.full((rows + 2, heads), -7.0, device="cuda")
    qs = torch.tensor(np.concatenate([[0], np.cumsum(news)]), dtype=torch.int32, device="cuda")
    ks = torch.tensor(k_starts, device="cuda")
    w = ws(kvq.kv_latent_expanded_attn_ws(B, heads, rows + 2, max(news), max(lens)))
    for _ in range(2):
        kvq.kv_latent_expanded_attn(q, kn, kr, v, qs, ks, max(news), max(lens), out, w, scale=scale, lse=lse)
    kvq.kvq_check(w)
    assert not bool(w.t.any())
    assert bool((out[rows:] == -7).all()) and bool((lse[rows:] == -7).all())
    row = 0
    for b, (t, n) in enumerate(zip(lens, news)):
        at = slice(int(k_starts[b]), int(k_starts[b]) + t)
        for h in range(heads):
            K = np.concatenate([R.as64(kn[at, h]), R.as64(kr[at])], -1)
            V = R.as64(v[at, h])
            for i in range(n):
                if sample is None or row + i in sample:
                    seen = np.arange(t) <= t - n + i
                    o, z, bo, bz = LR.attend(R.as64(q[row + i, h]), K, V, seen, scale or SCALE)
                    assert np.all(np.abs(R.as64(out[row + i, h]) - o) <= bo), (b, i, h)
                    assert abs(float(lse[row + i, h]) - z) <= bz, (b, i, h)
        row += n


@pytest.mark.parametrize("lens,news,heads,gap", [
    ([1], [1], 1, 0),
    ([127, 128, 129], [127, 128, 129], 2, 0),
    ([300, 5, 0, 64], [40, 5, 0, 1], 3, 7),
    ([600], [257], 1, 3),
    ([70, 33], [70, 20], 16, 1),
])
def test_expanded(lens, news, heads, gap):
    expanded(lens, news, heads, seed=1, gap=gap)


def test_expanded_long():
    expanded([3000, 1025], [1500, 1025], 2, seed=2, sample={0, 1, 255, 256, 1499, 1500, 2000, 2524})


def test_expanded_many_groups():
    """More groups of queries than SMs, of one and two tiles in turn and with sequences that have none: a CTA works through
    several of them."""
    lens = [(37 * b) % 401 + 1 for b in range(41)] + [900, 0, 128]
    news = [t if b % 3 else min(t, b % 5) for b, t in enumerate(lens)]
    rows = sum(news)
    expanded(lens, news, 16, seed=4, gap=5, sample={0, rows // 3, rows // 2, rows - 129, rows - 1})
    expanded([2300, 1], [2300, 1], 70, seed=5, sample={0, 1023, 2299, 2300})


def test_expanded_runs_alike():
    """Which CTA takes which group differs from run to run, the results do not."""
    require_gpu()
    lens, heads = [700, 129, 2000, 31, 256], 24
    starts = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    m = sum(lens)
    kv, lat, q = rnd((m, heads, 2 * D), 1).cuda(), rnd((m, ROW), 2).cuda(), rnd((m, heads, D + ROT), 3).cuda()
    w = ws(kvq.kv_latent_expanded_attn_ws(len(lens), heads, m, max(lens), max(lens)))
    first = None
    for _ in range(20):
        out = torch.empty((m, heads, D), dtype=torch.float16, device="cuda")
        lse = torch.empty((m, heads), device="cuda")
        kvq.kv_latent_expanded_attn(q, kv[..., :D], lat[:, LAT:], kv[..., D:], starts, starts, max(lens), max(lens), out, w, lse=lse)
        if first is None:
            first = out, lse
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    kvq.kvq_check(w)


def test_expanded_scales():
    for scale in (1e-6, 0.6, 3.0):
        expanded([200], [130], 1, seed=3, scale=scale)


def test_the_two_forms_agree():
    """One layer, absorbed and expanded by the same up-projections: the same attention within fp16 roundings."""
    require_gpu()
    H, T, n = 4, 100, 6
    lat = (rnd((T, ROW), 1).float() / 4).half().cuda()
    up_k, up_v = rnd((H, D, LAT), 2, dtype=torch.float32, scale=LAT ** -0.5).cuda(), rnd((H, D, LAT), 3, dtype=torch.float32, scale=LAT ** -0.5).cuda()
    q = rnd((n, H, D + ROT), 4).cuda()
    batch, bt = paged_batch([T], kvq.Allocator(8, seed=1))
    cache = kvq.LatentCache(8)
    for p in range(-(-T // 16)):
        part = lat[16 * p:16 * p + 16]
        cache.rows[bt[0, p], :len(part)] = part
    starts = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    c = lat[:, :LAT].float()
    kn = torch.einsum("tc,hdc->thd", c, up_k).half()
    v = torch.einsum("tc,hdc->thd", c, up_v).half()
    a = torch.empty((n, H, D), dtype=torch.float16, device="cuda")
    w = ws(kvq.kv_latent_expanded_attn_ws(1, H, n, n, T))
    kvq.kv_latent_expanded_attn(q, kn, lat[:, LAT:], v, starts, torch.tensor([0, T], dtype=torch.int32, device="cuda"), n, T, a, w)
    qa = torch.cat([torch.einsum("nhd,hdc->nhc", q[..., :D].float(), up_k), q[..., D:].float()], -1).half()
    o = torch.empty((n, H, LAT), dtype=torch.float16, device="cuda")
    w = ws(kvq.kv_latent_attn_ws(batch, H, n, n))
    kvq.kv_latent_attn(cache, batch, qa, starts, n, o, w)
    b = torch.einsum("nhc,hdc->nhd", o.float(), up_v)
    # keys, queries and outputs rounded to fp16 on either way: scores of size 1 off by under 2^-9, values by 2^-10
    assert float((a.float() - b).norm() / b.norm()) <= 2.0 ** -7
