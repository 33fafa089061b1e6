"""Outputs that begin on a 16-byte and no 32-byte boundary, as a slice of a larger buffer does: the bits of an aligned call,
and nothing around them is touched."""
import numpy as np
import pytest
import torch

from compressed_kv_cache_quant_gb300 import kvq, synth
from gpu_helpers import paged_batch, require_gpu, ws

pytestmark = pytest.mark.gpu
D, LAT, ROT, ROW = 128, 512, 64, 576


def rnd(shape, *ids):
    return synth.normal(shape, synth.mix(synth.BASE_SEED, 9500, *ids), scale=1.0, dtype=torch.float16).cuda()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def both(shape, call):
    """call(out) into an aligned tensor and into one 16 bytes further on."""
    n = int(np.prod(shape))
    plain = torch.empty(shape, dtype=torch.float16, device="cuda")
    call(plain)
    buf = torch.full((n + 24,), -7.0, dtype=torch.float16, device="cuda")
    out = buf[8:8 + n].view(shape)
    assert plain.data_ptr() % 32 == 0 and out.data_ptr() % 32 == 16
    call(out)
    assert torch.equal(plain, out) and not bool((plain == 0).all())
    assert bool((buf[:8] == -7).all()) and bool((buf[8 + n:] == -7).all())


@pytest.mark.parametrize("lens,news", [([400, 129], [70, 129]), ([9001], [30])])   # whole; in parts
@pytest.mark.parametrize("op", ["run", "tree"])
def test_runs_and_trees(op, lens, news):
    require_gpu()
    hq, hkv, n, B = 8, 2, sum(news), len(lens)
    pool = sum(-(-t // 16) for t in lens) + 2
    batch, _ = paged_batch(lens, kvq.Allocator(pool, seed=9))
    cache = kvq.LayerCache(hq, hkv, 16, pool, B)
    for b, t in enumerate(lens):
        kvq.kv_quant_pack(cache, batch, b, 0, t, rnd((t, hkv, D), b, 1), rnd((t, hkv, D), b, 2))
    q, starts = rnd((n, hq, D), 3), i32(np.concatenate([[0], np.cumsum(news)]))
    par = i32([(i - 1) // 2 if i else -1 for m in news for i in range(m)])
    w = ws(max(kvq.kv_chunk_attn_ws(cache, batch, n, max(news)), kvq.kv_tree_attn_ws(cache, batch, n, max(news))))
    if op == "run":
        both((n, hq, D), lambda out: kvq.kv_chunk_attn(cache, batch, q, starts, max(news), out, w))
    else:
        both((n, hq, D), lambda out: kvq.kv_tree_attn(cache, batch, q, par, starts, max(news), out, w))
    kvq.kvq_check(w)


@pytest.mark.parametrize("lens,news,heads", [([300, 129], [300, 40], 3), ([9001], [30], 2)])
def test_expanded(lens, news, heads):
    require_gpu()
    m, n, B = sum(lens), sum(news), len(lens)
    kv, kr, q = rnd((m, heads, 2 * D), 1), rnd((m, ROT), 2), rnd((n, heads, D + ROT), 3)
    qs, ks = i32(np.concatenate([[0], np.cumsum(news)])), i32(np.concatenate([[0], np.cumsum(lens)]))
    w = ws(kvq.kv_latent_expanded_attn_ws(B, heads, n, max(news), max(lens)))
    both((n, heads, D), lambda out: kvq.kv_latent_expanded_attn(q, kv[..., :D], kr, kv[..., D:], qs, ks, max(news), max(lens), out, w))
    kvq.kvq_check(w)


@pytest.mark.parametrize("lens,heads", [([200], 16), ([6000, 77], 16), ([200], 128), ([6000, 77], 64)])   # whole and in parts, alone and in pairs
def test_absorbed(lens, heads):
    require_gpu()
    B = len(lens)
    pool = sum(-(-t // 16) for t in lens) + 2
    batch, _ = paged_batch(lens, kvq.Allocator(pool, seed=9))
    cache = kvq.LatentCache(pool)
    cache.rows.copy_(rnd((pool, 16, ROW), 4))
    q, starts = rnd((B, heads, ROW), 5), i32(list(range(B + 1)))
    w = ws(kvq.kv_latent_attn_ws(batch, heads, B, 1))
    both((B, heads, LAT), lambda out: kvq.kv_latent_attn(cache, batch, q, starts, 1, out, w))
    kvq.kvq_check(w)


@pytest.mark.parametrize("t_cap", [0, 512])   # a plain fp16 layer and a scored one
def test_appended_queries(t_cap):
    require_gpu()
    T, hq, hkv = 77, 8, 2
    batch, _ = paged_batch([T], kvq.Allocator(8, seed=9))
    layer = kvq.LayerCache(hq, hkv, 16, 8, 1, t_cap=t_cap)
    q, k, v = rnd((T, hq, D), 6), rnd((T, hkv, D), 7), rnd((T, hkv, D), 8)
    tab, w = kvq.RopeTable(D), ws(kvq.kv_rope_append_ws())
    both((T, hq, D), lambda out: kvq.kv_rope_append(layer, batch, tab, i32([0, T]), q, k, v, out, w))
    kvq.kvq_check(w)
