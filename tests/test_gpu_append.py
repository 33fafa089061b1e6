"""GPU parity of kv_rope_append and kv_latent_append against plain 64-bit forms: every type, layout and cache, ragged
runs, rows that must stay as they were, and what the device checks skip."""
import numpy as np
import pytest
import torch

import latent_ref as LR
import new_token_ref as R
from compressed_kv_cache_quant_gb300 import _abi, kvq, synth
from gpu_helpers import paged_batch, require_gpu, ws

pytestmark = pytest.mark.gpu
D, LAT, ROT, ROW = 128, 512, 64, 576


def rnd(shape, *ids, dtype=torch.float16, scale=1.0):
    return synth.normal(shape, synth.mix(synth.BASE_SEED, 9100, *ids), scale=scale, dtype=dtype)


def starts_of(news, at=0):
    return torch.tensor(np.concatenate([[at], at + np.cumsum(news)]), dtype=torch.int32, device="cuda")


def places(lens, news):
    """(sequence, place) of every row."""
    return [(b, t - n + i) for b, (t, n) in enumerate(zip(lens, news)) for i in range(n)]


@pytest.mark.parametrize("lens,news,hq,hkv,dt,cache,norm,rot,inter", [
    ([1], [1], 8, 2, torch.float16, "f16", False, 128, False),
    ([40, 17, 5, 100], [1, 1, 1, 1], 32, 8, torch.bfloat16, "e4m3", True, 128, False),
    ([33, 0, 64, 200, 16], [33, 0, 3, 129, 0], 5, 3, torch.float16, "f16", True, 64, True),
    ([130, 77], [67, 77], 4, 4, torch.bfloat16, "scored", False, 96, False),
    ([300, 9, 64, 65, 128], [200, 1, 64, 2, 63], 8, 1, torch.float16, "scored", True, 32, True),
    ([1500], [1400], 2, 1, torch.float16, "e4m3", False, 16, False),
    ([70, 30], [5, 30], 40, 40, torch.bfloat16, "f16", True, 0, False),
    ([5000], [4999], 2, 2, torch.bfloat16, "scored", True, 128, True),
    ([20] * 75, [1, 3, 0] * 25, 4, 2, torch.float16, "f16", False, 128, False),
])
def test_rope_append(lens, news, hq, hkv, dt, cache, norm, rot, inter):
    require_gpu()
    B, rows, extra = len(lens), sum(news), 3
    batch, bt = paged_batch([max(t, 1) for t in lens], kvq.Allocator(sum(-(-max(t, 1) // 16) for t in lens) + 2, seed=5),
                            lengths=lens)
    pool = sum(-(-max(t, 1) // 16) for t in lens) + 2
    cap = (max(lens) + 7) // 8 * 8 if cache == "scored" else 0
    layer = kvq.LayerCache(hq, hkv, kvq.BITS_E4M3 if cache == "e4m3" else 16, pool, B, t_cap=cap)
    pages = [layer.k_codes, layer.v_codes] if cache == "e4m3" else [layer.k16, layer.v16]
    for p in pages:
        p.fill_(7)
    if cap:
        layer.kT.fill_(7)
        layer.k_absmax.fill_(1.5)
    x = rnd((rows + extra, (hq + 2 * hkv) * D + 8), rows, hq, dtype=dt).cuda()   # slices of wider rows
    q = x[:, :hq * D].view(-1, hq, D)
    k = x[:, hq * D:(hq + hkv) * D].view(-1, hkv, D)
    v = x[:, (hq + hkv) * D:(hq + 2 * hkv) * D].view(-1, hkv, D)
    if cache == "e4m3":
        v[0, 0, :4] = torch.tensor([449.0, -1e4, float("inf"), 1e-4], dtype=dt)
    wq, wk = ((rnd((D,), 1, dtype=torch.float32) + 2).cuda(), (rnd((D,), 2, dtype=torch.float32) + 2).cuda()) if norm else (None, None)
    q_out = torch.full((rows + extra, hq, D), -7.0, dtype=torch.float16, device="cuda")
    tab = kvq.RopeTable(rot, 500000.0, interleaved=inter)
    pos = None
    where = places(lens, news)
    at = np.array([p for _, p in where])
    if B % 2:   # positions of the caller's own, as a tree's
        at = 100000 - 3 * at
        pos = torch.tensor(np.concatenate([at, [0] * extra]), dtype=torch.int32, device="cuda")
    w = ws(kvq.kv_rope_append_ws())
    kvq.kv_rope_append(layer, batch, tab, starts_of(news), q, k, v, q_out, w, positions=pos, q_weight=wq, k_weight=wk, eps=1e-5)
    kvq.kvq_check(w)
    f = R.frequencies(rot, 500000.0)[0] if rot else np.zeros(0)
    as_w = lambda t: None if t is None else R.as64(t)  # noqa: E731
    zq, bq = R.norm_rope(R.as64(q[:rows]), at, f, 1.0, rot, inter, as_w(wq), 1e-5)
    zk, bk = R.norm_rope(R.as64(k[:rows]), at, f, 1.0, rot, inter, as_w(wk), 1e-5)
    assert np.all(np.abs(R.as64(q_out[:rows]) - zq) <= bq)
    assert bool((q_out[rows:] == -7).all())
    written = np.zeros((pool, 16), bool)
    got = [p.cpu().numpy() for p in pages]
    for r, (b, p) in enumerate(where):
        page, slot = bt[b, p // 16], p % 16
        written[page, slot] = True
        if cache == "e4m3":
            zv = R.as64(v[r])
            for mine, z, slack in ((got[0][page, :, slot], zk[r], 200 * R.U * 4 * np.abs(zk[r]).max()),
                                   (got[1][page, :, slot], zv, 0.0)):
                near, half = LR.e4m3(z)
                assert np.all(np.abs(LR.e4m3_value(mine) - np.clip(z, -448, 448)) <= half + slack)
                if not slack:
                    assert np.array_equal(LR.e4m3_value(mine), near)
        else:
            assert np.all(np.abs(got[0][page, :, slot].astype(np.float64) - zk[r]) <= bk[r])
            assert torch.equal(pages[1][page, :, slot], v[r].half())
    for g in got:   # nothing else is touched
        assert np.all(g.transpose(0, 2, 1, 3)[~written] == 7)
    if cap:
        kT, top = layer.kT.cpu(), layer.k_absmax.cpu()
        k16 = layer.k16.cpu()
        for b, (t, n) in enumerate(zip(lens, news)):
            new = torch.stack([k16[bt[b, p // 16], :, p % 16] for p in range(t - n, t)], -1) if n else kT[b, :, :, :0]
            assert torch.equal(kT[b, :, :, t - n:t], new)
            assert bool((kT[b, :, :, :t - n] == 7).all()) and bool((kT[b, :, :, t:] == 7).all())
            want = new.float().abs().amax(-1).clamp(min=1.5) if n else torch.full((hkv, D), 1.5)
            assert torch.equal(top[b], want)


@pytest.mark.parametrize("lens,news,hq,hkv,dt,norm,rot,inter", [
    ([50], [9], 24, 12, torch.bfloat16, True, 128, True),
    ([100, 7], [100, 1], 10, 5, torch.float16, False, 64, False),
    ([800, 33], [790, 20], 40, 40, torch.bfloat16, True, 96, False),
    ([33] * 40, [1] * 40, 32, 8, torch.float16, True, 128, False),
    ([4], [4], 1, 1, torch.float16, False, 0, True),
])
def test_scored_layers_by_heads(lens, news, hq, hkv, dt, norm, rot, inter):
    """A scored layer's key heads spread over several CTAs, by four and by eight, the last ones fewer."""
    test_rope_append(lens, news, hq, hkv, dt, "scored", norm, rot, inter)


def test_append_agrees_with_the_calls_it_replaces():
    """The same bits as kv_qk_norm_rope followed by kv_quant_pack (fp16), one token at a time included."""
    require_gpu()
    hq, hkv, T = 8, 2, 150
    batch, _ = paged_batch([T], kvq.Allocator(16, seed=3))
    one, two, three = (kvq.LayerCache(hq, hkv, 16, 16, 1, t_cap=152) for _ in range(3))
    q, k, v = rnd((T, hq, D), 1).cuda(), rnd((T, hkv, D), 2).cuda(), rnd((T, hkv, D), 3).cuda()
    tab, w = kvq.RopeTable(128, 10000.0), ws(256)
    qa, ka, qb = torch.empty_like(q), torch.empty_like(k), torch.empty_like(q)
    kvq.kv_qk_norm_rope(one, tab, torch.arange(T, dtype=torch.int32, device="cuda"), q, k, qa, ka)
    kvq.kv_quant_pack(one, batch, 0, 0, T, ka, v)
    kvq.kv_rope_append(two, batch, tab, starts_of([T]), q, k, v, qb, w)
    assert torch.equal(qa, qb)
    lens = torch.zeros(1, dtype=torch.int32, device="cuda")
    step = kvq.Batch(batch.block_table, lens, T)
    for t in range(T):   # q in place
        lens.fill_(t + 1)
        kvq.kv_rope_append(three, step, tab, starts_of([1]), q[t:t + 1], k[t:t + 1], v[t:t + 1], q[t:t + 1], w)
    kvq.kvq_check(w)
    assert torch.equal(q, qb)
    for other in (two, three):
        for a in ("k16", "v16", "kT", "k_absmax"):
            assert torch.equal(getattr(one, a), getattr(other, a)), a


@pytest.mark.parametrize("lens,news,heads,dt,norm,inter,base", [
    ([1], [1], 1, torch.float16, True, True, 10000.0),
    ([40, 17, 5, 100], [1, 1, 1, 1], 128, torch.bfloat16, True, False, 500000.0),
    ([33, 0, 64, 200, 16], [33, 0, 3, 129, 0], 16, torch.float16, False, True, 10000.0),
    ([2000, 77], [1990, 77], 7, torch.bfloat16, True, True, 10000.0),
    ([5001], [5001], 2, torch.float16, True, False, 10000.0),
    ([300], [300], 0, torch.float16, True, False, 10000.0),
])
def test_latent_append(lens, news, heads, dt, norm, inter, base):
    require_gpu()
    rows, extra = sum(news), 2
    pool = sum(-(-max(t, 1) // 16) for t in lens) + 2
    batch, bt = paged_batch([max(t, 1) for t in lens], kvq.Allocator(pool, seed=5), lengths=lens)
    cache = kvq.LatentCache(pool)
    cache.rows.fill_(7)
    x = rnd((rows + extra, ROW + 8), rows, heads, dtype=dt).cuda()
    c, k = x[:, :LAT], x[:, LAT:ROW]
    q = rnd((rows + extra, max(heads, 1), 192), rows, 5, dtype=dt).cuda()[:, :, D:]
    out = torch.full((rows + extra, max(heads, 1), ROW), -7.0, dtype=torch.float16, device="cuda")
    cw = (rnd((LAT,), 4, dtype=torch.float32) + 2).cuda() if norm else None
    tab, w = kvq.RopeTable(ROT, base, interleaved=inter), ws(kvq.kv_rope_append_ws())
    where = places(lens, news)
    at = np.array([p for _, p in where])
    pos = None
    if len(lens) % 2:
        at = 65536 - 2 * at
        pos = torch.tensor(np.concatenate([at, [0] * extra]), dtype=torch.int32, device="cuda")
    kvq.kv_latent_append(cache, batch, tab, starts_of(news), c, k, w, c_weight=cw, eps=1e-5, positions=pos,
                         q=q if heads else None, q_out=out[..., LAT:] if heads else None)
    kvq.kvq_check(w)
    f = R.frequencies(ROT, base)[0]
    zk, bk = R.norm_rope(R.as64(k[:rows, None]), at, f, 1.0, ROT, inter)
    zc = R.as64(c[:rows])
    if norm:
        zc = zc * R.as64(cw) / np.sqrt((zc * zc).mean(-1, keepdims=True) + 1e-5)
    # a sum of 512 squares, a root and two products: under 600 roundings of the value
    bc = 600 * R.U * np.abs(zc) + 2.0 ** -11 * np.abs(zc) + 2.0 ** -25
    got = cache.rows.cpu().numpy()
    written = np.zeros((pool, 16), bool)
    for r, (b, p) in enumerate(where):
        page, slot = bt[b, p // 16], p % 16
        written[page, slot] = True
        assert np.all(np.abs(got[page, slot, :LAT].astype(np.float64) - zc[r]) <= bc[r])
        assert np.all(np.abs(got[page, slot, LAT:].astype(np.float64) - zk[r, 0]) <= bk[r, 0])
    assert np.all(got[~written] == 7)
    if heads:
        zq, bq = R.norm_rope(R.as64(q[:rows]), at, f, 1.0, ROT, inter)
        assert np.all(np.abs(R.as64(out[:rows, :, LAT:]) - zq) <= bq)
        assert bool((out[rows:] == -7).all())
    assert bool((out[..., :LAT] == -7).all())


def test_device_checks():
    """Lengths that do not fit leave a sequence untouched, a table entry that is no page skips the row: flagged both."""
    require_gpu()
    hq, hkv = 4, 2
    tab, w = kvq.RopeTable(128), ws(256)
    q, k, v = rnd((6, hq, D), 1).cuda(), rnd((6, hkv, D), 2).cuda(), rnd((6, hkv, D), 3).cuda()
    bt = torch.tensor([[0, 1], [2, 99], [3, -1]], dtype=torch.int32, device="cuda")
    layer = kvq.LayerCache(hq, hkv, 16, 4, 3)
    lat, ltab = kvq.LatentCache(4), kvq.RopeTable(ROT)

    def calls(lens, starts):
        layer.k16.zero_(), lat.rows.zero_()
        batch = kvq.Batch(bt, torch.tensor(lens, dtype=torch.int32, device="cuda"), 32)
        st = torch.tensor(starts, dtype=torch.int32, device="cuda")
        bad = []
        for latent in (False, True):
            out = torch.zeros_like(q)
            if latent:
                kvq.kv_latent_append(lat, batch, ltab, st, rnd((6, LAT), 4).cuda(), rnd((6, ROT), 5).cuda(), w,
                                     q=q[..., :ROT], q_out=out[..., :ROT])
            else:
                kvq.kv_rope_append(layer, batch, tab, st, q, k, v, out, w)
            try:
                kvq.kvq_check(w)
                bad.append(False)
            except kvq.KvqError as e:
                assert e.code == _abi.KVQ_ERR_DEVICE_CHECK
                bad.append(True)
            assert not bool(out[5].any())
            if latent:
                assert [bool(r.any()) for r in out] == wrote
        return bad, [int((layer.k16[p].abs().sum((0, 2)) > 0).sum()) for p in range(4)], \
            [int((lat.rows[p].abs().sum(1) > 0).sum()) for p in range(4)]

    wrote = [True, True, True, True, True, False]
    assert calls([16, 17, 16], [0, 2, 4, 5]) == ([True] * 2, [2, 0, 1, 1], [2, 0, 1, 1])   # row 3 is on page 99
    wrote = [True, True, False, False, True, False]
    assert calls([16, 1, 16], [0, 2, 4, 5]) == ([True] * 2, [2, 0, 0, 1], [2, 0, 0, 1])    # more new rows than tokens
    assert calls([16, 33, 16], [0, 2, 4, 5]) == ([True] * 2, [2, 0, 0, 1], [2, 0, 0, 1])   # above max_len
    wrote = [False, False, True, True, True, False]
    assert calls([-3, 16, 16], [0, 2, 4, 5]) == ([True] * 2, [0, 0, 2, 1], [0, 0, 2, 1])
    wrote = [True, True, True, True, True, False]
    assert calls([16, 16, 16], [0, 2, 4, 5]) == ([False] * 2, [2, 0, 2, 1], [2, 0, 2, 1])
