"""The appends, tree attention and latent layers as a serving program has them: on streams of its own, captured and
replayed, with nothing to do, with lengths and pages that do not fit, with every way to cut and join the work, and a run
of them together."""
import math

import numpy as np
import pytest
import torch

import latent_ref as LR
import new_token_ref as R
import test_gpu_latent as TL
from compressed_kv_cache_quant_gb300 import _abi, kvq, synth
from gpu_helpers import paged_batch, require_gpu, ws

pytestmark = pytest.mark.gpu
D, LAT, ROT, ROW = 128, 512, 64, 576
SCALE = 1 / math.sqrt(192)


def rnd(shape, *ids, dtype=torch.float16, scale=1.0):
    return synth.normal(shape, synth.mix(synth.BASE_SEED, 9400, *ids), scale=scale, dtype=dtype)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def starts_of(news):
    return i32(np.concatenate([[0], np.cumsum(news)]))


class LatentLayer:
    """A latent layer with the given sequences in it."""

    def __init__(self, lens, seed=0, spare=4):
        pool = sum(-(-max(t, 1) // 16) for t in lens) + spare
        self.alloc = kvq.Allocator(pool, seed=7)
        self.batch, self.bt = paged_batch([max(t, 1) for t in lens], self.alloc, lengths=lens)
        self.cache = kvq.LatentCache(pool)
        self.cache.rows.fill_(float("nan"))
        self.rows = [rnd((t, ROW), seed, b) for b, t in enumerate(lens)]
        for b, t in enumerate(lens):
            for p in range(-(-t // 16)):
                part = self.rows[b][16 * p:16 * p + 16].cuda()
                self.cache.rows[self.bt[b, p], :len(part)] = part


def expect(q, K, lens, news, trees=None, rows=None):
    """{(row, head): (out, lse, bounds)} of absorbed attention."""
    row = 0
    for b, (t, n) in enumerate(zip(lens, news)):
        k = R.as64(K[b])
        for i in range(n):
            if rows is None or row in rows:
                seen = LR.tree_seen(t, trees[b] if trees else list(range(-1, n - 1)), i)
                for h in range(q.shape[1]):
                    yield (row, h), LR.attend(R.as64(q[row, h]), k, k[:, :LAT], seen, SCALE)
            row += 1


def agrees(out, lse, want):
    for (row, h), (o, z, bo, bz) in want:
        assert np.all(np.abs(R.as64(out[row, h]) - o) <= bo), (row, h)
        assert lse is None or abs(float(lse[row, h]) - z) <= bz, (row, h)


@pytest.mark.parametrize("heads,lens,news,rows", [
    (16, [20001], [1], {0}),                     # one row group in very many parts
    (8, [6000] * 12, [1] * 12, {0, 5, 11}),      # few parts each
    (128, [9000], [1], {0}),                     # pairs, very many parts
    (40, [3000, 50, 700], [3, 1, 2], {0, 2, 3, 5}),
    (96, [400] * 20, [1] * 20, {0, 9, 19}),
    (33, [100], [1], {0}),                       # the fewest rows of a pair, and the most without one
    (32, [100], [1], {0}),
    (1, [700] * 45, [1] * 45, {0, 31, 32, 44}),  # more than 32 sequences
    (64, [257] * 70, [2] * 70, {0, 64, 139}),
    (3, [500], [200], {0, 63, 64, 199}),         # a run as long as a prompt
])
def test_every_cut_and_join(heads, lens, news, rows):
    require_gpu()
    L = LatentLayer(lens, seed=heads)
    n = sum(news)
    q, out, lse = rnd((n, heads, ROW), heads, n).cuda(), torch.empty((n, heads, LAT), dtype=torch.float16, device="cuda"), torch.empty((n, heads), device="cuda")
    w = ws(kvq.kv_latent_attn_ws(L.batch, heads, n, max(news)))
    kvq.kv_latent_attn(L.cache, L.batch, q, starts_of(news), max(news), out, w, lse=lse)
    kvq.kvq_check(w)
    assert not bool(w.t.any())
    sample = torch.arange(0, heads, max(1, heads // 3)).tolist()
    agrees(out[:, sample], lse[:, sample], expect(q[:, sample], L.rows, lens, news, rows=rows))
    without = torch.empty_like(out)   # without lse: the same bits
    kvq.kv_latent_attn(L.cache, L.batch, q, starts_of(news), max(news), without, w)
    assert torch.equal(out, without)


def test_weights_that_grow_along_the_cache():
    """Scores that rise by thousands of log2 units over a part: anchors are set anew, many times."""
    require_gpu()
    for heads in (4, 64):
        T = 700
        L = LatentLayer([T], seed=5)
        up = torch.linspace(0, 24, T).half()[:, None]
        rows = L.rows[0].clone()
        rows[:, :4] = up
        L.rows[0] = rows
        for p in range(-(-T // 16)):
            part = rows[16 * p:16 * p + 16].cuda()
            L.cache.rows[L.bt[0, p], :len(part)] = part
        q = rnd((1, heads, ROW), 3, heads).cuda()
        q[..., :4] = torch.linspace(0, 30, heads, dtype=torch.float16, device="cuda")[None, :, None]
        out, lse = torch.empty((1, heads, LAT), dtype=torch.float16, device="cuda"), torch.empty((1, heads), device="cuda")
        w = ws(kvq.kv_latent_attn_ws(L.batch, heads, 1, 1))
        kvq.kv_latent_attn(L.cache, L.batch, q, i32([0, 1]), 1, out, w, lse=lse)
        agrees(out, lse, expect(q, L.rows, [T], [1]))


def test_nothing_to_do():
    """No rows, no sequences, sequences without new tokens: nothing is written, nothing is flagged."""
    require_gpu()
    L = LatentLayer([0, 40], seed=1)
    w = ws(1 << 20)
    q, out = rnd((3, 4, ROW), 1).cuda(), torch.full((3, 4, LAT), -7.0, dtype=torch.float16, device="cuda")
    kvq.kv_latent_attn(L.cache, L.batch, q, i32([0, 0, 0]), 1, out, w)
    kvq.kv_latent_attn(L.cache, L.batch, q[:0], i32([0, 0, 0]), 0, out[:0], w)
    none = kvq.Batch(torch.zeros((0, 1), dtype=torch.int32, device="cuda"), i32([]), 16)
    kvq.kv_latent_attn(L.cache, none, q, i32([0]), 1, out, w)
    o = torch.full((3, 4, D), -7.0, dtype=torch.float16, device="cuda")
    x = rnd((5, 4, 2 * D), 2).cuda()
    kvq.kv_latent_expanded_attn(rnd((3, 4, 192), 3).cuda(), x[..., :D], x[:, 0, :ROT], x[..., D:], i32([0, 0]), i32([0, 5]), 1, 5, o, w)
    assert bool((out == -7).all()) and bool((o == -7).all())
    kept = L.cache.rows.clone()
    tab = kvq.RopeTable(ROT)
    kvq.kv_latent_append(L.cache, L.batch, tab, i32([0, 0, 0]), q[:, 0, :LAT], q[:, 0, LAT:], w)
    kvq.kv_latent_append(L.cache, L.batch, tab, i32([0, 0, 0]), q[:0, 0, :LAT], q[:0, 0, LAT:], w)
    assert torch.equal(kept.view(torch.int16), L.cache.rows.view(torch.int16))
    layer = kvq.LayerCache(4, 2, 16, 6, 2, t_cap=48)
    k = rnd((3, 2, D), 4).cuda()
    kvq.kv_rope_append(layer, L.batch, kvq.RopeTable(D), i32([0, 0, 0]), None, k, k, None, w)
    t = torch.full((3, 4, D), -7.0, dtype=torch.float16, device="cuda")
    kvq.kv_tree_attn(layer, L.batch, rnd((3, 4, D), 5).cuda(), i32([-1, -1, -1]), i32([0, 0, 0]), 1, t, w)
    assert not bool(layer.k16.any()) and not bool(layer.kT.any()) and bool((t == -7).all())
    kvq.kvq_check(w)


@pytest.mark.parametrize("heads", [16, 128])
def test_lengths_and_pages_that_do_not_fit(heads):
    """Flagged; the sequence's rows stay as they were (lengths), or the page's tokens count as zeros."""
    require_gpu()
    L = LatentLayer([40, 100, 33], seed=2)
    q = rnd((6, heads, ROW), 1).cuda()
    w = ws(kvq.kv_latent_attn_ws(L.batch, heads, 6, 2))

    def call(lens, starts, max_new=2, bt=None):
        batch = kvq.Batch(L.batch.block_table if bt is None else bt, i32(lens), 100)
        out = torch.full((6, heads, LAT), -7.0, dtype=torch.float16, device="cuda")
        kvq.kv_latent_attn(L.cache, batch, q, i32(starts), max_new, out, w)
        try:
            kvq.kvq_check(w)
            flagged = False
        except kvq.KvqError as e:
            assert e.code == _abi.KVQ_ERR_DEVICE_CHECK
            flagged = True
        assert not bool(w.t[:256].any())
        w.t.zero_()   # (after a call that failed on the device)
        return flagged, [bool((r != -7).any()) for r in out], out

    good = call([40, 100, 33], [0, 2, 4, 5])
    assert good[:2] == (False, [True] * 5 + [False])
    for lens, starts, rows in (([40, 1, 33], [0, 2, 4, 5], [True, True, False, False, True, False]),
                               ([40, 101, 33], [0, 2, 4, 5], [True, True, False, False, True, False]),
                               ([40, -5, 33], [0, 2, 4, 5], [True, True, False, False, True, False]),
                               ([40, 100, 33], [0, 2, 5, 6], [True, True, False, False, False, True]),     # three rows, max_new 2
                               ([40, 100, 33], [0, 2, 4, 9], [True, True, True, True, False, False]),      # behind n_rows
                               ([40, 100, 33], [0, 2, 1, 3], [True, True, True, False, False, False]),     # not ascending
                               ([40, 100, 33], [-2, 0, 2, 4], [True, True, True, True, False, False])):
        got = call(lens, starts)
        assert got[:2] == (True, rows), (lens, starts, got[:2])
    bad = L.batch.block_table.clone()
    bad[1, 1] = 10 ** 6
    got = call([40, 100, 33], [0, 2, 4, 5], bt=bad)
    assert got[0] and torch.equal(got[2][:2], good[2][:2]) and torch.equal(got[2][4], good[2][4])
    assert bool(torch.isfinite(got[2].float()).all())


def test_expanded_lengths_that_do_not_fit():
    require_gpu()
    H = 2
    x = rnd((60, H, 2 * D), 1).cuda()
    kr = rnd((60, ROT), 2).cuda()
    q = rnd((6, H, 192), 3).cuda()
    w = ws(kvq.kv_latent_expanded_attn_ws(2, H, 6, 3, 40))
    for qs, ks, max_len, rows in (([0, 3, 5], [0, 40, 60], 40, [1, 1, 1, 1, 1, 0]), ([0, 3, 5], [0, 41, 60], 40, [0, 0, 0, 1, 1, 0]),
                                  ([0, 3, 5], [0, 2, 20], 40, [0, 0, 0, 1, 1, 0]), ([0, 3, 5], [0, 40, 61], 40, [1, 1, 1, 0, 0, 0]),
                                  ([0, 3, 5], [-1, 30, 50], 40, [0, 0, 0, 1, 1, 0]), ([0, 3, 5], [30, 20, 50], 40, [0, 0, 0, 1, 1, 0]),
                                  ([0, 4, 6], [0, 30, 50], 40, [0, 0, 0, 0, 1, 1])):
        out = torch.full((6, H, D), -7.0, dtype=torch.float16, device="cuda")
        kvq.kv_latent_expanded_attn(q, x[..., :D], kr, x[..., D:], i32(qs), i32(ks), 3, max_len, out, w)
        got = [int(bool((r != -7).any())) for r in out]
        assert got == rows, (qs, ks, got)
        if all(rows[:5]):
            kvq.kvq_check(w)
        else:
            with pytest.raises(kvq.KvqError):
                kvq.kvq_check(w)


def test_expanded_head_major_and_single():
    """Keys and values whose heads lie apart, one head, one key."""
    require_gpu()
    T, H, n = 150, 3, 40
    kn, v, kr = rnd((H, T, D), 1).cuda(), rnd((H, T, D), 2).cuda(), rnd((T, ROT), 3).cuda()
    q = rnd((n, H, 192), 4).cuda()
    w = ws(kvq.kv_latent_expanded_attn_ws(1, H, n, n, T))
    outs = []
    for a, b in ((kn.transpose(0, 1), v.transpose(0, 1)), (kn.transpose(0, 1).contiguous(), v.transpose(0, 1).contiguous())):
        out = torch.empty((n, H, D), dtype=torch.float16, device="cuda")
        kvq.kv_latent_expanded_attn(q, a, kr, b, i32([0, n]), i32([0, T]), n, T, out, w)
        outs.append(out)
    assert torch.equal(*outs)
    one = torch.empty((1, 1, D), dtype=torch.float16, device="cuda")
    kvq.kv_latent_expanded_attn(q[:1, :1].contiguous(), kn.transpose(0, 1)[:1, :1], kr[:1], v.transpose(0, 1)[:1, :1], i32([0, 1]), i32([0, 1]), 1, 1,
                                one, w)
    assert torch.equal(one[0, 0], v[0, 0])   # a softmax over one token


def test_binding_refuses_what_it_cannot_pass_on():
    require_gpu()
    L = LatentLayer([40], seed=3)
    w, tab = ws(1 << 20), kvq.RopeTable(ROT)
    q, out = rnd((1, 4, ROW), 1).cuda(), torch.empty((1, 4, LAT), dtype=torch.float16, device="cuda")
    s = i32([0, 1])
    go = lambda **k: kvq.kv_latent_attn(**{**dict(cache=L.cache, seqs=L.batch, q=q, q_starts=s, max_new=1, out=out, ws=w), **k})  # noqa: E731
    go()
    for bad in (dict(q=q.float()), dict(q=q.cpu()), dict(q=q[..., :LAT]), dict(q=torch.cat([q, q], -1)[..., :ROW]), dict(q=None), dict(out=out.float()),
                dict(out=out[:, :2]), dict(out=None), dict(q_starts=s.long()), dict(q_starts=i32([0, 1, 1])), dict(q_starts=None), dict(parents=i32([-1, 0])),
                dict(lse=torch.empty((1, 3), device="cuda")), dict(scale=-1.0)):
        with pytest.raises(kvq.KvqError):
            go(**bad)
    c, k = rnd((1, LAT), 2).cuda(), rnd((1, ROT), 3).cuda()
    qr = torch.empty((1, 4, ROT), dtype=torch.float16, device="cuda")
    ap = lambda **x: kvq.kv_latent_append(**{**dict(cache=L.cache, seqs=L.batch, rope=tab, row_starts=s, c=c, k_rope=k, ws=w), **x})  # noqa: E731
    ap()
    for bad in (dict(c=c.float()), dict(c=c.bfloat16()), dict(k_rope=k[:, :32]), dict(k_rope=None), dict(q=qr), dict(q_out=qr), dict(q=qr, q_out=qr.float()),
                dict(q=qr, q_out=qr[:, :2]), dict(c_weight=torch.ones(LAT, device="cuda").half()), dict(c_weight=torch.ones(ROT, device="cuda")),
                dict(rope=kvq.RopeTable(128)), dict(positions=i32([0, 1])), dict(c=rnd((1, 2 * LAT), 4).cuda()[:, ::2]), dict(row_starts=i32([0]))):
        with pytest.raises(kvq.KvqError):
            ap(**bad)
    layer = kvq.LayerCache(4, 2, 16, 8, 1)
    kv = rnd((1, 2, D), 5).cuda()
    ra = lambda **x: kvq.kv_rope_append(**{**dict(cache=layer, seqs=L.batch, rope=kvq.RopeTable(D), row_starts=s, q=None, k=kv, v=kv, q_out=None, ws=w), **x})  # noqa: E731
    ra()
    for bad in (dict(k=kv.float(), v=kv.float()), dict(v=kv.bfloat16()), dict(v=None), dict(k=rnd((1, 2, 2 * D), 6).cuda()[..., ::2]),
                dict(q=kv), dict(k_weight=torch.ones(64, device="cuda")), dict(cache=kvq.LayerCache(4, 2, 4, 8, 1))):
        with pytest.raises(kvq.KvqError):
            ra(**bad)
    x = rnd((5, 4, 2 * D), 2).cuda()
    ex = lambda **k: kvq.kv_latent_expanded_attn(**{**dict(q=rnd((1, 4, 192), 3).cuda(), k_nope=x[..., :D], k_rope=x[:, 0, :ROT], v=x[..., D:], q_starts=s,  # noqa: E731
                                                           k_starts=i32([0, 5]), max_new=1, max_len=5, out=torch.empty((1, 4, D), dtype=torch.float16, device="cuda"),
                                                           ws=w), **k})
    ex()
    for bad in (dict(k_nope=x[:4, :, :D]), dict(v=x[..., D:].float()), dict(k_rope=x[:, 0, :32]), dict(k_starts=i32([0])), dict(k_starts=None),
                dict(k_nope=rnd((5, 4, D + 4), 9).cuda()[..., 4:])):   # (8 bytes off)
        with pytest.raises(kvq.KvqError):
            ex(**bad)
    kvq.kvq_check(w)


def test_streams_and_graphs():
    """Calls on two streams with workspaces of their own at once, and all five captured into one graph and replayed."""
    require_gpu()
    lens, news, H = [900, 77], [5, 3], 64
    L = LatentLayer(lens, seed=4)
    n = sum(news)
    s = starts_of(news)
    q = rnd((n, H, ROW), 1).cuda()
    c, k = rnd((n, LAT), 2).cuda(), rnd((n, ROT), 3).cuda()
    tab, tab_d = kvq.RopeTable(ROT), kvq.RopeTable(D)
    layer = kvq.LayerCache(8, 2, 16, 80, 2, t_cap=904)
    kvq_rows = rnd((n, 2, D), 4).cuda()
    parents = i32([-1, 0, 0, 1, -1, -1, 0, 0])
    x = rnd((sum(lens), H, 2 * D), 5).cuda()
    kr = rnd((sum(lens), ROT), 6).cuda()

    class Turn:
        def __init__(self):
            f = lambda *shape: torch.empty(shape, dtype=torch.float16, device="cuda")  # noqa: E731
            self.qa, self.o, self.t, self.e, self.qd = f(n, H, ROW), f(n, H, LAT), f(n, 8, D), f(n, H, D), f(n, 8, D)
            self.w = [ws(kvq.kv_latent_attn_ws(L.batch, H, n, 5)), ws(kvq.kv_tree_attn_ws(layer, L.batch, n, 5)),
                      ws(kvq.kv_latent_expanded_attn_ws(2, H, n, 5, 900))]

        def go(self, stream=None):
            self.qa.copy_(q)
            kvq.kv_latent_append(L.cache, L.batch, tab, s, c, k, self.w[0], q=q[..., LAT:], q_out=self.qa[..., LAT:], stream=stream)
            kvq.kv_latent_attn(L.cache, L.batch, self.qa, s, 5, self.o, self.w[0], parents=parents, stream=stream)
            kvq.kv_rope_append(layer, L.batch, tab_d, s, q[:, :8, :D].contiguous(), kvq_rows, kvq_rows, self.qd, self.w[1], stream=stream)
            kvq.kv_tree_attn(layer, L.batch, self.qd, parents, s, 5, self.t, self.w[1], stream=stream)
            kvq.kv_latent_expanded_attn(q[..., :192].contiguous(), x[..., :D], kr, x[..., D:], s, i32(np.concatenate([[0], np.cumsum(lens)])) if stream is None else ks,
                                        5, 900, self.e, self.w[2], stream=stream)

        def outputs(self):
            return [t.clone() for t in (self.qa, self.o, self.t, self.e, self.qd)]

    ks = i32(np.concatenate([[0], np.cumsum(lens)]))
    first = Turn()
    first.go()
    torch.cuda.synchronize()
    want = first.outputs()
    assert not any(bool(torch.isnan(t.float()).any()) for t in want)
    turns, streams = [Turn(), Turn()], [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for t, st in zip(turns, streams):
            with torch.cuda.stream(st):
                t.go(st)
    torch.cuda.synchronize()
    for t in turns:
        assert all(torch.equal(a, b) for a, b in zip(t.outputs(), want))
    t, st, g = Turn(), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(st):
        t.go(st)
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=st):
            t.go(st)
    for o in (t.qa, t.o, t.t, t.e, t.qd):
        o.zero_()
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(t.outputs(), want))
    q.mul_(0.5)   # new inputs at the same addresses
    first.go()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(t.outputs(), first.outputs()))
    assert not torch.equal(first.o, want[1])


def test_drafts_are_checked_and_accepted():
    """A speculative step on an fp16 layer: a prompt goes in, a tree of drafts is appended and attended, the accepted path is
    appended again in its order, and the next token attends a cache that equals one written without drafts."""
    require_gpu()
    hq, hkv, T, n = 8, 2, 77, 9
    parents = [-1, 0, 0, 1, 1, 2, 3, -1, 7]
    path = [0, 1, 4]      # accepted
    depth = [len(p) - 1 for p in LR.paths(parents)]
    batch, _ = paged_batch([128], kvq.Allocator(12, seed=3), lengths=[T])
    lens = batch.seq_lens
    tab = kvq.RopeTable(D, 10000.0)
    w = ws(kvq.kv_tree_attn_ws(kvq.LayerCache(hq, hkv, 16, 12, 1), batch, n, n))
    proj = lambda m, i: (rnd((m, hq, D), i, 1).cuda(), rnd((m, hkv, D), i, 2).cuda(), rnd((m, hkv, D), i, 3).cuda())  # noqa: E731
    q0, k0, v0 = proj(T, 1)
    q1, k1, v1 = proj(n, 2)
    q2, k2, v2 = proj(1, 3)

    def prompt(layer):
        out = torch.empty_like(q0)
        kvq.kv_rope_append(layer, batch, tab, i32([0, T]), q0, k0, v0, out, w)

    layer, plain = (kvq.LayerCache(hq, hkv, 16, 12, 1, t_cap=128) for _ in range(2))
    prompt(layer)
    lens.fill_(T + n)
    qr = torch.empty_like(q1)
    pos = i32([T + d for d in depth])
    kvq.kv_rope_append(layer, batch, tab, i32([0, n]), q1, k1, v1, qr, w, positions=pos)
    out = torch.empty_like(q1)
    kvq.kv_tree_attn(layer, batch, qr, i32(parents), i32([0, n]), n, out, w)
    # every node attends as the last token of its own path would
    for i, p in enumerate(LR.paths(parents)):
        lens.fill_(T)
        prompt(plain)
        lens.fill_(T + len(p))
        rotated = torch.empty((len(p), hq, D), dtype=torch.float16, device="cuda")
        kvq.kv_rope_append(plain, batch, tab, i32([0, len(p)]), q1[p].contiguous(), k1[p].contiguous(), v1[p].contiguous(), rotated, w)
        alone = torch.empty((1, hq, D), device="cuda")
        kvq.kv_decode_attn(plain, batch, rotated[-1:].contiguous(), alone, ws(kvq.kv_decode_attn_ws(plain, batch)))
        # two weights' roundings and the outputs': 2^-11 each of a value of size under 4
        assert float((out[i].float() - alone[0]).abs().max()) <= 4 * 2 * 2.0 ** -10
        assert torch.equal(rotated[-1], qr[i])
    # the accepted path, in its order
    m = len(path)
    lens.fill_(T + m)
    kvq.kv_rope_append(layer, batch, tab, i32([0, m]), None, k1[path].contiguous(), v1[path].contiguous(), None, w)
    lens.fill_(T)
    prompt(plain)
    lens.fill_(T + m)
    kvq.kv_rope_append(plain, batch, tab, i32([0, m]), None, k1[path].contiguous(), v1[path].contiguous(), None, w)
    lens.fill_(T + m + 1)
    outs = []
    for c in (layer, plain):
        qn, o = torch.empty_like(q2), torch.empty((1, hq, D), device="cuda")
        kvq.kv_rope_append(c, batch, tab, i32([0, 1]), q2, k2, v2, qn, w)
        kvq.kv_decode_attn(c, batch, qn, o, ws(kvq.kv_decode_attn_ws(c, batch)))
        outs.append(o)
    assert torch.equal(*outs)
    kvq.kvq_check(w)


def test_latent_layer_from_prompt_to_decode():
    """A prompt attends in the expanded form over the rows it has just appended, decode steps in the absorbed form: both
    as the plain form has it."""
    require_gpu()
    H, T, steps = 4, 90, 3
    up_k = rnd((H, D, LAT), 2, dtype=torch.float32, scale=LAT ** -0.5).cuda()
    up_v = rnd((H, D, LAT), 3, dtype=torch.float32, scale=LAT ** -0.5).cuda()
    w_norm = (rnd((LAT,), 4, dtype=torch.float32) / 8 + 1).cuda()
    batch, bt = paged_batch([T + steps], kvq.Allocator(9, seed=5), lengths=[T])
    cache, tab, w = kvq.LatentCache(9), kvq.RopeTable(ROT, 10000.0, interleaved=True), ws(1 << 22)
    x = rnd((T + steps, ROW), 6).cuda()
    q = rnd((T + steps, H, 192), 7).cuda()

    def append(at, n):
        qr = torch.empty((n, H, 192), dtype=torch.float16, device="cuda")
        qr[..., :D] = q[at:at + n, :, :D]
        kvq.kv_latent_append(cache, batch, tab, i32([0, n]), x[at:at + n, :LAT], x[at:at + n, LAT:], w, c_weight=w_norm, q=q[at:at + n, :, D:],
                             q_out=qr[..., D:])
        return qr

    qr = append(0, T)
    rows = cache.rows[torch.tensor(bt[0, :-(-T // 16)], device="cuda").long()].view(-1, ROW)[:T]
    kn = torch.einsum("tc,hdc->thd", rows[:, :LAT].float(), up_k).half()
    v = torch.einsum("tc,hdc->thd", rows[:, :LAT].float(), up_v).half()
    out = torch.empty((T, H, D), dtype=torch.float16, device="cuda")
    kvq.kv_latent_expanded_attn(qr, kn, rows[:, LAT:], v, i32([0, T]), i32([0, T]), T, T, out, w)
    got = [out]
    for t in range(steps):
        batch.seq_lens.fill_(T + t + 1)
        one = append(T + t, 1)
        qa = torch.cat([torch.einsum("nhd,hdc->nhc", one[..., :D].float(), up_k), one[..., D:].float()], -1).half()
        o = torch.empty((1, H, LAT), dtype=torch.float16, device="cuda")
        kvq.kv_latent_attn(cache, batch, qa, i32([0, 1]), 1, o, w)
        got.append(torch.einsum("nhc,hdc->nhd", o.float(), up_v))
    kvq.kvq_check(w)
    # the plain form in 64 bits, from the inputs
    c = x[:, :LAT].double()
    c = c * w_norm.double() / (c.square().mean(-1, keepdim=True) + 1e-6).sqrt()
    f = torch.tensor(R.frequencies(ROT, 10000.0)[0], device="cuda")
    turn = torch.polar(torch.ones((T + steps, ROT // 2), dtype=torch.float64, device="cuda"), torch.arange(T + steps, device="cuda").double()[:, None] * f)
    rot = lambda y, a: torch.view_as_real(torch.view_as_complex(y.double().unflatten(-1, (-1, 2)).contiguous()) * a).flatten(-2)  # noqa: E731
    k = torch.cat([torch.einsum("tc,hdc->thd", c, up_k.double()), rot(x[:, LAT:], turn)[:, None].expand(-1, H, -1)], -1)
    qd = torch.cat([q[..., :D].double(), rot(q[..., D:], turn[:, None])], -1)
    s = torch.einsum("nhd,thd->hnt", qd, k) * SCALE
    s = s.masked_fill(torch.ones((T + steps, T + steps), device="cuda").triu(1).bool(), -math.inf)
    want = torch.einsum("hnt,thd->nhd", s.softmax(-1), torch.einsum("tc,hdc->thd", c, up_v.double()))
    have = torch.cat([g.double() for g in got])
    # rows, keys, values, queries and outputs rounded to fp16 on the way: scores of size 3 off by under 2^-8
    assert float((have - want).norm() / want.norm()) <= 2.0 ** -7
