"""GPU parity of the new-token operators against plain 64-bit forms: head norms with rotary positions,
attention of one token and of runs of tokens over fp16 pages, page and slot copies; their device checks;
and a run of them together, as a serving program would call them."""
import math

import numpy as np
import pytest
import torch

import new_token_ref as R
from compressed_kv_cache_quant_gb300 import _abi, kvq, synth
from gpu_helpers import ATTN_TOL, attn_err, paged_batch, require_gpu, ws

pytestmark = pytest.mark.gpu
D = 128


def rnd(shape, *ids, dtype=torch.float16, scale=1.0):
    return synth.normal(shape, synth.mix(synth.BASE_SEED, 7000, *ids), scale=scale, dtype=dtype)


# ------------------------------------------------------------------ norms and rotary positions

@pytest.mark.parametrize("n,hq,hkv,dt,norm,rot,inter,scaling,first", [
    (1, 8, 2, torch.float16, False, 128, False, "plain", 0),
    (7, 32, 8, torch.bfloat16, True, 128, False, "yarn", 131000),
    (33, 5, 3, torch.float16, True, 64, True, "ntk", 1000003),
    (130, 40, 40, torch.bfloat16, False, 96, False, "linear", 77),
    (5, 8, 1, torch.float16, True, 32, True, "knees", 2 ** 30),
    (9, 2, 1, torch.float16, False, 16, False, "knees", 5),
    (3, 4, 4, torch.bfloat16, True, 0, False, "plain", 0),
    (1300, 4, 2, torch.float16, True, 128, True, "plain", -600),
])
def test_norm_rope(n, hq, hkv, dt, norm, rot, inter, scaling, first):
    require_gpu()
    spec = dict(scaling=scaling, factor=1.0 if scaling == "plain" else 8.0, original_len=8192)
    tab = kvq.RopeTable(rot, 500000.0, interleaved=inter, **spec)
    f, m = R.frequencies(rot, 500000.0, scaling, spec["factor"], 8192,
                         *((32.0, 1.0) if scaling == "yarn" else (1.0, 4.0))) if rot else (np.zeros(0), 1.0)
    rows = rnd((n, (hq + 2 * hkv) * D + 8), n, hq, dtype=dt).cuda()   # a projection's rows, 8 values of something else behind
    q = rows[:, :hq * D].view(n, hq, D)
    k = rows[:, hq * D:(hq + hkv) * D].view(n, hkv, D)
    v = rows[:, (hq + hkv) * D:(hq + 2 * hkv) * D].view(n, hkv, D)
    step = 1 if n < 1000 else 3
    pos = first + step * np.arange(n)
    pos[::2] = pos[::2][::-1]   # any order
    p = torch.tensor(pos, dtype=torch.int32, device="cuda")
    wq, wk = ((rnd((D,), 1, dtype=torch.float32) + 2).cuda(), (rnd((D,), 2, dtype=torch.float32) + 2).cuda()) if norm else (None, None)
    out = [torch.full((n + 1, h, D), -7.0, dtype=torch.float16, device="cuda") for h in (hq, hkv, hkv)]
    kvq.kv_qk_norm_rope(kvq.make_layout(hq, hkv, 16), tab, p if rot else None, q, k, out[0][:n], out[1][:n], wq, wk, 1e-5,
                        v, out[2][:n])
    for x, y, w in ((q, out[0], wq), (k, out[1], wk)):
        z, bound = R.norm_rope(R.as64(x), pos, f, m, rot, inter, None if w is None else R.as64(w), 1e-5)
        assert np.all(np.abs(R.as64(y[:n]) - z) <= bound)
        assert bool((y[n] == -7).all())
    assert torch.equal(out[2][:n], v.half()) and bool((out[2][n] == -7).all())


def test_rope_in_place_inverse_and_parts():
    """In place, only k, only v; the inverse (negated positions) brings rows back to two roundings."""
    require_gpu()
    L, tab = kvq.make_layout(8, 2, 16), kvq.RopeTable(128, 10000.0)
    k = rnd((37, 2, D), 3).cuda()
    kept = k.clone()
    pos = torch.arange(5000, 5037, dtype=torch.int32, device="cuda")
    kvq.kv_qk_norm_rope(L, tab, pos, None, k, None, k)
    other = torch.empty_like(kept)
    kvq.kv_qk_norm_rope(L, tab, pos, None, kept, None, other)
    assert torch.equal(k, other) and not torch.equal(k, kept)
    kvq.kv_qk_norm_rope(L, tab, -pos, None, k, None, k)
    size = float(kept.float().abs().max()) * 2
    assert float((k.float() - kept.float()).abs().max()) <= size * (2 ** -11 * 2 + 400 * R.U)
    v = torch.empty_like(kept)
    kvq.kv_qk_norm_rope(L, tab, pos, None, None, None, None, v=kept, v_out=v)
    assert torch.equal(v, kept)
    kvq.kv_qk_norm_rope(L, tab, pos[:0], None, kept[:0], None, other[:0])   # no tokens: nothing happens


# ------------------------------------------------------------------ attention

MODS = {
    "plain": {},
    "cap": dict(softcap=20.0),
    "bias": dict(bias=True),
    "cap_bias_scale": dict(softcap=5.0, bias=True, scale=0.2),
    "window": dict(window=70),
    "window_sink": dict(window=33, n_sink=5),
    "window_one": dict(window=1),
    "docs": dict(docs=True),
    "docs_window_sink": dict(docs=True, window=40, n_sink=20),
    "prefix": dict(prefix=True),
    "prefix_window_bias": dict(prefix=True, window=50, n_sink=3, bias=True),
}


class Case:
    """Sequences of the given lengths in shuffled pages; the last news[b] tokens of each are the queries."""

    def __init__(self, hq, hkv, lens, news, mod, seed, poison=True):
        B = len(lens)
        self.hq, self.hkv, self.lens, self.news, self.spec = hq, hkv, lens, news, dict(MODS[mod])
        self.KV = [synth.kv_rows(T, hkv, synth.mix(seed, b)) for b, T in enumerate(lens)]
        pages = sum(math.ceil(T / 16) for T in lens) + 2
        self.batch, self.bt = paged_batch([max(T, 1) for T in lens], kvq.Allocator(pages + B, seed=9), lengths=lens)
        self.cache = kvq.LayerCache(hq, hkv, 16, pages + B, B)
        if poison:   # whatever no sequence holds: unused pages and the rows behind a sequence's last token
            self.cache.k16.fill_(float("nan"))
            self.cache.v16.fill_(float("nan"))
        for b, T in enumerate(lens):
            if T:
                kvq.kv_quant_pack(self.cache, self.batch, b, 0, T, self.KV[b][0].cuda(), self.KV[b][1].cuda())
        g = np.random.default_rng(seed)
        rows = sum(news)
        self.q = rnd((rows, hq, D), seed, 1).cuda()
        self.starts = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
        self.slopes = torch.tensor([2.0 ** (-8 * (h + 1) / hq) for h in range(hq)]) if self.spec.pop("bias", False) else None
        self.doc = self.prefix = None
        if self.spec.pop("docs", False):   # some begin behind their query: such a row sees nothing
            d = [g.integers(0, T + 2) if i % 3 else max(0, T - n + i - 20) for T, n in zip(lens, news) for i in range(n)]
            self.doc = np.array(d, dtype=np.int32)
        if self.spec.pop("prefix", False):
            self.prefix = np.array([g.integers(0, T + 3) for T in lens], dtype=np.int32)
        dev = lambda x: None if x is None else torch.as_tensor(x).cuda()  # noqa: E731
        self.mod = kvq.AttnMod(slopes=dev(self.slopes), prefix_len=dev(self.prefix), doc_start=dev(self.doc), **self.spec)

    def check(self, out, lse, fp16, rows=None):
        row = 0
        for b, (T, n) in enumerate(zip(self.lens, self.news)):
            K, V = R.as64(self.KV[b][0]), R.as64(self.KV[b][1])
            for i in range(n):
                if rows is None or row in rows:
                    pos = T - n + i
                    seen = R.visible(T, pos, 0 if self.prefix is None else int(self.prefix[b]),
                                     0 if self.doc is None else int(self.doc[row]), self.spec.get("window", 0),
                                     self.spec.get("n_sink", 0)) if T else np.zeros(0, bool)
                    for h in range(self.hq):
                        o, z, bo, bz = R.attend(R.as64(self.q[row, h]), K[:, h // (self.hq // self.hkv)],
                                                V[:, h // (self.hq // self.hkv)], seen, pos, self.spec.get("scale", 0.0),
                                                self.spec.get("softcap", 0.0),
                                                0.0 if self.slopes is None else float(self.slopes[h]), fp16)
                        assert np.all(np.abs(R.as64(out[row, h]) - o) <= bo), (b, i, h)
                        got = float(lse[row, h])
                        assert got == z if math.isinf(z) else abs(got - z) <= bz, (b, i, h, got, z)
                row += 1

    def decode(self, wk=None):
        out = torch.full((len(self.lens), self.hq, D), float("nan"), device="cuda")
        lse = torch.full((len(self.lens), self.hq), float("nan"), device="cuda")
        wk = wk or ws(kvq.kv_decode_attn_ws(self.cache, self.batch))
        kvq.kv_decode_attn(self.cache, self.batch, self.q, out, wk, mod=self.mod, lse=lse)
        kvq.kvq_check(wk)
        return out, lse, wk

    def chunk(self, wk=None, extra=2):
        """`extra` rows of out and lse lie behind the last sequence."""
        rows = self.q.shape[0] + extra
        q = torch.cat([self.q, torch.full((extra, self.hq, D), float("nan"), dtype=torch.float16, device="cuda")])
        out = torch.full((rows, self.hq, D), -7.0, dtype=torch.float16, device="cuda")
        lse = torch.full((rows, self.hq), -7.0, device="cuda")
        most = max(max(self.news), 1)
        wk = wk or ws(kvq.kv_chunk_attn_ws(self.cache, self.batch, rows, most))
        if self.doc is not None:
            self.mod = kvq.AttnMod(slopes=self.mod.slopes, prefix_len=self.mod.prefix_len,
                                   doc_start=torch.cat([torch.tensor(self.doc), torch.zeros(extra, dtype=torch.int32)]).cuda(),
                                   **self.spec)
        kvq.kv_chunk_attn(self.cache, self.batch, q, torch.tensor(self.starts).cuda(), most, out, wk, mod=self.mod, lse=lse)
        kvq.kvq_check(wk)
        if extra:
            assert bool((out[-extra:] == -7).all()) and bool((lse[-extra:] == -7).all())
        return out, lse, wk


@pytest.mark.parametrize("mod", sorted(MODS))
@pytest.mark.parametrize("hq,hkv", [(8, 2), (3, 3), (4, 2), (8, 1)])
def test_decode_attn(hq, hkv, mod):
    require_gpu()
    lens = [1, 0, 15, 16, 17, 130, 777, 2049]
    c = Case(hq, hkv, lens, [1] * len(lens), mod, 50 + hq)
    out, lse, wk = c.decode()
    c.check(out, lse, False)
    again, lse2, _ = c.decode(wk)      # the workspace was left as it was found; parts join in their order
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    assert not bool(wk.t.any())


@pytest.mark.parametrize("hq,hkv,mod", [(12, 3, "window_sink"), (12, 3, "cap_bias_scale"), (16, 16, "docs"), (20, 5, "plain")])
def test_decode_attn_many_rows(hq, hkv, mod):
    """More (sequence, kv head) rows than the one-launch form takes."""
    require_gpu()
    lens = [3001 - 150 * b for b in range(20)] + [0, 1]
    c = Case(hq, hkv, lens, [1] * len(lens), mod, 88)
    out, lse, wk = c.decode()
    c.check(out, lse, False)
    again, lse2, _ = c.decode(wk)
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    assert not bool(wk.t.any())


@pytest.mark.parametrize("mod", ["plain", "cap_bias_scale", "window_sink"])
def test_decode_attn_one_long_sequence(mod):
    require_gpu()
    c = Case(8, 2, [20011], [1], mod, 91)
    out, lse, wk = c.decode()
    c.check(out, lse, False)
    assert not bool(wk.t.any())


@pytest.mark.parametrize("mod", sorted(MODS))
@pytest.mark.parametrize("hq,hkv,lens,news", [
    (8, 2, [1, 5, 16, 200], [1, 5, 3, 200]),
    (2, 2, [0, 300, 129, 64], [0, 131, 129, 0]),
    (8, 1, [700], [45]),
    (4, 2, [517], [517]),
])
def test_chunk_attn(hq, hkv, lens, news, mod):
    require_gpu()
    c = Case(hq, hkv, lens, news, mod, 60 + hq)
    out, lse, wk = c.chunk()
    c.check(out, lse, True)
    again, lse2, _ = c.chunk(wk)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("mod", sorted(MODS))
@pytest.mark.parametrize("hq,hkv,lens,news", [
    (8, 2, [1, 700, 16, 333, 0], [1, 6, 3, 0, 0]),
    (8, 1, [95, 1300], [3, 2]),
    (3, 3, [24, 257], [24, 17]),
    (4, 2, [40, 1025, 31], [4, 1, 2]),
])
def test_chunk_attn_few_rows(hq, hkv, lens, news, mod):
    """A few query rows per kv head, most of a tile empty."""
    require_gpu()
    c = Case(hq, hkv, lens, news, mod, 70 + hq)
    out, lse, wk = c.chunk()
    c.check(out, lse, True)
    again, lse2, _ = c.chunk(wk)
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    assert not bool(wk.t.any())


@pytest.mark.parametrize("news,mod", [([3, 1], "plain"), ([40, 2], "cap_bias_scale"), ([9, 300], "window_sink"),
                                      ([700, 700], "docs_window_sink"), ([6, 6], "docs_window_sink")])
def test_chunk_attn_few_rows_over_a_long_cache(news, mod):
    require_gpu()
    c = Case(8, 2, [6011, 5000], news, mod, 92)
    out, lse, wk = c.chunk()
    rows = set(np.random.default_rng(4).integers(0, sum(news), 24).tolist()) | {0, sum(news) - 1}
    c.check(out, lse, True, rows)
    again, lse2, _ = c.chunk(wk)
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    assert not bool(wk.t.any())


def test_chunk_and_decode_agree_on_one_token():
    require_gpu()
    c = Case(8, 2, [1000, 31], [1, 1], "cap", 93)
    a, la, _ = c.decode()
    b, lb, _ = c.chunk(extra=0)
    assert torch.allclose(la, lb, rtol=1e-5, atol=1e-5)
    assert float((a - b.float()).abs().max()) <= 2 ** -10 * float(a.abs().max()) * 2


def test_batches_without_a_token():
    """Empty sequences only, with and without a block table; a batch of none; chunks without rows."""
    require_gpu()
    cache = kvq.LayerCache(8, 2, 16, 4, 3)
    for bt in (torch.zeros((3, 4), dtype=torch.int32, device="cuda"), torch.zeros((3, 0), dtype=torch.int32, device="cuda")):
        batch = kvq.Batch(bt, torch.zeros(3, dtype=torch.int32, device="cuda"), 0)
        batch.c.block_table = None
        q, out = rnd((3, 8, D), 40).cuda(), torch.full((3, 8, D), float("nan"), device="cuda")
        lse = torch.zeros((3, 8), device="cuda")
        wk = ws(kvq.kv_decode_attn_ws(cache, batch))
        kvq.kv_decode_attn(cache, batch, q, out, wk, lse=lse)
        kvq.kvq_check(wk)
        assert not bool(out.any()) and bool((lse == -math.inf).all())
        starts, o16 = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.full((3, 8, D), 7.0, device="cuda").half()
        wc = ws(kvq.kv_chunk_attn_ws(cache, batch, 3, 2))
        kvq.kv_chunk_attn(cache, batch, q, starts, 2, o16, wc)
        kvq.kvq_check(wc)
        assert bool((o16 == 7).all())
        kvq.kv_chunk_attn(cache, batch, q[:0], starts, 0, o16[:0], wc)
    none = kvq.Batch(torch.zeros((0, 4), dtype=torch.int32, device="cuda"), torch.zeros(0, dtype=torch.int32, device="cuda"), 64)
    kvq.kv_decode_attn(cache, none, q[:0], out[:0], wk)
    kvq.kv_chunk_attn(cache, none, q[:0], starts[:1], 1, o16[:0], wc)
    torch.cuda.synchronize()


def test_one_workspace_for_every_call():
    """Calls of all kinds and sizes in turn on one workspace: each finds it as it needs it."""
    require_gpu()
    cases = [Case(8, 2, [5000, 3], [40, 3], "cap", 110), Case(3, 3, [300] * 20, [1] * 20, "plain", 111),
             Case(8, 2, [9000], [1], "window_sink", 112), Case(4, 2, [50, 60], [1, 1], "docs", 113)]
    need = [max(kvq.kv_decode_attn_ws(c.cache, c.batch), kvq.kv_chunk_attn_ws(c.cache, c.batch, sum(c.news) + 2, max(c.news)))
            for c in cases]
    wk = ws(max(need))
    want = [(c.decode() if max(c.news) == 1 else c.chunk())[0] for c in cases]
    for _ in range(2):
        for c, w in zip(cases, want):
            got = (c.decode(wk) if max(c.news) == 1 else c.chunk(wk))[0]
            assert torch.equal(got, w)
    assert not bool(wk.t.any())


def test_pages_out_of_sight_may_be_stale():
    """With a window, pages behind it are given back: their table entries are stale, their rows another's."""
    require_gpu()
    for call, new in (("decode", 1), ("chunk", 50), ("chunk", 7)):
        c = Case(4, 2, [1000], [new], "window_sink", 94)
        gone = list(range(1, (1000 - 50 - 33) // 16))
        c.cache.k16[c.bt[0, gone].tolist()] = float("inf")
        c.cache.v16[c.bt[0, gone].tolist()] = float("nan")
        c.batch.block_table[0, gone] = torch.tensor([-1, 10 ** 6] * 100, dtype=torch.int32, device="cuda")[:len(gone)]
        out, lse, _ = getattr(c, call)()
        c.check(out, lse, call == "chunk")


def test_decode_attn_rows_out_of_sight_may_hold_nan():
    require_gpu()
    c = Case(8, 2, [300], [1], "docs", 95)
    c.doc = np.array([137], dtype=np.int32)
    c.mod = kvq.AttnMod(doc_start=torch.tensor(c.doc).cuda())
    for t in range(137):
        c.cache.k16[int(c.bt[0, t // 16]), :, t % 16] = float("nan")
        c.cache.v16[int(c.bt[0, t // 16]), :, t % 16] = float("inf")
    out, lse, _ = c.decode()
    c.check(out, lse, False)


def test_attention_device_checks():
    """A page outside the pool, a length outside its bounds and rows outside q are flagged, not followed."""
    require_gpu()
    c = Case(8, 2, [100, 40], [1, 1], "plain", 96)
    c.batch.block_table[0, 2] = 10 ** 6
    for call in (c.decode, lambda: c.chunk(extra=0)):
        with pytest.raises(kvq.KvqError) as e:
            call()
        assert e.value.code == _abi.KVQ_ERR_DEVICE_CHECK and "page id" in str(e.value)
    c = Case(8, 2, [100, 40], [1, 1], "plain", 97)
    c.batch.seq_lens[1] = 5000
    for call in (c.decode, lambda: c.chunk(extra=0)):
        with pytest.raises(kvq.KvqError) as e:
            call()
        assert "length" in str(e.value)
    c = Case(8, 2, [100, 40], [1, 1], "plain", 98)
    c.starts[2] = 9
    with pytest.raises(kvq.KvqError) as e:
        c.chunk(extra=0)
    assert "length" in str(e.value)


def test_attention_other_stream_and_graph():
    """On a stream of its own and captured: replays follow what the buffers hold then."""
    require_gpu()
    c = Case(8, 2, [900, 17], [1, 1], "cap", 99)
    want, _, wk = c.decode()
    want16, _, wk16 = c.chunk(extra=0)
    out, out16 = torch.zeros_like(want), torch.zeros_like(want16)
    starts = torch.tensor(c.starts).cuda()
    side, q = torch.cuda.Stream(), c.q.clone()
    side.wait_stream(torch.cuda.current_stream())
    def both():
        kvq.kv_decode_attn(c.cache, c.batch, q, out, wk, mod=c.mod, stream=side)
        kvq.kv_chunk_attn(c.cache, c.batch, q, starts, 1, out16, wk16, mod=c.mod, stream=side)
    both()
    side.synchronize()
    assert torch.equal(out, want) and torch.equal(out16, want16)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        both()
    q.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert not torch.equal(out, want)
    q.copy_(c.q)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(out16, want16)


# ------------------------------------------------------------------ pages and slots

def fill(cache, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    for name in ("k_codes", "v_codes", "k_sz", "v_sz", "k_tail", "k16", "v16", "kT", "k_absmax"):
        a = getattr(cache, name)
        if a is None:
            continue
        if a.dtype == torch.uint8:
            a.copy_(torch.randint(0, 256, a.shape, generator=g, device="cuda", dtype=torch.uint8))
        else:
            a.copy_(torch.randn(a.shape, generator=g, device="cuda"))
    return {n: getattr(cache, n).clone() for n in ("k_codes", "v_codes", "k_sz", "v_sz", "k_tail", "k16", "v16", "kT", "k_absmax")
            if getattr(cache, n) is not None}


@pytest.mark.parametrize("bits,G", [(1, 64), (2, 128), (4, 32), (4 | kvq.V_SYMMETRIC, 32), (8, 64), (kvq.BITS_E4M3, 64), (16, 64)])
@pytest.mark.parametrize("hkv,n", [(1, 1), (3, 7), (8, 40)])
def test_pages_copy(bits, G, hkv, n):
    require_gpu()
    c = kvq.LayerCache(hkv, hkv, bits, 2 * n + 5, 2, v_group_dims=G, t_cap=64 if bits == 16 else 0)
    before = fill(c, n)
    ids = torch.randperm(2 * n + 5, generator=torch.Generator().manual_seed(n))[:2 * n].to(torch.int32).view(n, 2)
    pairs = torch.cat([ids, torch.tensor([[3, 3]], dtype=torch.int32)])   # a pair of equal ids: nothing
    wk = ws(kvq.kv_pages_copy_ws())
    kvq.kv_pages_copy(c, pairs.cuda(), wk)
    kvq.kvq_check(wk)
    for name, a in before.items():
        if name in ("k_codes", "v_codes", "k_sz", "v_sz", "k16", "v16"):
            a[ids[:, 1].long()] = a[ids[:, 0].long()]
        assert torch.equal(getattr(c, name), a), name


def test_pages_copy_flags_bad_ids():
    require_gpu()
    c = kvq.LayerCache(4, 2, 16, 6, 1)
    before = fill(c, 1)
    wk = ws(kvq.kv_pages_copy_ws())
    kvq.kv_pages_copy(c, torch.tensor([[0, 6], [-1, 2], [4, 5]], dtype=torch.int32, device="cuda"), wk)
    with pytest.raises(kvq.KvqError) as e:
        kvq.kvq_check(wk)
    assert e.value.code == _abi.KVQ_ERR_DEVICE_CHECK
    for name, a in before.items():
        a[5] = a[4]
        assert torch.equal(getattr(c, name), a)
    kvq.kv_pages_copy(c, torch.zeros((0, 2), dtype=torch.int32, device="cuda"), wk)


@pytest.mark.parametrize("bits", [1, 4, kvq.BITS_E4M3, 16])
def test_slots_copy(bits):
    require_gpu()
    lens = [37, 0, 64, 5, 1]
    batch, _ = paged_batch([64] * 5, kvq.Allocator(20), lengths=lens)
    c = kvq.LayerCache(4, 2, bits, 20, 5, t_cap=64 if bits == 16 else 0)
    before = fill(c, bits)
    wk = ws(kvq.kv_slots_copy_ws())
    kvq.kv_slots_copy(c, batch, torch.tensor([[0, 3], [2, 4], [1, 1]], dtype=torch.int32, device="cuda"), wk)
    kvq.kvq_check(wk)
    for s, d in ((0, 3), (2, 4)):
        for name in ("k_tail", "k_absmax"):
            if name in before:
                before[name][d] = before[name][s]
    for name, a in before.items():
        got = getattr(c, name)
        if name == "kT":
            for s, d in ((0, 3), (2, 4)):
                assert torch.equal(got[d, ..., :lens[s]], a[s, ..., :lens[s]])
                keep = (lens[s] + 7) // 8 * 8
                assert torch.equal(got[d, ..., keep:], a[d, ..., keep:])
            assert torch.equal(got[:3], a[:3])
        else:
            assert torch.equal(got, a), name


@pytest.mark.parametrize("bits,T", [(4, 300), (4, 256), (1, 67), (16, 300), (16, 320), (kvq.BITS_E4M3, 77)])
def test_fork_then_append_keeps_both_branches(bits, T):
    """A fork shares full pages; both branches then append their own tokens past the end of a K group, and
    each attends exactly what a sequence of its own would hold."""
    require_gpu()
    Hq, Hkv, more = 8, 2, 70
    K, V = synth.kv_rows(T, Hkv, 5)
    tails = [synth.kv_rows(more, Hkv, 6 + b) for b in range(2)]
    cap = T + more
    alloc = kvq.Allocator(200, seed=3)
    n = math.ceil(T / 16)
    first = alloc.alloc(n)
    cache = kvq.LayerCache(Hq, Hkv, bits, 200, 2, v_group_dims=32)
    fork, pairs = alloc.fork(cache, T, first)
    assert len(pairs) == len(set(first) ^ set(fork)) // 2
    tables = [p + alloc.alloc(math.ceil(cap / 16) - n) for p in (first, fork)]
    batch = kvq.Batch(torch.tensor(tables, dtype=torch.int32, device="cuda"),
                      torch.tensor([T, T], dtype=torch.int32, device="cuda"), cap)
    kvq.kv_quant_pack(cache, batch, 0, 0, T, K.cuda(), V.cuda())
    wk = ws(256)
    if pairs:
        kvq.kv_pages_copy(cache, torch.tensor(pairs, dtype=torch.int32, device="cuda"), wk)
    kvq.kv_slots_copy(cache, batch, torch.tensor([[0, 1]], dtype=torch.int32, device="cuda"), wk)
    for i in range(more):
        kvq.kvq_seq_lens_add(batch.seq_lens, 1)
        kvq.kv_page_append(cache, batch, torch.stack([t[0][i] for t in tails]).cuda(),
                           torch.stack([t[1][i] for t in tails]).cuda(), wk)
    kvq.kvq_check(wk)
    q = rnd((2, Hq, D), 8).cuda()
    got = torch.empty((2, Hq, D), device="cuda")
    alone = torch.empty((2, Hq, D), device="cuda")
    attend = (lambda c, b, o: kvq.kv_decode_attn(c, b, q, o, ws(kvq.kv_decode_attn_ws(c, b)))) if bits == 16 else \
        (lambda c, b, o: kvq.kv_decode_attn_quant(c, b, q, o, ws(kvq.kv_decode_attn_quant_ws(c, b))))
    attend(cache, batch, got)
    ref = kvq.LayerCache(Hq, Hkv, bits, 200, 2, v_group_dims=32)
    rb, _ = paged_batch([cap, cap], kvq.Allocator(200))
    for b in range(2):
        k, v = torch.cat([K, tails[b][0]]).cuda(), torch.cat([V, tails[b][1]]).cuda()
        kvq.kv_quant_pack(ref, rb, b, 0, cap, k, v)
    attend(ref, rb, alone)
    assert torch.equal(got, alone)


def test_compaction_keeps_every_sequence():
    """Pages of finished sequences leave holes; compacting moves the others down, and attention is the same."""
    require_gpu()
    lens = [200, 333, 48, 500]
    alloc = kvq.Allocator(100, seed=11)
    held = [alloc.alloc(20), alloc.alloc(7)]
    batch, bt = paged_batch(lens, alloc)
    cache = kvq.LayerCache(4, 2, 16, 100, 4)
    for b, T in enumerate(lens):
        K, V = synth.kv_rows(T, 2, 30 + b)
        kvq.kv_quant_pack(cache, batch, b, 0, T, K.cuda(), V.cuda())
    q = rnd((4, 4, D), 9).cuda()
    a, b2 = torch.empty((4, 4, D), device="cuda"), torch.empty((4, 4, D), device="cuda")
    wk = ws(kvq.kv_decode_attn_ws(cache, batch))
    kvq.kv_decode_attn(cache, batch, q, a, wk)
    for pages in held:
        alloc.free_n(pages)
    pairs, new_id = alloc.compact()
    assert pairs
    kvq.kv_pages_copy(cache, torch.tensor(pairs, dtype=torch.int32, device="cuda"), wk)
    kvq.kvq_table_remap(batch.block_table, torch.tensor(new_id, dtype=torch.int32, device="cuda"), wk)
    used = sum(math.ceil(T / 16) for T in lens)
    table = batch.block_table.cpu().numpy()
    assert table.max() < used and np.array_equal(table < 0, bt < 0)
    kvq.kv_decode_attn(cache, batch, q, b2, wk)
    kvq.kvq_check(wk)
    assert torch.equal(a, b2)


# ------------------------------------------------------------------ together

def test_prompt_fork_and_decode_together():
    """A prompt in two chunks (norms, positions, pack, attention), a fork, then decode steps of both
    branches with norms, positions, append and attention, against the 64-bit forms on the same inputs."""
    require_gpu()
    Hq, Hkv, T, cut, steps = 8, 2, 150, 64, 3
    f, m = R.frequencies(128, 10000.0)
    tab, L = kvq.RopeTable(128, 10000.0), kvq.make_layout(8, 2, 16)
    w = (rnd((D,), 20, dtype=torch.float32).abs() + 0.5)
    rows = rnd((T + 2 * steps, (Hq + 2 * Hkv) * D), 21, dtype=torch.bfloat16)
    alloc = kvq.Allocator(64, seed=2)
    pages = alloc.alloc(math.ceil(T / 16))
    cache = kvq.LayerCache(Hq, Hkv, 16, 64, 2, t_cap=160)

    def project(x, pos):
        n = len(pos)
        x = x.cuda()
        q, k, v = (torch.empty((n, h, D), dtype=torch.float16, device="cuda") for h in (Hq, Hkv, Hkv))
        kvq.kv_qk_norm_rope(L, tab, torch.tensor(pos, dtype=torch.int32, device="cuda"), x[:, :Hq * D].view(n, Hq, D),
                            x[:, Hq * D:(Hq + Hkv) * D].view(n, Hkv, D), q, k, w.cuda(), w.cuda(), 1e-6,
                            x[:, (Hq + Hkv) * D:].view(n, Hkv, D), v)
        for y, x0, h in ((q, 0, Hq), (k, Hq, Hkv)):
            z, bound = R.norm_rope(R.as64(x[:, x0 * D:(x0 + h) * D].view(n, h, D)), np.array(pos), f, m, 128, False, R.as64(w))
            assert np.all(np.abs(R.as64(y) - z) <= bound)
        return q, k, v

    hist_k, hist_v = [[], []], [[], []]

    def expect(b, q, got, pos, fp16):
        K, V = np.concatenate(hist_k[b]), np.concatenate(hist_v[b])
        for h in range(Hq):
            o, _, bound, _ = R.attend(R.as64(q[h]), K[:, h // 4], V[:, h // 4], R.visible(len(K), pos), pos, fp16=fp16)
            assert np.all(np.abs(R.as64(got[h]) - o) <= bound)

    table = torch.full((2, 10), -1, dtype=torch.int32, device="cuda")
    table[0, :len(pages)] = torch.tensor(pages, dtype=torch.int32)
    lens = torch.zeros(2, dtype=torch.int32, device="cuda")
    batch = kvq.Batch(table, lens, 160)
    for lo, hi in ((0, cut), (cut, T)):
        q, k, v = project(rows[lo:hi], list(range(lo, hi)))
        kvq.kv_quant_pack(cache, batch, 0, lo, hi - lo, k, v)
        lens[0] = hi
        out = torch.empty((hi - lo, Hq, D), dtype=torch.float16, device="cuda")
        wk = ws(kvq.kv_chunk_attn_ws(cache, batch, hi - lo, hi - lo))
        kvq.kv_chunk_attn(cache, batch, q, torch.tensor([0, hi - lo, hi - lo], dtype=torch.int32, device="cuda"), hi - lo, out, wk)
        kvq.kvq_check(wk)
        hist_k[0].append(R.as64(k))
        hist_v[0].append(R.as64(v))
        for i in (0, 1, hi - lo - 1):
            expect(0, q[i], out[i], lo + i, True)
    fork, pairs = alloc.fork(cache, T, pages)
    wk = ws(256)
    kvq.kv_pages_copy(cache, torch.tensor(pairs, dtype=torch.int32, device="cuda"), wk)
    kvq.kv_slots_copy(cache, batch, torch.tensor([[0, 1]], dtype=torch.int32, device="cuda"), wk)
    table[1, :len(fork)] = torch.tensor(fork, dtype=torch.int32)
    lens[1] = T
    batch = kvq.Batch(table, lens, 160)
    hist_k[1], hist_v[1] = list(hist_k[0]), list(hist_v[0])
    out = torch.empty((2, Hq, D), device="cuda")
    wd = ws(kvq.kv_decode_attn_ws(cache, batch))
    for s in range(steps):
        q, k, v = project(rows[T + 2 * s:T + 2 * s + 2], [T + s, T + s])
        kvq.kvq_seq_lens_add(lens, 1)
        kvq.kv_page_append(cache, batch, k, v, wk)
        kvq.kv_decode_attn(cache, batch, q, out, wd)
        kvq.kvq_check(wd)
        for b in range(2):
            hist_k[b].append(R.as64(k[b:b + 1]))
            hist_v[b].append(R.as64(v[b:b + 1]))
            expect(b, q[b], out[b], T + s, False)
    # the sparse path of the same layer reads the fork's slot state
    sparse = torch.empty((2, Hq, D), device="cuda")
    qn, kn, vn = project(rows[:2], [T + steps, T + steps])
    kvq.kvq_seq_lens_add(lens, 1)
    kvq.kv_sparse_layer_decode(cache, batch, kn, vn, qn, 8, 160, 0.0, 4, 16, sparse, ws(kvq.kv_sparse_layer_decode_ws()))
    kvq.kv_decode_attn(cache, batch, qn, out, wd)
    for b in range(2):
        for h in range(Hq):
            assert attn_err(sparse[b, h].cpu().numpy(), out[b, h].cpu().numpy()) <= ATTN_TOL


# ------------------------------------------------------------------ what the binding refuses

def test_binding_refuses_wrong_tensors():
    """Wrong type, shape, gaps or place: refused before a bare pointer is taken."""
    require_gpu()
    c = Case(8, 2, [40], [1], "plain", 101)
    wk = ws(kvq.kv_decode_attn_ws(c.cache, c.batch))
    wc = ws(kvq.kv_chunk_attn_ws(c.cache, c.batch, 1, 1))
    out, out16 = torch.zeros((1, 8, D), device="cuda"), torch.zeros((1, 8, D), device="cuda", dtype=torch.float16)
    starts = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    gaps = torch.zeros((1, 16, D), device="cuda", dtype=torch.float16)[:, ::2]
    few = kvq.AttnMod(slopes=torch.ones(4, device="cuda"))
    docs = kvq.AttnMod(doc_start=torch.zeros(0, dtype=torch.int32, device="cuda"))
    L, tab = kvq.make_layout(8, 2, 16), kvq.RopeTable(128)
    pos, k = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros((1, 2, D), dtype=torch.float16, device="cuda")
    pairs = torch.zeros((1, 2), dtype=torch.int32, device="cuda")
    for call in (
            lambda: kvq.kv_decode_attn(c.cache, c.batch, c.q.float(), out, wk),
            lambda: kvq.kv_decode_attn(c.cache, c.batch, c.q.cpu(), out, wk),
            lambda: kvq.kv_decode_attn(c.cache, c.batch, gaps, out, wk),
            lambda: kvq.kv_decode_attn(c.cache, c.batch, c.q, out16, wk),
            lambda: kvq.kv_decode_attn(c.cache, c.batch, c.q, out[:, :4], wk),
            lambda: kvq.kv_decode_attn(c.cache, c.batch, None, out, wk),
            lambda: kvq.kv_decode_attn(c.cache, c.batch, c.q, out, wk, mod=few),
            lambda: kvq.kv_decode_attn(c.cache, c.batch, c.q, out, wk, mod=docs),
            lambda: kvq.kv_decode_attn(c.cache, c.batch, c.q, out, wk, lse=out),
            lambda: kvq.kv_chunk_attn(c.cache, c.batch, c.q, starts.long(), 1, out16, wc),
            lambda: kvq.kv_chunk_attn(c.cache, c.batch, c.q, starts[:1], 1, out16, wc),
            lambda: kvq.kv_chunk_attn(c.cache, c.batch, c.q, starts, 1, out, wc),
            lambda: kvq.kv_chunk_attn(c.cache, c.batch, c.q, starts, 0, out16, wc),
            lambda: kvq.kv_qk_norm_rope(L, tab, pos, None, k, None, k.float()),
            lambda: kvq.kv_qk_norm_rope(L, tab, pos, None, k.float(), None, k),
            lambda: kvq.kv_qk_norm_rope(L, tab, pos, None, k, None, None),
            lambda: kvq.kv_qk_norm_rope(L, tab, None, None, k, None, k),
            lambda: kvq.kv_qk_norm_rope(L, tab, pos.long(), None, k, None, k),
            lambda: kvq.kv_qk_norm_rope(L, tab, pos, None, None, None, None),
            lambda: kvq.kv_qk_norm_rope(L, tab, pos, k, None, k, None),
            lambda: kvq.kv_qk_norm_rope(L, tab, pos, None, k, None, k, k_weight=torch.ones(64, device="cuda")),
            lambda: kvq.kv_qk_norm_rope(L, tab, pos, None, k.transpose(1, 2).contiguous().transpose(1, 2), None, torch.zeros_like(k)),
            lambda: kvq.kv_pages_copy(c.cache, pairs.long(), wk),
            lambda: kvq.kv_pages_copy(c.cache, pairs.flatten(), wk),
            lambda: kvq.kv_slots_copy(c.cache, c.batch, pairs.cpu(), wk),
            lambda: kvq.kvq_table_remap(c.batch.block_table, pairs.cpu(), wk),
            lambda: kvq.AttnMod(slopes=torch.ones(8, device="cuda", dtype=torch.float16))):
        with pytest.raises(kvq.KvqError) as e:
            call()
        assert e.value.code in (_abi.KVQ_ERR_INVALID_ARG, _abi.KVQ_ERR_UNSUPPORTED)
    with pytest.raises(kvq.KvqError):
        kvq.RopeTable(128, scaling="other")


# ------------------------------------------------------------------ at the edges of what the calls allow

def test_two_streams_at_once():
    """Calls that overlap on the GPU, each with its own workspace, give what they give alone."""
    require_gpu()
    cases = [Case(8, 2, [3000, 2000], [700, 300], "plain", 120), Case(8, 2, [2500, 900], [600, 900], "cap", 121)]
    dec = [Case(8, 2, [20000], [1], "plain", 122), Case(3, 3, [900] * 20, [1] * 20, "bias", 123)]
    want = [c.chunk(extra=0)[0] for c in cases] + [c.decode()[0] for c in dec]
    streams = [torch.cuda.Stream() for _ in range(4)]
    outs, keep = [], []
    for c in cases:
        outs.append(torch.empty((c.q.shape[0], c.hq, D), dtype=torch.float16, device="cuda"))
        keep.append((torch.tensor(c.starts).cuda(), ws(kvq.kv_chunk_attn_ws(c.cache, c.batch, c.q.shape[0], max(c.news)))))
    for c in dec:
        outs.append(torch.empty((len(c.lens), c.hq, D), device="cuda"))
        keep.append((None, ws(kvq.kv_decode_attn_ws(c.cache, c.batch))))
    torch.cuda.synchronize()
    for _ in range(10):
        for c, o, (st, wk), s in zip(cases, outs, keep, streams):
            kvq.kv_chunk_attn(c.cache, c.batch, c.q, st, max(c.news), o, wk, mod=c.mod, stream=s)
        for c, o, (_, wk), s in zip(dec, outs[2:], keep[2:], streams[2:]):
            kvq.kv_decode_attn(c.cache, c.batch, c.q, o, wk, mod=c.mod, stream=s)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)


def test_pages_beyond_32_bit_offsets():
    """A pool whose last pages lie more than 2^31 values from its first."""
    require_gpu()
    H, n, T = 8, 140000, 300
    low = kvq.LayerCache(H, H, 16, 40, 1)
    cache = kvq.LayerCache(H, H, 16, n, 1)
    assert (n - 40) * H * 16 * D > 2 ** 31
    K, V = synth.kv_rows(T, H, 77)
    pages = math.ceil(T / 16)
    far = torch.arange(n - pages, n, dtype=torch.int32, device="cuda")[None]
    near = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    lens = torch.tensor([T], dtype=torch.int32, device="cuda")
    batches = [kvq.Batch(far, lens, T), kvq.Batch(near, lens, T)]
    for c, b in zip((cache, low), batches):
        kvq.kv_quant_pack(c, b, 0, 0, T, K.cuda(), V.cuda())
    q = rnd((40, H, D), 50).cuda()
    starts = torch.tensor([0, 40], dtype=torch.int32, device="cuda")
    got = []
    for c, b in zip((cache, low), batches):
        o, o16 = torch.empty((1, H, D), device="cuda"), torch.empty((40, H, D), dtype=torch.float16, device="cuda")
        kvq.kv_decode_attn(c, b, q[:1], o, ws(kvq.kv_decode_attn_ws(c, b)))
        kvq.kv_chunk_attn(c, b, q, starts, 40, o16, ws(kvq.kv_chunk_attn_ws(c, b, 40, 40)))
        got.append((o, o16))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    wk = ws(256)
    kvq.kv_pages_copy(cache, torch.stack([far[0], near[0]], dim=1).contiguous(), wk)
    kvq.kvq_check(wk)
    assert torch.equal(cache.k16[:pages], low.k16[:pages]) and torch.equal(cache.v16[:pages], low.v16[:pages])


@pytest.mark.parametrize("window,sink", [(2 ** 31 - 1, 2 ** 31 - 1), (2 ** 31 - 1, 0), (1, 2 ** 31 - 1)])
def test_largest_window_and_sinks_see_everything(window, sink):
    require_gpu()
    for news in ([1], [33]):
        c = Case(4, 2, [700], news, "plain", 130)
        run = c.decode if news == [1] else c.chunk
        want = run()
        c.mod = kvq.AttnMod(window=window, n_sink=sink)
        got = run()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_document_starts_outside_the_sequence():
    """Before its beginning: all of it; behind its end: nothing."""
    require_gpu()
    for news in ([1], [5]):
        c = Case(4, 2, [90], news, "plain", 131)
        run = c.decode if news == [1] else (lambda: c.chunk(extra=0))
        want = run()
        for start, same in ((-2 ** 31, True), (-1, True), (90, False), (2 ** 31 - 1, False)):
            c.mod = kvq.AttnMod(doc_start=torch.full((news[0],), start, dtype=torch.int32, device="cuda"))
            out, lse, _ = run()
            if same:
                assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
            else:
                assert not bool(out.any()) and bool((lse == -math.inf).all())


def test_more_new_tokens_than_announced():
    """max_new bounds every sequence's rows: a longer run is flagged and left out, the others are attended."""
    require_gpu()
    c = Case(4, 2, [90, 200], [5, 80], "plain", 132)
    want = c.chunk(extra=0)[0]
    out = torch.full((85, 4, D), -7.0, dtype=torch.float16, device="cuda")
    wk = ws(kvq.kv_chunk_attn_ws(c.cache, c.batch, 85, 80))
    kvq.kv_chunk_attn(c.cache, c.batch, c.q, torch.tensor(c.starts).cuda(), 79, out, wk)
    with pytest.raises(kvq.KvqError) as e:
        kvq.kvq_check(wk)
    assert e.value.code == _abi.KVQ_ERR_DEVICE_CHECK
    assert torch.equal(out[:5], want[:5]) and bool((out[5:] == -7).all())


def test_scores_of_minus_infinity():
    """A visible key of -inf against a positive query: weight 0; nothing else visible: output 0."""
    require_gpu()
    c = Case(2, 2, [40], [1], "plain", 133)
    c.q[:] = 1.0
    for t in range(20, 40):
        c.cache.k16[int(c.bt[0, t // 16]), :, t % 16] = -math.inf
    out, lse, _ = c.decode()
    c.lens, keep = [40], [(K.clone(), V) for K, V in c.KV]
    K, V = R.as64(keep[0][0]), R.as64(keep[0][1])
    for h in range(2):
        o, z, bo, bz = R.attend(np.ones(D), K[:, h], V[:, h], np.arange(40) < 20, 39)
        assert np.all(np.abs(R.as64(out[0, h]) - o) <= bo) and abs(float(lse[0, h]) - z) <= bz
    c.mod = kvq.AttnMod(window=20)
    out, lse, _ = c.decode()
    assert not bool(out.any()) and bool((lse == -math.inf).all())
