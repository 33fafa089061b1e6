"""Host side of the new-token operators: rotary frequencies, fork / compaction / bulk free of the page
allocator, and what the calls refuse before anything is launched."""
import ctypes
import math
from fractions import Fraction

import numpy as np
import pytest

import new_token_ref as R
from compressed_kv_cache_quant_gb300 import _abi, kvq
from compressed_kv_cache_quant_gb300.build import build

pytestmark = pytest.mark.cpu
BAD, UNSUP = _abi.KVQ_ERR_INVALID_ARG, _abi.KVQ_ERR_UNSUPPORTED
by = ctypes.byref


@pytest.fixture(scope="module")
def lib():
    build()
    return kvq.lib()


def steps_of(lib, *spec):
    r = _abi.Rope(*spec)
    out, m = (ctypes.c_uint64 * 64)(), ctypes.c_float(0)
    st = lib.kvq_rope_steps(by(r), out, by(m))
    return st, [out[i] for i in range(r.rot_dim // 2)], m.value


@pytest.mark.parametrize("rot", [16, 64, 96, 128])
@pytest.mark.parametrize("kind,name,factor,original,low,high", [
    (0, "plain", 1.0, 0, 0.0, 0.0), (1, "linear", 4.0, 0, 0.0, 0.0), (2, "ntk", 8.0, 0, 0.0, 0.0),
    (3, "yarn", 4.0, 32768, 32.0, 1.0), (4, "knees", 8.0, 8192, 1.0, 4.0)])
def test_rope_steps(lib, rot, kind, name, factor, original, low, high):
    st, steps, m = steps_of(lib, rot, 0, kind, original, 500000.0, factor, low, high)
    f, want_m = R.frequencies(rot, 500000.0, name, factor, original, low, high)
    assert st == 0 and m == np.float32(want_m)
    for s, x in zip(steps, f):
        # a few roundings of a double (pow and log are within an ulp or two), and the fraction's last bits
        assert abs(s - x / (2 * math.pi) * 2 ** 64) <= 2 ** 64 * x * 2.0 ** -49 + 2


def test_rope_angle_is_exact_at_far_positions(lib):
    """position * step modulo 2^64 is the angle modulo one turn."""
    _, steps, _ = steps_of(lib, 128, 0, 0, 0, 10000.0, 1.0, 0.0, 0.0)
    for p in (1, 131071, 10 ** 6 + 3, 2 ** 31 - 1, -77777):
        for s in steps[::7]:
            exact = Fraction(p * s, 2 ** 64) % 1
            assert Fraction((p * s) % 2 ** 64, 2 ** 64) == exact


def test_rope_refusals(lib):
    for spec, want in (((24, 0, 0, 0, 1e4, 1.0, 0.0, 0.0), UNSUP), ((144, 0, 0, 0, 1e4, 1.0, 0.0, 0.0), UNSUP),
                       ((-16, 0, 0, 0, 1e4, 1.0, 0.0, 0.0), UNSUP), ((64, 2, 0, 0, 1e4, 1.0, 0.0, 0.0), BAD),
                       ((64, 0, 5, 0, 1e4, 1.0, 0.0, 0.0), UNSUP), ((64, 0, 0, 0, 1.0, 1.0, 0.0, 0.0), BAD),
                       ((64, 0, 0, 0, math.nan, 1.0, 0.0, 0.0), BAD), ((64, 0, 1, 0, 1e4, 0.5, 0.0, 0.0), BAD),
                       ((64, 0, 3, 0, 1e4, 4.0, 32.0, 1.0), BAD), ((64, 0, 3, 8192, 1e4, 4.0, 1.0, 32.0), BAD),
                       ((64, 0, 4, 8192, 1e4, 4.0, 4.0, 1.0), BAD), ((64, 0, 4, 8192, 1e4, 4.0, 0.0, 1.0), BAD)):
        assert lib.kvq_rope_steps(by(_abi.Rope(*spec)), (ctypes.c_uint64 * 128)(), by(ctypes.c_float())) == want, spec
    assert lib.kvq_rope_steps(None, None, None) == BAD
    assert steps_of(lib, 0, 0, 0, 0, 0.0, 0.0, 0.0, 0.0)[0] == 0   # no rotation: nothing to describe


def norm_rope(lib, rot=128, inter=0, dtype=0, n=4, pos=256, q=256, qs=1024, k=256, ks=256, v=None, vs=0, wq=None, wk=None,
              eps=1e-6, qo=512, ko=512, vo=None, steps=256, layout=None, mscale=1.0):
    L = layout or kvq.make_layout(8, 2, 16)
    r = _abi.Rope(rot, inter, 0, 0, 1e4, 1.0, 0.0, 0.0)
    return lib.kv_qk_norm_rope(by(L), by(r), steps, mscale, dtype, n, pos, q, qs, k, ks, v, vs, wq, wk, eps, qo, ko, vo, None)


def test_norm_rope_refusals(lib):
    """Pointers here are never followed: each call is refused on the host (or has no tokens)."""
    assert norm_rope(lib, n=0) == 0
    for bad in (dict(rot=24), dict(dtype=2)):
        assert norm_rope(lib, **bad) == UNSUP, bad
    for bad in (dict(inter=7), dict(n=-1), dict(pos=None), dict(steps=None), dict(qs=1016), dict(ks=255), dict(ks=260),
                dict(q=264), dict(ko=520), dict(qo=None), dict(q=None, k=None, qo=None, ko=None), dict(v=256, vs=256),
                dict(vo=256), dict(q=None, qo=None, wq=256), dict(eps=-1.0), dict(eps=math.nan), dict(mscale=math.inf),
                dict(q=256, qo=256, qs=1032), dict(q=256, qo=256, dtype=1)):
        assert norm_rope(lib, **bad) == BAD, bad
    assert lib.kv_qk_norm_rope(None, None, None, 1.0, 0, 0, *([None] * 2), 0, None, 0, None, 0, None, None, 0.0, *([None] * 4)) == BAD


def seqs(batch=2, max_blocks=8, max_len=100, bt=256, lens=256):
    return _abi.Seqs(bt, lens, batch, max_blocks, max_len, 0)


def pool(**k):
    return _abi.Pool(**{**dict(num_blocks=16, max_seqs=4, t_cap=0, k16=256, v16=256), **k})


@pytest.mark.parametrize("call", ["decode", "chunk"])
def test_attention_refusals(lib, call):
    L = kvq.make_layout(8, 2, 16)
    big = 1 << 30

    def go(layout=L, P=None, S=None, q=256, out=256, ws=256, nbytes=big, mod=None, starts=256, rows=4, most=2):
        P, S, mod = P or pool(), S or seqs(), by(mod) if mod is not None else None
        if call == "decode":
            return lib.kv_decode_attn(by(layout), by(P), by(S), q, mod, out, None, ws, nbytes, None)
        return lib.kv_chunk_attn(by(layout), by(P), by(S), q, starts, rows, most, mod, out, None, ws, nbytes, None)

    assert go(S=seqs(batch=0)) == 0
    assert go(layout=kvq.make_layout(8, 2, 4)) == UNSUP and go(layout=kvq.make_layout(24, 2, 16)) == UNSUP
    assert go(layout=kvq.make_layout(6, 4, 16)) == BAD
    for bad in (dict(P=pool(k16=None)), dict(P=pool(num_blocks=0)), dict(P=pool(v16=264)), dict(S=seqs(max_len=129)),
                dict(S=seqs(batch=-1)), dict(S=seqs(lens=None)), dict(S=seqs(bt=None)), dict(q=None), dict(q=264), dict(out=None),
                dict(out=264), dict(ws=None), dict(ws=264), dict(nbytes=128)):
        assert go(**bad) == BAD, bad
    M = _abi.AttnModStruct
    for bad in (M(-1.0), M(math.nan), M(math.inf), M(0.0, -1.0), M(0.0, math.nan), M(0.0, 0.0, -1), M(0.0, 0.0, 1, -1),
                M(1e38, 1e-38)):
        assert go(mod=bad) == BAD, (bad.scale, bad.softcap, bad.window, bad.n_sink)
    if call == "chunk":
        for bad in (dict(starts=None), dict(rows=-1), dict(most=-1), dict(rows=4, most=0)):
            assert go(**bad) == BAD, bad
        assert go(rows=0) == 0
        assert lib.kv_chunk_attn_ws(by(L), by(seqs()), -1, 2) == 0 and lib.kv_chunk_attn_ws(by(L), by(seqs()), 4, 2) % 256 == 0
    assert lib.kv_decode_attn_ws(None, None) == 0 and lib.kv_decode_attn_ws(by(L), by(seqs())) % 256 == 0


def test_copy_refusals(lib):
    L, S = kvq.make_layout(8, 2, 16), seqs()
    assert lib.kv_pages_copy(by(L), by(pool()), None, 0, 256, 256, None) == 0
    for args in ((by(L), None, 256, 1, 256, 256), (by(L), by(pool()), None, 1, 256, 256), (by(L), by(pool()), 256, -1, 256, 256),
                 (by(L), by(pool(v16=None)), 256, 1, 256, 256), (by(L), by(pool(k16=8)), 256, 1, 256, 256),
                 (by(L), by(pool()), 256, 1, None, 256), (by(L), by(pool()), 256, 1, 256, 8), (None, by(pool()), 256, 1, 256, 256)):
        assert lib.kv_pages_copy(*args, None) == BAD
    Q = kvq.make_layout(8, 2, 4)
    assert lib.kv_pages_copy(by(Q), by(pool()), 256, 1, 256, 256, None) == BAD          # no code arrays
    assert lib.kv_pages_copy(by(kvq.make_layout(8, 2, 4, 48)), by(pool()), 256, 1, 256, 256, None) == UNSUP
    assert lib.kv_slots_copy(by(L), by(pool()), by(S), 256, 1, 256, 256, None) == 0     # no slot state: nothing to copy
    for args in ((by(Q), by(pool()), by(S), 256, 1, 256, 256), (by(L), by(pool(kT=256)), by(S), 256, 1, 256, 256),
                 (by(L), by(pool(kT=256, k_absmax=256)), by(S), 256, 1, 256, 256), (by(L), by(pool()), None, 256, 1, 256, 256),
                 (by(L), by(pool(kT=264, k_absmax=256, t_cap=64)), by(S), 256, 1, 256, 256),
                 (by(L), by(pool()), by(seqs(batch=5)), 256, 1, 256, 256)):
        assert lib.kv_slots_copy(*args, None) == BAD
    assert lib.kvq_table_remap(None, 0, 256, 4, 256, 256, None) == 0
    for args in ((None, 1, 256, 4, 256, 256), (256, -1, 256, 4, 256, 256), (256, 1, None, 4, 256, 256), (256, 1, 256, 0, 256, 256),
                 (256, 1, 256, 4, None, 256)):
        assert lib.kvq_table_remap(*args, None) == BAD


# ------------------------------------------------------------------ allocator

@pytest.mark.parametrize("bits,T,copied", [(16, 0, 0), (16, 1, 1), (16, 16, 0), (16, 17, 1), (16, 100, 1), (kvq.BITS_E4M3, 33, 1),
                                           (4, 64, 0), (4, 65, 1), (4, 96, 2), (4, 127, 4), (1, 130, 1), (8, 63, 4), (2, 128, 0)])
def test_fork(lib, bits, T, copied):
    a = kvq.Allocator(40, seed=4)
    n = math.ceil(T / 16)
    pages = a.alloc(n)
    fork, pairs = a.fork(kvq.make_layout(8, 2, bits), T, pages)
    assert len(pairs) == copied and len(fork) == n
    assert [p[0] for p in pairs] == pages[n - copied:] and [p[1] for p in pairs] == fork[n - copied:]
    assert fork[:n - copied] == pages[:n - copied] and not set(fork[n - copied:]) & set(pages)
    assert all(a.refcount(p) == 2 for p in pages[:n - copied]) and all(a.refcount(p) == 1 for p in pages[n - copied:] + fork[n - copied:])
    assert a.num_free() == 40 - n - copied
    a.free_n(fork)
    a.free_n(pages)
    assert a.num_free() == 40


def test_fork_refusals_take_nothing(lib):
    a = kvq.Allocator(5)
    pages = a.alloc(4)
    L = kvq.make_layout(8, 2, 4)
    with pytest.raises(kvq.KvqError) as e:
        a.fork(L, 63, pages)          # four pages to copy, one free
    assert e.value.code == _abi.KVQ_ERR_NO_SPACE
    for bad in ([pages[0], 4, pages[2], pages[3]], [pages[0], -1, 1, 1], [99] + pages[1:]):
        with pytest.raises(kvq.KvqError):
            a.fork(L, 63, bad)
    with pytest.raises(kvq.KvqError):
        a.fork(L, 65, pages)          # too few pages for the tokens
    with pytest.raises(kvq.KvqError):
        a.fork(kvq.make_layout(8, 2, 3), 16, pages)
    assert a.num_free() == 1 and all(a.refcount(p) == 1 for p in pages)


def test_free_n(lib):
    a = kvq.Allocator(6)
    x = a.alloc(4)
    a.ref(x[1])
    for bad in (x + [x[0]], x + [5], x + [-1], x + [6], [x[1]] * 3):
        with pytest.raises(kvq.KvqError):
            a.free_n(bad)
        assert [a.refcount(p) for p in x] == [1, 2, 1, 1] and a.num_free() == 2
    a.free_n([x[1], x[0], x[1]])
    assert [a.refcount(p) for p in x] == [0, 0, 1, 1] and a.num_free() == 4
    a.free_n([])
    assert len(set(a.alloc(4)) | {x[2], x[3]}) == 6     # every freed page is handed out once


@pytest.mark.parametrize("seed", range(6))
def test_compact(lib, seed):
    g = np.random.default_rng(seed)
    a = kvq.Allocator(60, seed=seed)
    live = {p: 1 for p in a.alloc(50)}
    for p in list(live)[::3]:
        a.ref(p)
        live[p] = 2
    for p in g.permutation(list(live))[:25].tolist():
        for _ in range(live.pop(p)):
            a.free(p)
    if seed == 5:
        pairs, _ = a.compact(3)
        assert len(pairs) <= 3
        live = {dict(pairs).get(p, p): r for p, r in live.items()}
    pairs, new_id = a.compact()
    src, dst = {p[0] for p in pairs}, {p[1] for p in pairs}
    assert not src & dst and len(src) == len(dst) == len(pairs) and src <= set(live)
    moved = {new_id[p]: r for p, r in live.items()}
    assert sorted(moved) == list(range(len(live))) and all(a.refcount(p) == r for p, r in moved.items())
    assert all(a.refcount(p) == 0 for p in range(len(live), 60)) and a.num_free() == 60 - len(live)
    assert a.alloc(2) == [len(live), len(live) + 1]
    assert a.compact(0)[0] == []
