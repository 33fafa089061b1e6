"""Host side of the appends, of tree attention and of latent layers: what the calls refuse before anything is launched,
and the sizes of their workspaces."""
import ctypes
import math

import pytest
import torch

from compressed_kv_cache_quant_gb300 import _abi, kvq
from compressed_kv_cache_quant_gb300.build import build

pytestmark = pytest.mark.cpu
BAD, UNSUP = _abi.KVQ_ERR_INVALID_ARG, _abi.KVQ_ERR_UNSUPPORTED
by = ctypes.byref


@pytest.fixture(scope="module")
def lib():
    build()
    return kvq.lib()


def seqs(batch=2, max_blocks=4, max_len=64, bt=256, lens=256):
    return _abi.Seqs(bt, lens, batch, max_blocks, max_len, 0)


def pool(bits=16, kT=None, top=None, t_cap=64, blocks=8, max_seqs=2, k=256, v=256):
    fp8 = bits == _abi.BITS_E4M3
    return _abi.Pool(blocks, max_seqs, t_cap, k if fp8 else None, v if fp8 else None, None, None, None,
                     None if fp8 else k, None if fp8 else v, kT, top)


def rope(rot=128, inter=0):
    return _abi.Rope(rot, inter, 0, 0, 1e4, 1.0, 0.0, 0.0)


# Pointers here are never followed: each call is refused on the host (or has no rows).

def append(lib, bits=16, P=None, S=None, R=None, steps=256, mscale=1.0, dtype=0, n=4, starts=256, pos=None, q=256, qs=1024, k=256,
           ks=256, v=256, vs=256, wq=None, wk=None, eps=1e-6, qo=512, ws=256, nbytes=256, hq=8, hkv=2):
    L = kvq.make_layout(hq, hkv, bits)
    return lib.kv_rope_append(by(L), by(P or pool(bits)), by(S or seqs()), by(R or rope()), steps, mscale, dtype, n, starts, pos, q, qs,
                              k, ks, v, vs, wq, wk, eps, qo, ws, nbytes, None)


def test_rope_append_refusals(lib):
    assert append(lib, n=0) == 0 and append(lib, S=seqs(batch=0)) == 0
    assert append(lib, n=0, q=None, qo=None, k=None, v=None) == 0
    for bad in (dict(bits=4), dict(bits=8), dict(bits=16 | _abi.V_SYMMETRIC), dict(dtype=2), dict(R=rope(24)),
                dict(S=seqs(max_blocks=1 << 27, max_len=(1 << 30) + 1))):
        assert append(lib, **bad) == UNSUP, bad
    for bad in (dict(R=rope(64, 3)), dict(n=-1), dict(n=1 << 31), dict(starts=None), dict(S=seqs(bt=None)), dict(S=seqs(lens=None)),
                dict(S=seqs(batch=3)), dict(S=seqs(max_len=65)), dict(k=None), dict(v=None), dict(q=None), dict(qo=None),
                dict(q=None, qo=None, wq=256), dict(steps=None), dict(mscale=math.nan), dict(eps=-1.0), dict(eps=math.inf),
                dict(qs=1016), dict(ks=248), dict(vs=255), dict(ks=260), dict(q=264), dict(k=8), dict(v=8), dict(qo=520),
                dict(q=512, qs=1032), dict(q=512, dtype=1), dict(ws=None), dict(ws=264), dict(nbytes=255),
                dict(P=pool(k=None)), dict(P=pool(v=8)), dict(P=pool(kT=256)), dict(P=pool(top=256)), dict(P=pool(kT=256, top=256, t_cap=60)),
                dict(P=pool(kT=264, top=256)), dict(P=pool(kT=256, top=256, t_cap=0)), dict(P=pool(blocks=0)), dict(P=pool(blocks=1 << 31)),
                dict(bits=_abi.BITS_E4M3, P=pool(16)), dict(bits=_abi.BITS_E4M3, P=pool(_abi.BITS_E4M3, k=264))):
        assert append(lib, **bad) == BAD, bad
    assert lib.kv_rope_append(None, None, None, None, None, 1.0, 0, 0, None, None, None, 0, None, 0, None, 0, None, None, 0.0, None, None, 0,
                              None) == BAD
    assert lib.kv_rope_append_ws() == 256


def test_rope_append_refuses_head_counts_that_pass_32_bits(lib):
    """2 + 2 (2^31 - 1) is 0 in 32 bits: no such count may reach the division of a CTA's rows."""
    most = (1 << 31) - 1
    for heads in (dict(hq=2, hkv=most), dict(hq=most, hkv=most), dict(hq=2, hkv=1 << 30), dict(hq=(1 << 16) + 1), dict(hkv=(1 << 16) + 1)):
        for bits in (16, _abi.BITS_E4M3):
            assert append(lib, bits=bits, qs=1 << 39, ks=1 << 39, vs=1 << 39, **heads) == UNSUP, heads
    assert "65536" in _abi.last_error()


def latent(dim=512, rot=64, blocks=8, rows=256):
    return _abi.Latent(dim, rot, blocks, rows)


def latent_append(lib, C=None, S=None, R=None, steps=256, dtype=0, n=4, starts=256, pos=None, c=256, cs=576, k=256, ks=576, cw=None, eps=1e-6,
                  heads=2, q=256, qs=128, qh=64, qo=512, os=1152, oh=576, ws=256, nbytes=256, mscale=1.0):
    return lib.kv_latent_append(by(C or latent()), by(S or seqs()), by(R or rope(64)), steps, mscale, dtype, n, starts, pos, c, cs, k, ks, cw, eps,
                                heads, q, qs, qh, qo, os, oh, ws, nbytes, None)


def test_latent_append_refusals(lib):
    assert latent_append(lib, n=0) == 0 and latent_append(lib, S=seqs(batch=0)) == 0
    for bad in (dict(C=latent(dim=256)), dict(C=latent(rot=32)), dict(R=rope(128)), dict(R=rope(0)), dict(dtype=3),
                dict(S=seqs(max_blocks=1 << 27, max_len=(1 << 30) + 1))):
        assert latent_append(lib, **bad) == UNSUP, bad
    for bad in (dict(C=latent(rows=None)), dict(C=latent(rows=8)), dict(C=latent(blocks=0)), dict(C=latent(blocks=1 << 31)), dict(n=-1),
                dict(starts=None), dict(c=None), dict(k=None), dict(steps=None), dict(cs=504), dict(ks=56), dict(cs=580), dict(qs=56), dict(qh=68),
                dict(oh=56), dict(os=1156), dict(c=264), dict(k=264), dict(q=264), dict(qo=520), dict(cw=260), dict(q=None), dict(qo=None),
                dict(heads=0), dict(q=None, qo=None), dict(heads=(1 << 16) + 1), dict(q=512, qs=1152, qh=64), dict(q=512, os=128, oh=64, dtype=1),
                dict(eps=math.nan), dict(mscale=math.inf), dict(ws=None), dict(nbytes=128)):
        assert latent_append(lib, **bad) == BAD, bad


def tree(lib, S=None, bits=16, n=4, max_new=4, q=256, par=256, starts=256, mod=None, out=256, ws=256, nbytes=1 << 40):
    L = kvq.make_layout(8, 2, bits)
    return lib.kv_tree_attn(by(L), by(pool(bits)), by(S or seqs()), q, par, starts, n, max_new, None if mod is None else by(mod), out, None, ws,
                            nbytes, None)


def test_tree_refusals(lib):
    assert tree(lib, n=0, max_new=0) == 0 and tree(lib, S=seqs(batch=0)) == 0
    for bad in (dict(max_new=257), dict(bits=4), dict(bits=_abi.BITS_E4M3), dict(mod=_abi.AttnModStruct(0, 0, 0, 0, None, 256, None)),
                dict(S=seqs(max_blocks=1 << 27, max_len=(1 << 30) + 1))):
        assert tree(lib, **bad) == UNSUP, bad
    for bad in (dict(par=None), dict(starts=None), dict(q=None), dict(out=None), dict(q=264), dict(out=8), dict(n=-1), dict(max_new=-1), dict(max_new=0),
                dict(ws=None), dict(nbytes=255), dict(mod=_abi.AttnModStruct(-1.0, 0, 0, 0, None, None, None)),
                dict(mod=_abi.AttnModStruct(0, math.nan, 0, 0, None, None, None)), dict(mod=_abi.AttnModStruct(0, 0, -1, 0, None, None, None))):
        assert tree(lib, **bad) == BAD, bad
    L = kvq.make_layout(8, 2, 16)
    assert lib.kv_tree_attn_ws(by(L), by(seqs()), 4, 257) == 0
    assert lib.kv_tree_attn_ws(by(L), by(seqs()), 4, 4) >= 256


def attn(lib, C=None, S=None, heads=16, q=256, par=None, starts=256, n=4, max_new=4, scale=0.0, out=256, ws=256, nbytes=1 << 40):
    return lib.kv_latent_attn(by(C or latent()), by(S or seqs()), heads, q, par, starts, n, max_new, scale, out, None, ws, nbytes, None)


def test_latent_attn_refusals(lib):
    assert attn(lib, n=0, max_new=0) == 0 and attn(lib, S=seqs(batch=0)) == 0
    for bad in (dict(C=latent(dim=256)), dict(C=latent(blocks=1 << 27)), dict(par=256, max_new=257), dict(n=1 << 30, heads=2, max_new=1),
                dict(S=seqs(max_blocks=1 << 27, max_len=(1 << 30) + 1)),
                dict(S=seqs(batch=1 << 20, max_blocks=1 << 26, max_len=1 << 30), n=1 << 20, heads=128, max_new=1)):
        assert attn(lib, **bad) == UNSUP, bad
    for bad in (dict(C=latent(rows=None)), dict(heads=0), dict(heads=(1 << 16) + 1), dict(n=-1), dict(max_new=0), dict(max_new=-4), dict(scale=-1.0),
                dict(scale=math.nan), dict(scale=math.inf), dict(scale=3e38), dict(q=None), dict(out=None), dict(starts=None), dict(S=seqs(bt=None)),
                dict(q=264), dict(out=8), dict(ws=None), dict(ws=260), dict(nbytes=256), dict(S=seqs(max_len=65))):
        assert attn(lib, **bad) == BAD, bad
    assert attn(lib, par=None, max_new=300, n=0) == 0   # a chain may be longer than a tree
    ws = lambda **k: lib.kv_latent_attn_ws(by(k.get("S", seqs())), k.get("heads", 16), k.get("n", 4), k.get("max_new", 4))  # noqa: E731
    assert ws() > 256 and ws(heads=0) == 0 and ws(max_new=0) == 0 and ws(S=seqs(batch=-1)) == 0
    # enough for what the call asks, whatever the number of rows in it
    for heads, n, m in ((1, 1, 1), (16, 4, 2), (128, 9, 5), (5, 1000, 600)):
        need = ws(heads=heads, n=n, max_new=m, S=seqs(batch=3))
        assert attn(lib, heads=heads, n=n, max_new=m, S=seqs(batch=3), nbytes=need - 1) == BAD


def test_latent_attn_sizes_that_pass_32_bits(lib):
    """Products of batch, rows, heads and lengths that no 64-bit number holds are refused, and whatever the call refuses has no
    workspace size."""
    ws = lambda S, heads, n, max_new: lib.kv_latent_attn_ws(by(S), heads, n, max_new)  # noqa: E731
    most = (1 << 31) - 1
    far = dict(max_blocks=1 << 26, max_len=1 << 30)
    for S, heads, n, max_new in ((seqs(batch=1 << 30), 1 << 16, 4, most),       # 2^70 row groups
                                 (seqs(batch=1 << 27), 1 << 16, 4, 1 << 30),    # 2^66
                                 (seqs(batch=most, **far), 1 << 16, most, most),
                                 (seqs(batch=1 << 20, **far), 128, 1 << 20, 1), # 2^44 steps
                                 (seqs(), 2, 1 << 30, 1)):                      # 2^31 query rows
        assert attn(lib, S=S, heads=heads, n=n, max_new=max_new, out=None) == UNSUP, (S.batch, heads, n, max_new)
        assert ws(S, heads, n, max_new) == 0, (S.batch, heads, n, max_new)
    # a bound on the new tokens far above their number costs nothing but the choice of the kernel
    assert 256 < ws(seqs(), 128, 4, most) == ws(seqs(), 128, 4, 1 << 20)


def expanded(lib, batch=2, heads=4, q=256, kn=256, kns=1024, knh=256, kr=256, krs=576, v=512, vs=1024, vh=256, m=64, qs=256, ks=256, n=4, max_new=4,
             max_len=32, scale=0.0, out=256, ws=256, nbytes=1 << 40):
    return lib.kv_latent_expanded_attn(batch, heads, q, kn, kns, knh, kr, krs, v, vs, vh, m, qs, ks, n, max_new, max_len, scale, out, None, ws, nbytes,
                                       None)


def test_expanded_refusals(lib):
    assert expanded(lib, n=0, max_new=0) == 0 and expanded(lib, batch=0) == 0
    assert expanded(lib, max_len=(1 << 30) + 1) == UNSUP
    for bad in (dict(batch=-1), dict(heads=0), dict(n=-1), dict(max_new=0), dict(max_len=-1), dict(m=-1), dict(m=0), dict(m=1 << 31), dict(q=None),
                dict(kn=None), dict(kr=None), dict(v=None), dict(qs=None), dict(ks=None), dict(out=None), dict(q=8), dict(kn=264), dict(kr=264),
                dict(v=520), dict(out=8), dict(kns=1028), dict(knh=132), dict(krs=60), dict(vs=120), dict(vh=120), dict(knh=64), dict(kns=1 << 40),
                dict(scale=-0.5), dict(scale=math.inf), dict(ws=None), dict(nbytes=100)):
        assert expanded(lib, **bad) == BAD, bad
    assert lib.kv_latent_expanded_attn_ws(2, 4, 4, 4, 32) >= 256
    assert lib.kv_latent_expanded_attn_ws(2, 0, 4, 4, 32) == 0 and lib.kv_latent_expanded_attn_ws(-2, 4, 4, 4, 32) == 0


def test_what_is_refused_has_no_workspace_size(lib):
    """Trees and expanded runs of more than 2^31 - 1 groups of query rows over all heads."""
    most = (1 << 31) - 1
    S = seqs(batch=1 << 20)
    L = kvq.make_layout(1 << 15, 1 << 14, 16)
    rows = 1 << 30
    assert lib.kv_tree_attn(by(L), by(pool()), by(S), 256, 256, 256, rows, 256, None, 256, None, 256, 1 << 40, None) == UNSUP
    assert lib.kv_tree_attn_ws(by(L), by(S), rows, 256) == 0
    assert expanded(lib, batch=1 << 20, heads=1 << 16, n=most, max_new=most, max_len=1 << 30) == UNSUP
    assert lib.kv_latent_expanded_attn_ws(1 << 20, 1 << 16, most, most, 1 << 30) == 0
    # with nothing to do, nothing is refused
    assert lib.kv_tree_attn_ws(by(L), by(S), 0, 0) == 256 and lib.kv_latent_expanded_attn_ws(0, 1 << 16, most, most, 1 << 30) == 256


def test_refusals_say_why(lib):
    assert tree(lib, max_new=300) == UNSUP and "256" in _abi.last_error()
    assert attn(lib, C=latent(dim=448)) == UNSUP and "448" in _abi.last_error()
    assert append(lib, bits=4) == UNSUP and "bits 4" in _abi.last_error()


class On:
    """Stands for an int32 tensor on a GPU."""
    dtype, shape = torch.int32, (1, 4)

    def __init__(self, gpu):
        self.gpu = gpu

    def contiguous(self):
        return self

    def data_ptr(self):
        return 256

    def get_device(self):
        return self.gpu


def test_a_batch_is_on_a_gpu_only_when_both_of_its_tables_are():
    """The calls compare Batch.gpu with the current GPU: a block table elsewhere would be read through a foreign address."""
    assert kvq.Batch(On(0), On(0), 64).gpu == 0 and kvq.Batch(On(3), On(3), 64).gpu == 3
    for table, lens in ((0, 1), (1, 0), (-1, 0), (0, -1), (-1, -1)):
        assert kvq.Batch(On(table), On(lens), 64).gpu < 0, (table, lens)


@pytest.mark.parametrize("q", [torch.zeros(4), torch.zeros((4, 576)), torch.zeros(()), torch.zeros((2, 3, 4, 5))])
def test_queries_without_heads_are_refused_as_such(monkeypatch, q):
    """Not an unpacking or an index error from inside the binding."""
    monkeypatch.setattr(kvq, "_gpu", lambda: 0)
    x = torch.zeros((4, 8), dtype=torch.float16)
    with pytest.raises(kvq.KvqError) as e:
        kvq.kv_latent_attn(None, None, q, None, 1, None, None)
    assert e.value.code == BAD and "q:" in str(e.value)
    with pytest.raises(kvq.KvqError) as e:
        kvq.kv_latent_expanded_attn(q, x, x, x, x, x, 1, 1, None, None)
    assert e.value.code == BAD and "q:" in str(e.value)

    class Part:
        gpu = 0

    monkeypatch.setattr(kvq, "_strided", lambda x, shape, dtype, gpu, fn, name: (256, 64, 64)[:len(shape)])
    with pytest.raises(kvq.KvqError) as e:
        kvq.kv_latent_append(Part, Part, Part, None, x, x, Part, q=q, q_out=q)
    assert e.value.code == BAD and "q:" in str(e.value)
