"""GPU tests of the new tokens' attention where its arithmetic is tight: weights far below a dominant token's,
scores beyond 2^24, NaN in a query or a key, and rows that no query sees."""
import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import new_token_ref as R
from compressed_kv_cache_quant_gb300 import kvq
from gpu_helpers import require_gpu, ws
from test_gpu_new_tokens import Case

pytestmark = pytest.mark.gpu
D = 128


def store(c, K, V):
    """Puts K, V [T][H_kv][d] (fp16) into sequence 0 .. of Case c, the same rows for every sequence (cut to its length)."""
    for b, T in enumerate(c.lens):
        c.KV[b] = (K[:T].clone(), V[:T].clone())
        if T:
            kvq.kv_quant_pack(c.cache, c.batch, b, 0, T, c.KV[b][0].cuda(), c.KV[b][1].cuda())


def dominated(c, every, low):
    """Scores of 8 at every `every`-th token, whose V is 0, and of 8 - low at the others, whose V is of one sign: the
    output is what the small weights add up to.  Products and sums of the scores are exact."""
    T, H = max(c.lens), c.hkv
    K = torch.zeros((T, H, D), dtype=torch.float16)
    K[..., 0] = 8.0 - low
    K[::every, :, 0] = 8.0
    V = torch.from_numpy(np.random.default_rng(5).uniform(500.0, 1000.0, (T, H, D))).half()
    V[::every] = 0
    store(c, K, V)
    c.q[..., 0] = 1.0
    c.spec["scale"] = 1.0
    c.mod = kvq.AttnMod(scale=1.0, softcap=c.spec.get("softcap", 0.0))


def check_dominated(c, out, lse, rows, half, floor, fp16):
    """A weight is kept to `half` of itself or, in units of the row's largest, to `floor` (2^-25, half the smallest fp16 step,
    over the scale of the weights); the rest of the bound is the 64-bit form's for the scores and sums."""
    row = 0
    for b, (T, n) in enumerate(zip(c.lens, c.news)):
        K, V = R.as64(c.KV[b][0]), R.as64(c.KV[b][1])
        for i in range(n):
            if row in rows:
                pos = T - n + i
                for h in range(c.hq):
                    k, v = K[:pos + 1, h // (c.hq // c.hkv)], V[:pos + 1, h // (c.hq // c.hkv)]
                    o, z, bo, bz = R.attend(R.as64(c.q[row, h]), k, v, np.ones(pos + 1, bool), pos, 1.0, c.spec.get("softcap", 0.0))
                    top = 8.0 if "softcap" not in c.spec else c.spec["softcap"] * math.tanh(8.0 / c.spec["softcap"])
                    bo = bo + half * o + floor * v.sum(0) / math.exp(z - top)
                    if fp16:
                        bo = bo + 2.0 ** -11 * (o + bo) + 2.0 ** -25
                    assert np.all(np.abs(R.as64(out[row, h]) - o) <= bo), (b, i, h, R.as64(out[row, h])[:2], o[:2], bo[:2])
                    assert abs(float(lse[row, h]) - z) <= bz
            row += 1


@pytest.mark.parametrize("mod", ["plain", "cap"])
@pytest.mark.parametrize("every,low", [(64, 16.25), (64, 17.0), (100000, 17.0), (100000, 17.5)])
@pytest.mark.parametrize("hq,hkv,lens,news", [(8, 2, [4096], [300]), (2, 2, [6011, 900], [5, 130]), (8, 1, [1500], [1500])])
def test_chunk_weights_far_below_the_largest(hq, hkv, lens, news, every, low, mod):
    """One fp16 rounding of a weight: 2^-11 of itself, and 2^-25 where the largest is 2^7."""
    require_gpu()
    c = Case(hq, hkv, lens, news, mod, 140, poison=False)
    dominated(c, every, low)
    out, lse, _ = c.chunk(extra=0)
    total = sum(news)
    rows = set(np.random.default_rng(6).integers(0, total, 10).tolist()) | {0, total - 1}
    check_dominated(c, out, lse, rows, 2.0 ** -11, 2.0 ** -32, True)


@pytest.mark.parametrize("sign", ["both", "negative"])
@pytest.mark.parametrize("hq,hkv,lens,news", [(8, 2, [700], [1]), (8, 2, [700, 333], [70, 333]), (2, 2, [5000], [3])])
def test_scores_beyond_fp32_whole_numbers(hq, hkv, lens, news, sign):
    """Finite keys and queries whose scores lie far beyond 2^24, where neighbouring fp32 values are more than a step of the
    exponent apart: the largest score takes all the weight."""
    require_gpu()
    c = Case(hq, hkv, lens, news, "plain", 142, poison=False)
    T = max(lens)
    if sign == "both":
        K = c_rnd((T, hkv, D), 1) * 20000
        c.q.copy_((c_rnd(c.q.shape, 2) * 20000).clamp(-60000, 60000))
    else:
        K = (c_rnd((T, hkv, D), 1) * 0.3 + 1) * 20000
        c.q.fill_(-20000.0)
    K = K.clamp(-60000, 60000).half()
    store(c, K, c_rnd((T, hkv, D), 3).half())
    runs = [(c.chunk(extra=0), True)] + ([(c.decode(), False)] if news == [1] else [])
    row = 0
    for b, (T, n) in enumerate(zip(lens, news)):
        K, V = R.as64(c.KV[b][0]), R.as64(c.KV[b][1])
        for i in range(n):
            for h in range(hq):
                q, g = R.as64(c.q[row, h]), h // (hq // hkv)
                k = K[:T - n + i + 1, g]
                s = k @ q / math.sqrt(D)
                eps = 130 * 2 * R.U / math.sqrt(D) * np.max(np.abs(k) @ np.abs(q))
                at = int(np.argmax(s))
                others = np.delete(s, at)
                if len(others) and s[at] - others.max() < 4 * eps:
                    continue   # too close to tell
                for (out, lse, _), half in runs:
                    assert bool((R.as64(out[row, h]) == V[at, g]).all()), (b, i, h)
                    assert abs(float(lse[row, h]) - s[at]) <= 2 * eps
            row += 1


def c_rnd(shape, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed))


@pytest.mark.parametrize("mod", ["cap", "cap_bias_scale"])
def test_rows_that_no_query_sees_leave_no_trace(mod):
    """Queries behind the last sequence and keys behind a sequence's last token may hold anything: not one bit of what the
    others give depends on them."""
    require_gpu()
    got = []
    for fill in (0.0, 60000.0):
        c = Case(8, 2, [777, 390], [9, 3], mod, 144, poison=False)
        for b, T in enumerate(c.lens):
            page = int(c.bt[b, T // 16])
            c.cache.k16[page, :, T % 16:] = fill
            c.cache.v16[page, :, T % 16:] = fill
        q = torch.cat([c.q, torch.full((30, 8, D), fill, dtype=torch.float16, device="cuda")])
        out = torch.zeros((42, 8, D), dtype=torch.float16, device="cuda")
        lse = torch.zeros((42, 8), device="cuda")
        wk = ws(kvq.kv_chunk_attn_ws(c.cache, c.batch, 42, 9))
        kvq.kv_chunk_attn(c.cache, c.batch, q, torch.tensor(c.starts).cuda(), 9, out, wk, mod=c.mod, lse=lse)
        kvq.kvq_check(wk)
        c.check(out, lse, True)
        got.append((out, lse))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


@pytest.mark.parametrize("mod", ["plain", "cap"])
@pytest.mark.parametrize("every,low", [(16, 8.0), (16, 16.25), (16, 17.0), (64, 17.5), (100000, 17.0)])
@pytest.mark.parametrize("hq,hkv,lens", [(8, 2, [2049]), (8, 2, [20011]), (16, 16, [3001, 700, 17] * 8)])
def test_decode_weights_far_below_the_largest(hq, hkv, lens, every, low, mod):
    """Two fp16 halves of a weight: 2^-22 of itself (each half rounds by 2^-11 of what it takes), and 2^-25 where the largest
    of its warp is 2^15."""
    require_gpu()
    c = Case(hq, hkv, lens, [1] * len(lens), mod, 141, poison=False)
    dominated(c, every, low)
    out, lse, _ = c.decode()
    check_dominated(c, out, lse, range(3), 2.0 ** -22, 2.0 ** -40, False)


@pytest.mark.parametrize("hq,hkv,lens", [(8, 2, [40, 700]), (8, 2, [20011]), (16, 16, [3001, 700, 17] * 8)])
@pytest.mark.parametrize("where", ["query", "key"])
def test_nan_in_what_a_query_sees(hq, hkv, lens, where):
    """A NaN in a query, or in every key that it sees, gives NaN in its rows and in no other's."""
    require_gpu()
    c = Case(hq, hkv, lens, [1] * len(lens), "plain", 143, poison=False)
    clean = [c.decode()[:2], c.chunk(extra=0)[:2]]
    GQ, last = hq // hkv, len(lens) - 1
    hit = torch.zeros((len(lens), hq), dtype=torch.bool, device="cuda")
    if where == "query":
        c.q[last, 1, 5] = math.nan
        hit[last, 1] = True
    else:
        for t in range(lens[last]):
            c.cache.k16[int(c.bt[last, t // 16]), 1, t % 16, 3] = math.nan
        hit[last, GQ:2 * GQ] = True
    for (out, lse), (want, wlse) in zip([c.decode()[:2], c.chunk(extra=0)[:2]], clean):
        assert bool(out[hit].isnan().all()) and bool(lse[hit].isnan().all())
        assert torch.equal(out[~hit], want[~hit]) and torch.equal(lse[~hit], wlse[~hit])


def test_first_calls_from_many_threads():
    """Threads whose first CUDA call is the library's, and whose calls come together, each on a stream and a workspace of its
    own, give what one thread gives."""
    require_gpu()
    prog = '''
import threading, torch
import new_token_ref
from compressed_kv_cache_quant_gb300 import kvq
from gpu_helpers import ws
from test_gpu_new_tokens import Case, D
c = Case(8, 2, [300, 90], [20, 7], "cap", 145)
starts = torch.tensor(c.starts).cuda()
need = kvq.kv_chunk_attn_ws(c.cache, c.batch, 27, 20)
own = [(torch.cuda.Stream(), ws(need), torch.empty((27, 8, D), dtype=torch.float16, device="cuda")) for _ in range(8)]
torch.cuda.synchronize()
ready, errors = threading.Barrier(8), []
def call(s, w, o):
    try:
        ready.wait()
        kvq.kv_chunk_attn(c.cache, c.batch, c.q, starts, 20, o, w, mod=c.mod, stream=s)
    except Exception as e:
        errors.append(e)
threads = [threading.Thread(target=call, args=x) for x in own]
for t in threads: t.start()
for t in threads: t.join()
torch.cuda.synchronize()
want = c.chunk(extra=0)[0]
assert not errors and all(torch.equal(o, want) for _, _, o in own), errors
print("as one")
'''
    here = os.path.dirname(os.path.abspath(__file__))
    env = dict(os.environ, PYTHONPATH=os.pathsep.join([here, os.path.dirname(here)]))
    got = subprocess.run([sys.executable, "-c", prog], env=env, capture_output=True, text=True, timeout=300)
    assert got.returncode == 0 and "as one" in got.stdout, got.stdout + got.stderr


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("n", [1, 37, 5000])
def test_v_alone_needs_no_positions(n, dt):
    """v is only cast: with a table that rotates, a call for v alone takes no positions."""
    require_gpu()
    v = (c_rnd((n, 3, D), 7) * 3).to(dt).cuda()
    out = torch.full((n + 1, 3, D), -7.0, dtype=torch.float16, device="cuda")
    for tab in (kvq.RopeTable(128), kvq.RopeTable(64, interleaved=True), kvq.RopeTable(0)):
        out[:n] = 0
        kvq.kv_qk_norm_rope(kvq.make_layout(6, 3, 16), tab, None, None, None, None, None, v=v, v_out=out[:n])
        assert torch.equal(out[:n], v.half()) and bool((out[n] == -7).all())


@pytest.mark.parametrize("most", [2 ** 31 - 1, 2 ** 31 - 100])
def test_largest_bound_on_the_new_tokens(most):
    """max_new is an upper bound: the largest there is gives what the exact one gives."""
    require_gpu()
    c = Case(8, 2, [300, 700, 90], [300, 150, 9], "plain", 146)
    want = c.chunk(extra=0)[0]
    out = torch.full_like(want, -7.0)
    wk = ws(kvq.kv_chunk_attn_ws(c.cache, c.batch, 459, most))
    kvq.kv_chunk_attn(c.cache, c.batch, c.q, torch.tensor(c.starts).cuda(), most, out, wk, mod=c.mod)
    kvq.kvq_check(wk)
    assert not bool((out == -7).all(-1).any())
    c.check(out, c.chunk(extra=0)[1], True)
