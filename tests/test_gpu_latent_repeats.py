"""The absorbed form's pairs of CTAs, many times over: weights that one CTA of a pair writes are read by products that the
other one issues, at every step, with anchors that move and tails that end inside a page."""
import numpy as np
import pytest
import torch

from compressed_kv_cache_quant_gb300 import kvq
from gpu_helpers import require_gpu, ws
from test_gpu_latent_forms import LAT, ROW, LatentLayer, agrees, expect, rnd, starts_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads,lens,news", [
    (128, [3001, 130, 700, 65], [1, 1, 1, 1]),           # parts of many steps and of few, joined
    (64, [129, 64, 1000, 383, 17], [5, 1, 2, 3, 4]),     # tails inside a page, a step, a pair's half
    (40, [50, 380, 128, 1], [1, 3, 2, 1]),               # groups of up to six steps, not cut
])
def test_pairs_repeat_themselves(heads, lens, news):
    """Sixty calls give the same bits, and those agree with the plain form; scores rise along the cache, so that anchors are
    set anew while products of the step before run."""
    require_gpu()
    L = LatentLayer(lens, seed=heads)
    for b, t in enumerate(lens):
        rows = L.rows[b].clone()
        rows[:, :4] = torch.linspace(0, 24, t).half()[:, None]
        L.rows[b] = rows
        for p in range(-(-t // 16)):
            part = rows[16 * p:16 * p + 16].cuda()
            L.cache.rows[L.bt[b, p], :len(part)] = part
    n = sum(news)
    q = rnd((n, heads, ROW), heads, 1).cuda()
    q[..., :4] = torch.linspace(0, 30, heads, dtype=torch.float16, device="cuda")[None, :, None]
    w = ws(kvq.kv_latent_attn_ws(L.batch, heads, n, max(news)))
    starts = starts_of(news)
    first = None
    for turn in range(60):
        out = torch.full((n, heads, LAT), -7.0, dtype=torch.float16, device="cuda")
        lse = torch.full((n, heads), -7.0, device="cuda")
        kvq.kv_latent_attn(L.cache, L.batch, q, starts, max(news), out, w, lse=lse)
        if first is None:
            first = out, lse
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1]), turn
    kvq.kvq_check(w)
    assert not bool(w.t.any())
    pick = sorted({0, 1, heads // 2, heads - 1})
    rows = set(np.cumsum(news).tolist()) - {n} | {0, n - 1}
    agrees(first[0][:, pick], first[1][:, pick], expect(q[:, pick], L.rows, lens, news, rows=rows))


def test_one_workspace_for_calls_of_every_kind():
    """Calls of other sizes, heads and kinds in turn, with parts and without, all in one workspace: what each gives alone."""
    require_gpu()
    cases = [(16, [5000, 77], [1, 1]), (128, [3000], [1]), (64, [60, 90], [2, 1]), (1, [20001], [1]), (40, [700, 1, 1500], [3, 1, 2]), (8, [100] * 40, [1] * 40)]
    calls = []
    for heads, lens, news in cases:
        L, n = LatentLayer(lens, seed=heads), sum(news)
        q, starts = rnd((n, heads, ROW), heads, 7).cuda(), starts_of(news)
        need = kvq.kv_latent_attn_ws(L.batch, heads, n, max(news))

        def call(w, L=L, q=q, starts=starts, n=n, heads=heads, news=news):
            out, lse = torch.empty((n, heads, LAT), dtype=torch.float16, device="cuda"), torch.empty((n, heads), device="cuda")
            kvq.kv_latent_attn(L.cache, L.batch, q, starts, max(news), out, w, lse=lse)
            return out, lse

        calls.append((need, call))
    alone = [call(ws(need)) for need, call in calls]
    w = ws(max(need for need, _ in calls))
    for order in (range(len(calls)), reversed(range(len(calls))), [0, 3, 1, 3, 4, 0, 5, 1, 2, 4]):
        got = [(i, calls[i][1](w)) for i in order]   # (no wait between them)
        for i, (out, lse) in got:
            assert torch.equal(out, alone[i][0]) and torch.equal(lse, alone[i][1]), i
    kvq.kvq_check(w)
    assert not bool(w.t.any())
