"""GPU parity in the forms that sizes choose.  kv_decode_attn in each way to join a row's parts, with every score form: a second
launch (many rows), the part that arrives last (few rows of long sequences), a cluster (short contexts); kv_chunk_attn over
many sequences, whole and split; kv_qk_norm_rope with several tokens per CTA.  Each test asserts that its sizes take the
form it is for."""
import math

import numpy as np
import pytest
import torch

import new_token_ref as R
from compressed_kv_cache_quant_gb300 import kvq
from gpu_helpers import require_gpu
from test_gpu_new_tokens import Case, D, rnd

pytestmark = pytest.mark.gpu
TICKETS = 56   # most (sequence, kv head) rows that the last part joins
FORMS = ["plain", "cap", "bias", "cap_bias_scale", "wide_window", "docs", "prefix"]


def case(hq, hkv, lens, form, seed):
    """A Case whose windows and documents leave most of a long sequence to see, so that its parts have to be joined."""
    c = Case(hq, hkv, lens, [1] * len(lens), form if form not in ("wide_window", "docs") else "plain", seed)
    if form == "wide_window":
        c.spec.update(window=max(lens) * 2 // 3, n_sink=40)
    if form == "docs":
        g = np.random.default_rng(seed)
        c.doc = np.array([g.integers(0, T // 4 + 1) if b % 5 else T for b, T in enumerate(lens)], dtype=np.int32)
        c.doc[0] = lens[0] // 7
    if form in ("wide_window", "docs"):
        c.mod = kvq.AttnMod(doc_start=None if c.doc is None else torch.tensor(c.doc).cuda(), **c.spec)
    return c


def parts(c):
    """Parts that the workspace has room for: 128 floats of output, a maximum and a sum per part and query head."""
    rows = len(c.lens) * c.hq
    return round((kvq.kv_decode_attn_ws(c.cache, c.batch) - 256) / (rows * (128 * 4 + 8)))


def run(c):
    out, lse, wk = c.decode()
    c.check(out, lse, False)
    again, lse2, _ = c.decode(wk)      # the workspace was left as it was found; parts join in their order
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    assert not bool(wk.t.any())


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("hq,hkv", [(20, 5), (6, 6)])
def test_many_rows_joined_by_a_second_launch(hq, hkv, form):
    require_gpu()
    c = case(hq, hkv, [3001 - 140 * b for b in range(20)] + [0, 1], form, 200)
    assert len(c.lens) * hkv > TICKETS and parts(c) > 1
    run(c)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("hq,hkv,lens", [(8, 2, [9001, 7000, 33]), (5, 5, [6500, 0, 6777]), (8, 1, [12345, 17])])
def test_few_rows_joined_by_the_last_part(hq, hkv, lens, form):
    require_gpu()
    c = case(hq, hkv, lens, form, 201)
    rows, pages = len(lens) * hkv, math.ceil(max(lens) / 16)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert rows <= TICKETS and parts(c) > 1 and rows * pages <= 16 * 12 * sms
    run(c)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("hq,hkv,lens", [(8, 2, [4000, 300]), (6, 3, [2500, 0, 2501, 1])])
def test_short_contexts_joined_within_a_cluster(hq, hkv, lens, form):
    require_gpu()
    c = case(hq, hkv, lens, form, 202)
    assert parts(c) == 0 and max(lens) > 12 * 16   # no room for parts, more pages than one CTA's warps
    run(c)


@pytest.mark.parametrize("form", ["plain", "cap_bias_scale", "docs_window_sink"])
@pytest.mark.parametrize("hq,hkv,longest,most", [(4, 1, 1600, 3), (8, 2, 260, 150)])
def test_chunks_of_more_sequences_than_a_warp_has_lanes(hq, hkv, longest, most, form):
    """A CTA finds its sequence 32 at a time: 75 sequences, some of them empty or without a new token, split over the cache
    (longest 1600, few CTAs) and whole (many)."""
    require_gpu()
    g = np.random.default_rng(7)
    lens = [int(x) for x in g.integers(0, longest, 75)]
    lens[40] = longest
    news = [min(T, int(g.integers(0, most + 1))) for T in lens]
    news[40] = most
    c = Case(hq, hkv, lens, news, form, 203)
    rows = sum(news)
    split = kvq.kv_chunk_attn_ws(c.cache, c.batch, rows + 2, most) > 256
    assert split == (longest == 1600)
    out, lse, wk = c.chunk()
    c.check(out, lse, True, set(g.integers(0, rows, 40).tolist()) | {0, rows - 1})
    again, lse2, _ = c.chunk(wk)
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    assert not bool(wk.t.any())


@pytest.mark.parametrize("inter,rot", [(False, 128), (True, 64), (False, 96)])
def test_norm_rope_with_several_tokens_a_cta(inter, rot):
    """5003 tokens: more than 32 per SM, so that a CTA takes eight; the last one fewer."""
    require_gpu()
    n, hq, hkv = 5003, 5, 2
    tab = kvq.RopeTable(rot, 10000.0, interleaved=inter)
    f, m = R.frequencies(rot, 10000.0)
    q, k = rnd((n, hq, D), 1, dtype=torch.bfloat16).cuda(), rnd((n, hkv, D), 2, dtype=torch.bfloat16).cuda()
    w = (rnd((D,), 3, dtype=torch.float32).abs() + 0.5).cuda()
    pos = torch.arange(n, dtype=torch.int32, device="cuda") * 7 - 900
    qo = torch.full((n + 1, hq, D), -7.0, dtype=torch.float16, device="cuda")
    ko = torch.full((n + 1, hkv, D), -7.0, dtype=torch.float16, device="cuda")
    kvq.kv_qk_norm_rope(kvq.make_layout(hq, hkv, 16), tab, pos, q, k, qo[:n], ko[:n], w, None, 1e-6)
    for x, y, wt in ((q, qo, R.as64(w)), (k, ko, None)):
        z, bound = R.norm_rope(R.as64(x), pos.cpu().numpy().astype(np.float64), f, m, rot, inter, wt)
        assert np.all(np.abs(R.as64(y[:n]) - z) <= bound) and bool((y[n] == -7).all())
