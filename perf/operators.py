"""Cases of the operators that prepare, attend and move a KV cache's rows.

Four operators, each as a serving program calls it:

  rope   -- norms of the query and key heads and their rotary positions in one pass (kv_qk_norm_rope)
  decode -- attention of one new token over the fp16 pages, split over the length (kv_decode_attn)
  chunk  -- attention of a run of new tokens per sequence over the same pages (kv_chunk_attn)
  pages  -- copies of pages for forks and for compaction (kv_pages_copy)

Scores of decode and chunk may be capped by a tanh, carry a bias that falls with distance, and be masked by a window
with sinks, by documents and (chunk) by a bidirectional prefix.  Without `own`, run() is the plain form in elementary
torch operations; with it, the library's calls.
"""
import math
import random

import torch

own = False

D = 128          # head dimension
PAGE = 16        # tokens per page


# ------------------------------------------------------------------ cases

def _rope(name, **k):
    c = {"name": name, "op": "rope", "tokens": 1, "hq": 32, "hkv": 8, "dtype": "f16", "norm": False, "rot": 128,
         "interleaved": False, "scaling": "plain", "base": 10000.0, "factor": 1.0, "original": 8192, "first_pos": 0,
         "with_v": False}
    return {**c, **k}


def _attn(name, op, **k):
    c = {"name": name, "op": op, "batch": 1, "hq": 32, "hkv": 8, "len_lo": 1, "len_hi": 1, "cap": 0.0, "bias": False,
         "window": 0, "sink": 0, "docs": 0}
    if op == "chunk":
        c.update(new_lo=1, new_hi=1, prefix=0)
    return {**c, **k}


def _pages(name, **k):
    return {**{"name": name, "op": "pages", "hq": 32, "hkv": 8, "bits": 16, "group": 64, "pairs": 1, "pool": 4}, **k}


def listed():
    return [
        # one decode step of eight sequences near 32K: the smallest call, all latency
        _rope("rope_decode_8", tokens=8, first_pos=32000, base=500000.0, scaling="knees", factor=8.0),
        # a bf16 model with normed heads takes a long prompt in, positions stretched to 128K; v is cast on the way
        _rope("rope_prompt_32k", tokens=32768, dtype="bf16", norm=True, base=1000000.0, scaling="yarn", factor=4.0,
              original=32768, first_pos=98304, with_v=True),
        # an odd chunk of a model that rotates half of each head, interleaved pairs
        _rope("rope_chunk_part", tokens=4097, hq=40, hkv=40, rot=64, interleaved=True, first_pos=1),
        # the small single layer: one sequence of 4096 tokens
        _attn("decode_4k", "decode", hq=8, hkv=2, len_lo=4096, len_hi=4096),
        # a serving batch of sixteen ragged sequences, one kv head per query head, scores falling with distance
        _attn("decode_batch16", "decode", batch=16, hq=32, hkv=32, len_lo=4096, len_hi=32767, bias=True),
        # one sequence of 128K with capped scores
        _attn("decode_128k", "decode", len_lo=131072, len_hi=131072, cap=50.0),
        # eight sequences near 32K each check five drafted tokens
        _attn("chunk_drafts", "chunk", batch=8, len_lo=30011, len_hi=32768, new_lo=5, new_hi=5),
        # ragged prompts packed from short documents, capped scores
        _attn("chunk_documents", "chunk", batch=5, hq=8, hkv=2, len_lo=333, len_hi=4001, new_lo=333, new_hi=4001,
              cap=30.0, docs=3),
        # a chunk of 2048 prompt tokens behind 30720 cached ones, 4096-token window with four sinks
        _attn("chunk_window", "chunk", len_lo=32768, len_hi=32768, new_lo=2048, new_hi=2048, window=4096, sink=4),
        # a whole prompt of 16384 tokens, causal
        _attn("chunk_prompt_16k", "chunk", len_lo=16384, len_hi=16384, new_lo=16384, new_hi=16384),
        # sixteen forks: the last page of each sequence is copied before the branches append to it
        _pages("pages_fork_16", pairs=16, pool=4096),
        # an INT4 pool is compacted: every high page moves down
        _pages("pages_compact_int4", pairs=20001, pool=50000, hkv=32, bits=4, group=32),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "decode", "chunk", "pages"])
    hq, hkv = rng.choice([(8, 2), (32, 8), (32, 32), (40, 40), (8, 1), (16, 8)])
    if op == "rope":
        norm = rng.random() < 0.5
        scaling = rng.choice(["plain", "linear", "ntk", "yarn", "knees"])
        c = _rope("", tokens=_log(rng, 1, 20000), hq=hq, hkv=hkv, dtype=rng.choice(["f16", "bf16"]), norm=norm,
                  rot=rng.choice([32, 64, 96, 128]), interleaved=rng.random() < 0.5, scaling=scaling,
                  base=rng.choice([10000.0, 500000.0, 1000000.0]),
                  factor=1.0 if scaling == "plain" else rng.choice([2.0, 4.0, 8.0]), first_pos=_log(rng, 1, 200000),
                  with_v=rng.random() < 0.5)
    elif op == "pages":
        bits = rng.choice([1, 4, 16])
        n = _log(rng, 1, 10000)
        c = _pages("", hq=hq, hkv=hkv, bits=bits, group=rng.choice([32, 64, 128]), pairs=n, pool=2 * n + rng.randrange(64))
    else:
        batch = _log(rng, 1, 24)
        hi = _log(rng, 1, 100000 if op == "decode" else 24000)
        c = _attn("", op, batch=batch, hq=hq, hkv=hkv, len_lo=rng.randint(1, hi), len_hi=hi,
                  cap=rng.choice([0.0, 0.0, 20.0, 50.0]), bias=rng.random() < 0.3, docs=rng.choice([0, 0, 0, 2, 7]))
        if rng.random() < 0.3:
            c.update(window=_log(rng, 1, 8192), sink=rng.choice([0, 4, 17]))
        if op == "chunk":
            new = hi if rng.random() < 0.4 else _log(rng, 1, hi)
            c.update(new_lo=min(c["len_lo"], rng.randint(1, new)), new_hi=new)
            if rng.random() < 0.25:
                c["prefix"] = _log(rng, 1, hi)
        # no dearer than the largest listed cases: fewer sequences until it fits
        top = 32 * 16384 * 16384 if op == "chunk" else 16 * 32767 * 32
        while c["batch"] > 1 and c["batch"] * c["hq"] * hi * c.get("new_hi", 1) > top:
            c["batch"] -= 1
        while c["batch"] * c["hq"] * c["len_hi"] * c.get("new_hi", 1) > top:
            c["len_hi"] = c["len_hi"] * 2 // 3
            c["len_lo"] = min(c["len_lo"], c["len_hi"])
            if op == "chunk":
                c["new_hi"] = min(c["new_hi"], c["len_hi"])
                c["new_lo"] = min(c["new_lo"], c["new_hi"], c["len_lo"])
    del c["name"]
    return c


def _spread(lo, hi, n):
    """n whole numbers from lo to hi, the longest first, odd ones among them."""
    return [hi - (hi - lo) * b // max(n - 1, 1) for b in range(n)]


def _lens(c):
    lens = _spread(c["len_lo"], c["len_hi"], c["batch"])
    if c["op"] == "decode":
        return lens, [1] * c["batch"]
    return lens, [min(n, t) for n, t in zip(_spread(c["new_lo"], c["new_hi"], c["batch"]), lens)]


# ------------------------------------------------------------------ inputs

def _randn(shape, g, dtype=torch.float16):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _freqs(c):
    """Radians per position of each rotated pair, and the factor on the rotated values (64 bits)."""
    r, base = c["rot"], c["base"]
    if c["scaling"] == "ntk":
        base = base * c["factor"] ** (r / (r - 2))
    f = base ** (-2.0 * torch.arange(r // 2, dtype=torch.float64) / r)
    m = 1.0
    if c["scaling"] == "linear":
        f = f / c["factor"]
    elif c["scaling"] == "yarn":
        # pairs that turn over 32 times within the original length stay, those under once are stretched
        edge = [r * math.log(c["original"] / (b * 2 * math.pi)) / (2 * math.log(base)) for b in (32.0, 1.0)]
        lo, hi = max(math.floor(edge[0]), 0), min(math.ceil(edge[1]), r - 1)
        ramp = ((torch.arange(r // 2, dtype=torch.float64) - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        f = f / c["factor"] * ramp + f * (1 - ramp)
        m = 0.1 * math.log(c["factor"]) + 1.0
    elif c["scaling"] == "knees":
        # full turns within the original length: over 4 stay, under 1 are stretched, a line between
        s = ((c["original"] * f / (2 * math.pi) - 1.0) / (4.0 - 1.0)).clamp(0, 1)
        f = f * s + f / c["factor"] * (1 - s)
    return f, m


def prepare(case, seed):
    c = {"name": "", **case}
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    h = random.Random(seed)
    if own:
        from compressed_kv_cache_quant_gb300 import kvq
    s = {"case": c}
    if c["op"] == "rope":
        n, hq, hkv = c["tokens"], c["hq"], c["hkv"]
        dt = torch.float16 if c["dtype"] == "f16" else torch.bfloat16
        # the rows of one projection: q, k and v of a token side by side
        rows = _randn((n, (hq + 2 * hkv) * D), g, dt)
        s.update(q=rows[:, :hq * D].view(n, hq, D), k=rows[:, hq * D:(hq + hkv) * D].view(n, hkv, D),
                 v=rows[:, (hq + hkv) * D:].view(n, hkv, D) if c["with_v"] else None)
        s["pos"] = c["first_pos"] + torch.arange(n, device="cuda", dtype=torch.int32)
        s["wq"] = torch.rand(D, generator=g, device="cuda") + 0.5 if c["norm"] else None
        s["wk"] = torch.rand(D, generator=g, device="cuda") + 0.5 if c["norm"] else None
        f, m = _freqs(c)
        s["freqs"], s["mscale"] = f.cuda(), m
        if own:
            s["layout"] = kvq.make_layout(hq, hkv, 16)
            low, high = (32.0, 1.0) if c["scaling"] == "yarn" else (1.0, 4.0)
            s["rope"] = kvq.RopeTable(c["rot"], c["base"], interleaved=c["interleaved"], scaling=c["scaling"],
                                      factor=c["factor"], original_len=c["original"], low=low, high=high)
            s["q_out"] = torch.empty((n, hq, D), dtype=torch.float16, device="cuda")
            s["k_out"] = torch.empty((n, hkv, D), dtype=torch.float16, device="cuda")
            s["v_out"] = torch.empty((n, hkv, D), dtype=torch.float16, device="cuda") if c["with_v"] else None
        return s
    if c["op"] == "pages":
        ids = torch.randperm(c["pool"], generator=g, device="cuda").to(torch.int32)
        s["pairs"] = ids[:2 * c["pairs"]].view(c["pairs"], 2).contiguous()
        if own:
            s["cache"] = kvq.LayerCache(c["hq"], c["hkv"], c["bits"], c["pool"], 1, v_group_dims=c["group"])
            s["ws"] = kvq.Workspace(kvq.kv_pages_copy_ws())
        p, hkv = c["pool"], c["hkv"]
        if c["bits"] == 16:
            s["arrays"] = {"k16": _randn((p, hkv, PAGE, D), g), "v16": _randn((p, hkv, PAGE, D), g)}
        else:
            r = D * c["bits"] // 8
            byte = lambda: torch.randint(0, 256, (p, hkv, PAGE, r), generator=g, device="cuda", dtype=torch.uint8)  # noqa: E731
            s["arrays"] = {"k_codes": byte(), "v_codes": byte(), "k_sz": _randn((p, hkv, D, 2), g),
                           "v_sz": _randn((p, hkv, PAGE, D // c["group"], 2), g)}
        if own:  # the layer's own arrays hold them
            for name in s["arrays"]:
                s["arrays"][name] = getattr(s["cache"], name).copy_(s["arrays"][name])
        return s
    # attention over pages in shuffled order, as a server's allocator leaves them
    lens, news = _lens(c)
    batch, hq, hkv = c["batch"], c["hq"], c["hkv"]
    blocks = [-(-t // PAGE) for t in lens]
    total = sum(blocks) + 3
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    bt = torch.full((batch, max(blocks)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b in range(batch):
        bt[b, :blocks[b]] = order[at:at + blocks[b]]
        at += blocks[b]
    if own:
        s["cache"] = kvq.LayerCache(hq, hkv, 16, total, batch)
        s["k16"], s["v16"] = s["cache"].k16, s["cache"].v16
    else:
        s["k16"] = torch.empty((total, hkv, PAGE, D), dtype=torch.float16, device="cuda")
        s["v16"] = torch.empty((total, hkv, PAGE, D), dtype=torch.float16, device="cuda")
    s["k16"].copy_(_randn((total, hkv, PAGE, D), g))
    s["v16"].copy_(_randn((total, hkv, PAGE, D), g))
    for head in range(hkv):  # a few key channels are large, as in real models
        s["k16"][:, head, :, h.sample(range(D), 4)] *= 10
    rows = sum(news)
    s["bt"], s["lens"] = bt, torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["q"] = _randn((rows, hq, D), g)
    s["starts"] = torch.tensor([sum(news[:b]) for b in range(batch + 1)], dtype=torch.int32, device="cuda")
    s["max_new"], s["max_len"] = max(news), max(lens)
    s["slopes"] = 2.0 ** (-8.0 * (torch.arange(hq, device="cuda") + 1) / hq) if c["bias"] else None
    s["prefix"] = None
    if c.get("prefix"):
        s["prefix"] = torch.tensor([min(c["prefix"] + b, t) for b, t in enumerate(lens)], dtype=torch.int32, device="cuda")
    s["doc"] = None
    if c["docs"]:  # documents end at seeded places of each sequence; a query's own begins at the last of them
        starts = []
        for t, n in zip(lens, news):
            cuts = sorted(h.randrange(t) for _ in range(c["docs"]))
            starts += [max([0] + [x for x in cuts if x <= i]) for i in range(t - n, t)]
        s["doc"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
    s["lse"] = torch.empty((rows, hq), device="cuda")
    if own:
        s["seqs"] = kvq.Batch(bt, s["lens"], max(lens))
        s["mod"] = kvq.AttnMod(softcap=c["cap"], window=c["window"], n_sink=c["sink"], slopes=s["slopes"],
                               prefix_len=s["prefix"], doc_start=s["doc"])
        if c["op"] == "decode":
            s["out"] = torch.empty((rows, hq, D), device="cuda")
            s["ws"] = kvq.Workspace(kvq.kv_decode_attn_ws(s["cache"], s["seqs"]))
        else:
            s["out"] = torch.empty((rows, hq, D), dtype=torch.float16, device="cuda")
            s["ws"] = kvq.Workspace(kvq.kv_chunk_attn_ws(s["cache"], s["seqs"], rows, s["max_new"]))
    return s


# ------------------------------------------------------------------ one pass

def _plain_rope(s):
    c = s["case"]
    a = s["pos"].double()[:, None] * s["freqs"]
    cos, sin = (torch.cos(a) * s["mscale"]).float()[:, None], (torch.sin(a) * s["mscale"]).float()[:, None]
    r = c["rot"]

    def turn(x, w):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w
        y = x.clone()
        if c["interleaved"]:
            u, v = x[..., 0:r:2], x[..., 1:r:2]
            y[..., 0:r:2], y[..., 1:r:2] = u * cos - v * sin, v * cos + u * sin
        else:
            u, v = x[..., :r // 2], x[..., r // 2:r]
            y[..., :r // 2], y[..., r // 2:r] = u * cos - v * sin, v * cos + u * sin
        return y.half()

    out = {"q": turn(s["q"], s["wq"]), "k": turn(s["k"], s["wk"])}
    if s["v"] is not None:
        out["v"] = s["v"].half()
    return out


def _plain_attention(s):
    c = s["case"]
    batch, hq, hkv = c["batch"], c["hq"], c["hkv"]
    n, t = s["max_new"], s["bt"].shape[1] * PAGE
    lens, starts = s["lens"].long(), s["starts"].long()
    news = starts[1:] - starts[:-1]
    rows = s["q"].shape[0]
    # new token i of sequence b is row starts[b] + i, at position lens[b] - news[b] + i; short ones are padded
    i = torch.arange(n, device="cuda")
    row = (starts[:-1, None] + i).clamp(max=rows - 1)
    pos = (lens - news)[:, None] + i
    page = s["bt"].clamp(min=0).long()
    k = s["k16"][page].transpose(2, 3).reshape(batch, t, hkv, D).permute(0, 2, 3, 1).float()
    q = s["q"][row].float().view(batch, n, hkv, hq // hkv, D).permute(0, 2, 3, 1, 4).reshape(batch, hkv, -1, D)
    x = torch.matmul(q, k).view(batch, hkv, hq // hkv, n, t)
    del k
    x *= 1.0 / math.sqrt(D)
    if c["cap"]:
        x = x.div_(c["cap"]).tanh_().mul_(c["cap"])
    j = torch.arange(t, device="cuda")
    if s["slopes"] is not None:
        far = (pos[:, :, None] - j).abs().float()
        x -= s["slopes"].view(1, hkv, -1, 1, 1) * far[:, None, None]
    hi = (pos + 1).clamp(max=t)
    if s["prefix"] is not None:
        hi = torch.maximum(hi, s["prefix"].long()[:, None])
    lo = s["doc"].long()[row] if s["doc"] is not None else torch.zeros_like(pos)
    seen = (j >= lo[..., None]) & (j < torch.minimum(hi, lens[:, None])[..., None])
    if c["window"]:
        seen &= (j > (pos - c["window"])[..., None]) | (j < (lo + c["sink"])[..., None])
    x.masked_fill_(~seen[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    x = x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    v = s["v16"][page].transpose(2, 3).reshape(batch, t, hkv, D).permute(0, 2, 1, 3).float()
    y = torch.matmul(x.view(batch, hkv, -1, t), v).view(batch, hkv, -1, n, D)
    y = y / torch.where(total > 0, total, torch.ones_like(total))
    b = torch.repeat_interleave(torch.arange(batch, device="cuda"), news, output_size=rows)
    at = torch.arange(rows, device="cuda") - starts[b]
    y = y.reshape(batch, hq, n, D)[b, :, at]
    lse = (top + total.log()).reshape(batch, hq, n)[b, :, at]
    return {"out": y if c["op"] == "decode" else y.half(), "lse": lse}


def run(s):
    c = s["case"]
    if own:
        from compressed_kv_cache_quant_gb300 import kvq
        if c["op"] == "rope":
            kvq.kv_qk_norm_rope(s["layout"], s["rope"], s["pos"], s["q"], s["k"], s["q_out"], s["k_out"],
                                q_weight=s["wq"], k_weight=s["wk"], eps=1e-6, v=s["v"], v_out=s["v_out"])
            out = {"q": s["q_out"], "k": s["k_out"]}
            if s["v"] is not None:
                out["v"] = s["v_out"]
            return out
        if c["op"] == "pages":
            kvq.kv_pages_copy(s["cache"], s["pairs"], s["ws"])
            return s["arrays"]
        if c["op"] == "decode":
            kvq.kv_decode_attn(s["cache"], s["seqs"], s["q"], s["out"], s["ws"], mod=s["mod"], lse=s["lse"])
        else:
            kvq.kv_chunk_attn(s["cache"], s["seqs"], s["q"], s["starts"], s["max_new"], s["out"], s["ws"],
                              mod=s["mod"], lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    if c["op"] == "rope":
        return _plain_rope(s)
    if c["op"] == "pages":
        src, dst = s["pairs"][:, 0].long(), s["pairs"][:, 1].long()
        return {name: a.index_copy_(0, dst, a[src]) for name, a in s["arrays"].items()}
    return _plain_attention(s)


# ------------------------------------------------------------------ work and values

def _page_bytes(c):
    if c["bits"] == 16:
        return c["hkv"] * PAGE * D * 4
    r = D * c["bits"] // 8
    return c["hkv"] * (2 * PAGE * r + 4 * D + 4 * PAGE * (D // c["group"]))


def work(case):
    c = {"name": "", **case}
    if c["op"] == "rope":
        vals = c["tokens"] * (c["hq"] + (2 if c["with_v"] else 1) * c["hkv"]) * D
        return {"bytes": 4.0 * vals + 4 * c["tokens"], "flops": 10.0 * vals}
    if c["op"] == "pages":
        return {"bytes": 2.0 * c["pairs"] * _page_bytes(c) + 8 * c["pairs"], "flops": 0.0}
    lens, news = _lens(c)
    pairs, read = 0.0, 0
    for b, (t, n) in enumerate(zip(lens, news)):
        pre = min(c.get("prefix", 0) + b, t) if c.get("prefix") else 0
        first = t - n
        # documents end at seeded places: about half of what a causal row sees stays on average with one cut
        part = 1.0 if not c["docs"] else 2.0 / (c["docs"] + 2)
        if c["window"]:
            seen = sum(min(max(i + 1, pre), max(i + 1, pre) - i - 1 + c["window"] + c["sink"]) for i in range(first, t))
            rows = min(t, n + c["window"] + c["sink"])
        else:
            seen = sum(max(i + 1, pre) for i in range(first, t)) if pre else (first + 1 + t) * n / 2.0
            rows = t
        pairs += seen * part
        read += rows if n > 1 else max(1, int(rows * part))
    rows = sum(news)
    out = 4 if c["op"] == "decode" else 2
    return {"bytes": float(read * c["hkv"] * D * 4 + rows * c["hq"] * (D * (2 + out) + 4)),
            "flops": 4.0 * D * c["hq"] * pairs}


def exact(case, seed):
    """The operators from their definitions in 64 bits, one sequence and one kv head at a time."""
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    c = s["case"]
    if c["op"] == "pages":
        moved = {}
        for name, a in s["arrays"].items():
            new = a.clone()
            new[s["pairs"][:, 1].long()] = a[s["pairs"][:, 0].long()]
            moved[name] = new
        return moved
    if c["op"] == "rope":
        r = c["rot"]
        turn = torch.polar(torch.full((c["tokens"], r // 2), float(s["mscale"]), dtype=torch.float64, device="cuda"),
                           s["pos"].double()[:, None] * s["freqs"])[:, None]
        out = {}
        for name, w in (("q", s["wq"]), ("k", s["wk"])):
            x = s[name].double()
            if w is not None:
                x = w.double() * x / ((x ** 2).sum(-1, keepdim=True) / D + 1e-6).sqrt()
            z = x[..., :r]
            z = z.unflatten(-1, (r // 2, 2)) if c["interleaved"] else z.unflatten(-1, (2, r // 2)).transpose(-1, -2)
            z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * turn)
            z = z if c["interleaved"] else z.transpose(-1, -2)
            out[name] = torch.cat([z.flatten(-2), x[..., r:]], -1)
        if s["v"] is not None:
            out["v"] = s["v"].double()
        return out
    lens, news = _lens(c)
    gq = c["hq"] // c["hkv"]
    rows = sum(news)
    out = torch.zeros((rows, c["hq"], D), dtype=torch.float64, device="cuda")
    lse = torch.full((rows, c["hq"]), -math.inf, dtype=torch.float64, device="cuda")
    first = 0
    for b, (t, n) in enumerate(zip(lens, news)):
        pages = s["bt"][b, :-(-t // PAGE)].long()
        i = torch.arange(t - n, t, device="cuda")[:, None]
        j = torch.arange(t, device="cuda")[None]
        doc = s["doc"][first:first + n].long()[:, None] if s["doc"] is not None else torch.zeros_like(i)
        seen = (j <= i) | (j < (int(s["prefix"][b]) if s["prefix"] is not None else 0))
        seen = seen & (j >= doc)
        if c["window"]:
            seen = seen & ((i - j < c["window"]) | (j - doc < c["sink"]))
        for g in range(c["hkv"]):
            k = s["k16"][pages, g].reshape(-1, D)[:t].double()
            v = s["v16"][pages, g].reshape(-1, D)[:t].double()
            for h in range(g * gq, (g + 1) * gq):
                x = s["q"][first:first + n, h].double() @ k.T / math.sqrt(D)
                if c["cap"]:
                    x = c["cap"] * torch.tanh(x / c["cap"])
                if s["slopes"] is not None:
                    x = x - float(s["slopes"][h]) * (i - j).abs()
                x = x.masked_fill(~seen, -math.inf)
                z = torch.logsumexp(x, -1)
                p = torch.exp(x - torch.where(torch.isinf(z), torch.zeros_like(z), z)[:, None])
                out[first:first + n, h] = p @ v
                lse[first:first + n, h] = z
        first += n
    return {"out": out, "lse": lse}
