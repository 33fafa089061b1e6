"""Cases of the operators that write new tokens into a cache, check trees of drafts, and serve latent layers.

Five operators, each as a serving program calls it:

  append        -- new tokens' keys and values into the pages, normed and rotated on the way (kv_rope_append)
  tree          -- attention of a tree of drafted tokens over the fp16 pages (kv_tree_attn)
  latent_append -- the shared latent row of every new token into its page, normed and rotated (kv_latent_append)
  latent        -- absorbed attention over latent pages: one row per token is key and value (kv_latent_attn)
  expanded      -- attention of a run over keys and values expanded from the latent rows (kv_latent_expanded_attn)

Without `own`, run() is the plain form in elementary torch operations; with it, the library's calls.
"""
import math
import random

import torch

own = False

D = 128          # head dimension
PAGE = 16        # tokens per page
LAT, ROT = 512, 64           # a latent row: shared latent values, then rotated key values
ROW = LAT + ROT


# ------------------------------------------------------------------ cases

def _append(name, **k):
    c = {"name": name, "op": "append", "batch": 1, "len_lo": 16, "len_hi": 16, "new_lo": 1, "new_hi": 1, "hq": 32, "hkv": 8,
         "dtype": "f16", "cache": "f16", "norm": False, "rot": 128, "interleaved": False, "base": 500000.0}
    return {**c, **k}


def _tree(name, **k):
    c = {"name": name, "op": "tree", "batch": 1, "len_lo": 16, "len_hi": 16, "new_lo": 1, "new_hi": 1, "hq": 32, "hkv": 8,
         "cap": 0.0, "bias": False, "window": 0, "sink": 0}
    return {**c, **k}


def _latent_append(name, **k):
    c = {"name": name, "op": "latent_append", "batch": 1, "len_lo": 16, "len_hi": 16, "new_lo": 1, "new_hi": 1, "heads": 16,
         "dtype": "f16", "norm": True, "interleaved": True, "base": 10000.0}
    return {**c, **k}


def _latent(name, **k):
    c = {"name": name, "op": "latent", "batch": 1, "len_lo": 16, "len_hi": 16, "new_lo": 1, "new_hi": 1, "heads": 16,
         "tree": False}
    return {**c, **k}


def _expanded(name, **k):
    c = {"name": name, "op": "expanded", "batch": 1, "len_lo": 16, "len_hi": 16, "new_lo": 1, "new_hi": 1, "heads": 16}
    return {**c, **k}


def listed():
    return [
        # a decode step of sixteen sequences: one token each, all latency
        _append("append_decode_16", batch=16, len_lo=500, len_hi=4096),
        # two long prompts of a bf16 model with normed heads go into an FP8 cache
        _append("append_prompts_fp8", batch=2, len_lo=16001, len_hi=16384, new_lo=16001, new_hi=16384, dtype="bf16",
                cache="e4m3", norm=True),
        # an odd chunk behind cached tokens into a sparse layer, whose channel-major keys and channel maxima follow
        _append("append_chunk_scored", len_lo=8200, len_hi=8200, new_lo=4097, new_hi=4097, cache="scored", rot=64,
                interleaved=True),
        # one sequence of 4096 tokens checks a small tree, scores capped
        _tree("tree_25", len_lo=4121, len_hi=4121, new_lo=25, new_hi=25, hq=8, hkv=2, cap=30.0),
        # eight sequences near 32K each check 64 drafted tokens
        _tree("tree_64_batch8", batch=8, len_lo=30011, len_hi=32768, new_lo=64, new_hi=64),
        # a decode step of 64 sequences on a latent layer of 128 heads
        _latent_append("latent_append_64", batch=64, len_lo=100, len_hi=3000, heads=128),
        # a long prompt of a bf16 model, 16 heads
        _latent_append("latent_append_prompt", len_lo=16385, len_hi=16385, new_lo=16385, new_hi=16385, dtype="bf16"),
        # one short sequence, one token: latency
        _latent("latent_decode_1k", len_lo=1025, len_hi=1025),
        # a serving batch of ragged sequences, 16 heads (a model's heads spread over eight GPUs)
        _latent("latent_decode_batch32", batch=32, len_lo=4096, len_hi=32767),
        # eight sequences of 128 heads each check a chain of four drafted tokens behind the newest
        _latent("latent_drafts_128", batch=8, len_lo=12001, len_hi=16384, new_lo=5, new_hi=5, heads=128),
        # packed prompts of ragged lengths, the longer ones' first parts cached already
        _expanded("expanded_ragged", batch=5, len_lo=333, len_hi=4001, new_lo=333, new_hi=2049),
        # a whole prompt
        _expanded("expanded_prompt_16k", len_lo=16384, len_hi=16384, new_lo=16384, new_hi=16384),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "tree", "latent_append", "latent", "expanded"])
    batch = _log(rng, 1, 24)
    hi = _log(rng, 1, {"append": 16384, "tree": 40000, "latent_append": 16384, "latent": 40000, "expanded": 12000}[op])
    c = {"batch": batch, "len_lo": rng.randint(1, hi), "len_hi": hi}
    few = {"tree": 256, "latent": 16}.get(op, hi)
    new = min(hi, few) if rng.random() < 0.4 else _log(rng, 1, min(hi, few))
    c.update(new_lo=min(c["len_lo"], rng.randint(1, new)), new_hi=new)
    hq, hkv = rng.choice([(8, 2), (32, 8), (32, 32), (40, 40), (8, 1), (16, 8)])
    heads = rng.choice([1, 8, 12, 16, 20, 32, 64, 128])
    if op == "append":
        c = _append("", **c, hq=hq, hkv=hkv, dtype=rng.choice(["f16", "bf16"]), cache=rng.choice(["f16", "f16", "e4m3", "scored"]),
                    norm=rng.random() < 0.5, rot=rng.choice([32, 64, 96, 128]), interleaved=rng.random() < 0.5,
                    base=rng.choice([10000.0, 500000.0, 1000000.0]))
        top = 2 * 16384 * 48
        size = lambda: c["batch"] * c["len_hi"] * (c["hq"] + 2 * c["hkv"])  # noqa: E731
    elif op == "tree":
        c = _tree("", **c, hq=hq, hkv=hkv, cap=rng.choice([0.0, 0.0, 20.0, 50.0]), bias=rng.random() < 0.3)
        if rng.random() < 0.3:
            c.update(window=_log(rng, 1, 8192), sink=rng.choice([0, 4, 17]))
        top = 8 * 32768 * 32 * 64
        size = lambda: c["batch"] * c["len_hi"] * max(c["hq"] * c["new_hi"], 64 * c["hkv"])  # noqa: E731
    elif op == "latent_append":
        c = _latent_append("", **c, heads=heads, dtype=rng.choice(["f16", "bf16"]), norm=rng.random() < 0.8,
                           interleaved=rng.random() < 0.5, base=rng.choice([10000.0, 500000.0]))
        top = 16385 * (2 * 16 * ROT + 2 * ROW)
        size = lambda: c["batch"] * c["len_hi"] * (2 * c["heads"] * ROT + 2 * ROW)  # noqa: E731
    elif op == "latent":
        c = _latent("", **c, heads=heads, tree=rng.random() < 0.4)
        top = 8 * 16384 * 5 * 128
        size = lambda: c["batch"] * c["len_hi"] * max(c["new_hi"] * c["heads"], 64)  # noqa: E731
    else:
        c = _expanded("", **c, heads=min(heads, 32))
        top = 16384 * 16384 * 16
        size = lambda: c["batch"] * c["len_hi"] * max(c["new_hi"], 512) * c["heads"]  # noqa: E731
    # no dearer than the largest listed cases: fewer sequences until it fits, then shorter ones
    while c["batch"] > 1 and size() > top:
        c["batch"] -= 1
    while size() > top:
        c["len_hi"] = c["len_hi"] * 2 // 3
        c["len_lo"] = min(c["len_lo"], c["len_hi"])
        c["new_hi"] = min(c["new_hi"], c["len_hi"])
        c["new_lo"] = min(c["new_lo"], c["new_hi"], c["len_lo"])
    del c["name"]
    return c


def _spread(lo, hi, n):
    """n whole numbers from lo to hi, the longest first, odd ones among them."""
    return [hi - (hi - lo) * b // max(n - 1, 1) for b in range(n)]


def _lens(c):
    lens = _spread(c["len_lo"], c["len_hi"], c["batch"])
    return lens, [min(n, t) for n, t in zip(_spread(c["new_lo"], c["new_hi"], c["batch"]), lens)]


# ------------------------------------------------------------------ inputs

def _randn(shape, g, dtype=torch.float16):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _parents(h, n):
    """A drafting model's tree in the order of drafting: a node hangs from a late one, now and then from the last cached token."""
    return [-1 if i == 0 or h.random() < 0.05 else h.randrange(max(0, i - 8), i) for i in range(n)]


def prepare(case, seed):
    c = {"name": "", **case}
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    h = random.Random(seed)
    if own:
        from compressed_kv_cache_quant_gb300 import kvq
    lens, news = _lens(c)
    batch, rows = c["batch"], sum(news)
    s = {"case": c, "lens": _i32(lens), "max_new": max(news), "max_len": max(lens), "parents": None}
    s["starts"] = _i32([sum(news[:b]) for b in range(batch + 1)])
    dt = torch.bfloat16 if c.get("dtype") == "bf16" else torch.float16
    if c["op"] == "expanded":
        # one product expands the rows of all sequences: a head's key values, then its values
        total, nh = sum(lens), c["heads"]
        s["k_starts"] = _i32([sum(lens[:b]) for b in range(batch + 1)])
        s["kv"] = _randn((total, nh, 2 * D), g)
        s["lat"] = _randn((total, ROW), g)
        s["q"] = _randn((rows, nh, D + ROT), g)
        s["out"] = torch.empty((rows, nh, D), dtype=torch.float16, device="cuda")
        s["lse"] = torch.empty((rows, nh), device="cuda")
        if own:
            s["ws"] = kvq.Workspace(kvq.kv_latent_expanded_attn_ws(batch, nh, rows, s["max_new"], s["max_len"]))
        return s
    # pages in shuffled order, as a server's allocator leaves them
    blocks = [-(-t // PAGE) for t in lens]
    pool = sum(blocks) + 3
    order = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    bt = torch.full((batch, max(blocks)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b in range(batch):
        bt[b, :blocks[b]] = order[at:at + blocks[b]]
        at += blocks[b]
    s["bt"] = bt
    if own:
        s["seqs"] = kvq.Batch(bt, s["lens"], s["max_len"])
    if c["op"] in ("append", "latent_append"):
        rot = c["rot"] if c["op"] == "append" else ROT
        s["freqs"] = (c["base"] ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64) / rot)).cuda()
        if own:
            s["rope"] = kvq.RopeTable(rot, c["base"], interleaved=c["interleaved"])
            s["ws"] = kvq.Workspace(kvq.kv_rope_append_ws())
    if c["op"] == "append":
        hq, hkv = c["hq"], c["hkv"]
        # the rows of one projection: q, k and v of a token side by side
        x = _randn((rows, (hq + 2 * hkv) * D), g, dt)
        s.update(q=x[:, :hq * D].view(rows, hq, D), k=x[:, hq * D:(hq + hkv) * D].view(rows, hkv, D),
                 v=x[:, (hq + hkv) * D:].view(rows, hkv, D))
        s["wq"] = torch.rand(D, generator=g, device="cuda") + 0.5 if c["norm"] else None
        s["wk"] = torch.rand(D, generator=g, device="cuda") + 0.5 if c["norm"] else None
        s["q_out"] = torch.empty((rows, hq, D), dtype=torch.float16, device="cuda")
        fp8, cap = c["cache"] == "e4m3", (max(lens) + 7) // 8 * 8 if c["cache"] == "scored" else 0
        if own:
            s["cache"] = kvq.LayerCache(hq, hkv, kvq.BITS_E4M3 if fp8 else 16, pool, batch, t_cap=cap)
            a = s["cache"]
            s["k_pages"], s["v_pages"] = (a.k_codes, a.v_codes) if fp8 else (a.k16, a.v16)
            s["kT"], s["k_absmax"] = a.kT, a.k_absmax
        else:
            of = lambda shape, t: torch.zeros(shape, dtype=t, device="cuda")  # noqa: E731
            s["k_pages"] = of((pool, hkv, PAGE, D), torch.uint8 if fp8 else torch.float16)
            s["v_pages"] = of((pool, hkv, PAGE, D), torch.uint8 if fp8 else torch.float16)
            s["kT"] = of((batch, hkv, D, cap), torch.float16) if cap else None
            s["k_absmax"] = of((batch, hkv, D), torch.float32) if cap else None
        if cap:
            s["k_absmax"].fill_(2.0)   # of the tokens before
        return s
    if c["op"] == "latent_append":
        nh = c["heads"]
        x = _randn((rows, ROW), g, dt)   # a token's latent values and its key's rotated part, of one projection
        s["c"], s["k"] = x[:, :LAT], x[:, LAT:]
        s["q"] = _randn((rows, nh, D + ROT), g, dt)[:, :, D:]   # the rotated part of its query heads
        s["w"] = torch.rand(LAT, generator=g, device="cuda") + 0.5 if c["norm"] else None
        s["q_out"] = torch.zeros((rows, nh, ROW), dtype=torch.float16, device="cuda")   # the absorbed queries
        if own:
            s["cache"] = kvq.LatentCache(pool)
            s["pages"] = s["cache"].rows
        else:
            s["pages"] = torch.zeros((pool, PAGE, ROW), dtype=torch.float16, device="cuda")
        return s
    if c["op"] == "tree" or c["tree"]:
        s["parents"] = _i32([p for n in news for p in _parents(h, n)])
    if c["op"] == "tree":
        hq, hkv = c["hq"], c["hkv"]
        if own:
            s["cache"] = kvq.LayerCache(hq, hkv, 16, pool, batch)
            s["k16"], s["v16"] = s["cache"].k16, s["cache"].v16
        else:
            s["k16"] = torch.empty((pool, hkv, PAGE, D), dtype=torch.float16, device="cuda")
            s["v16"] = torch.empty((pool, hkv, PAGE, D), dtype=torch.float16, device="cuda")
        s["k16"].copy_(_randn((pool, hkv, PAGE, D), g))
        s["v16"].copy_(_randn((pool, hkv, PAGE, D), g))
        for head in range(hkv):  # a few key channels are large, as in real models
            s["k16"][:, head, :, h.sample(range(D), 4)] *= 10
        s["q"] = _randn((rows, hq, D), g)
        s["slopes"] = 2.0 ** (-8.0 * (torch.arange(hq, device="cuda") + 1) / hq) if c["bias"] else None
        s["out"] = torch.empty((rows, hq, D), dtype=torch.float16, device="cuda")
        s["lse"] = torch.empty((rows, hq), device="cuda")
        if own:
            s["mod"] = kvq.AttnMod(softcap=c["cap"], window=c["window"], n_sink=c["sink"], slopes=s["slopes"])
            s["ws"] = kvq.Workspace(kvq.kv_tree_attn_ws(s["cache"], s["seqs"], rows, s["max_new"]))
        return s
    nh = c["heads"]
    if own:
        s["cache"] = kvq.LatentCache(pool)
        s["pages"] = s["cache"].rows
    else:
        s["pages"] = torch.empty((pool, PAGE, ROW), dtype=torch.float16, device="cuda")
    s["pages"].copy_(_randn((pool, PAGE, ROW), g))
    s["pages"][..., h.sample(range(ROW), 4)] *= 4
    s["q"] = _randn((rows, nh, ROW), g)
    s["out"] = torch.empty((rows, nh, LAT), dtype=torch.float16, device="cuda")
    s["lse"] = torch.empty((rows, nh), device="cuda")
    if own:
        s["ws"] = kvq.Workspace(kvq.kv_latent_attn_ws(s["seqs"], nh, rows, s["max_new"]))
    return s


# ------------------------------------------------------------------ one pass

def _slots(s, rows):
    """(sequence, position) of every new row."""
    starts, lens = s["starts"].long(), s["lens"].long()
    news = starts[1:] - starts[:-1]
    b = torch.repeat_interleave(torch.arange(len(lens), device="cuda"), news, output_size=rows)
    return b, lens[b] - news[b] + torch.arange(rows, device="cuda") - starts[b]


def _turn(x, pos, freqs, interleaved):
    """The first 2 * len(freqs) values of x [n][heads][d] (32 bits) at positions pos, angles in 64."""
    r = 2 * len(freqs)
    a = pos.double()[:, None] * freqs
    cos, sin = torch.cos(a).float()[:, None], torch.sin(a).float()[:, None]
    y = x.clone()
    if interleaved:
        u, v = x[..., 0:r:2], x[..., 1:r:2]
        y[..., 0:r:2], y[..., 1:r:2] = u * cos - v * sin, v * cos + u * sin
    else:
        u, v = x[..., :r // 2], x[..., r // 2:r]
        y[..., :r // 2], y[..., r // 2:r] = u * cos - v * sin, v * cos + u * sin
    return y


def _normed(x, w):
    x = x.float()
    return x if w is None else x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w


def _plain_append(s):
    c = s["case"]
    b, pos = _slots(s, s["q"].shape[0])
    s["q_out"].copy_(_turn(_normed(s["q"], s["wq"]), pos, s["freqs"], c["interleaved"]))
    k, v = _turn(_normed(s["k"], s["wk"]), pos, s["freqs"], c["interleaved"]), s["v"].float()
    if c["cache"] == "e4m3":
        k, v = (x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8) for x in (k, v))
    else:
        k, v = k.half(), v.half()
    page = s["bt"][b, pos // PAGE].long()
    s["k_pages"][page, :, pos % PAGE] = k
    s["v_pages"][page, :, pos % PAGE] = v
    if s["kT"] is not None:
        s["kT"][b, :, :, pos] = k
        at = b[:, None, None].expand(k.shape)
        s["k_absmax"].scatter_reduce_(0, at, k.float().abs(), "amax")
    return _appended(s)


def _appended(s):
    fp8 = s["case"]["cache"] == "e4m3"
    as_is = lambda x: x.view(torch.float8_e4m3fn) if fp8 else x  # noqa: E731
    out = {"q": s["q_out"], "k": as_is(s["k_pages"]), "v": as_is(s["v_pages"])}
    if s["kT"] is not None:
        out.update(kT=s["kT"], k_absmax=s["k_absmax"])
    return out


def _plain_latent_append(s):
    c = s["case"]
    b, pos = _slots(s, s["q"].shape[0])
    s["q_out"][..., LAT:] = _turn(s["q"].float(), pos, s["freqs"], c["interleaved"]).half()
    k = _turn(s["k"].float()[:, None], pos, s["freqs"], c["interleaved"])[:, 0]
    s["pages"][s["bt"][b, pos // PAGE].long(), pos % PAGE] = torch.cat([_normed(s["c"], s["w"]), k], -1).half()
    return {"q": s["q_out"], "pages": s["pages"]}


def _padded(s):
    """New token i of sequence b is row starts[b] + i, short sequences padded: (rows, their number per sequence)."""
    starts = s["starts"].long()
    i = torch.arange(s["max_new"], device="cuda")
    return (starts[:-1, None] + i).clamp(max=int(s["q"].shape[0]) - 1), starts[1:] - starts[:-1], i


def _tree_of(s, row, news, i):
    """Which node [b][i] comes from or is which node [b][j], and the nodes' depths."""
    n = s["max_new"]
    up = s["parents"].long()[row]                                     # [b][n]
    real = i < news[:, None]
    eye = torch.eye(n, device="cuda")
    reach = (eye + (up[:, :, None] == i) * real[:, :, None]).clamp(max=1)
    steps = max(1, math.ceil(math.log2(max(n, 2))))
    for _ in range(steps):                                            # paths of twice the length each time
        reach = torch.matmul(reach, reach).clamp(max=1)
    seen = reach > 0
    return seen, seen.sum(-1) - 1


def _seen(s, row, news, i, t, far=False):
    """[b][n][t]: what each new token sees; with `far` also how far away it is, in positions."""
    c = s["case"]
    lens = s["lens"].long()
    first = (lens - news)[:, None]                                    # where the new tokens begin
    j = torch.arange(t, device="cuda")
    pos, key = first + i, j.expand(len(lens), t)
    seen = (j <= pos[..., None]) & (j < lens[:, None, None])
    if s["parents"] is not None:
        tree, depth = _tree_of(s, row, news, i)
        node = j - first                                              # [b][t]
        inside = (node >= 0) & (node < s["max_new"])
        at = node.clamp(0, s["max_new"] - 1)
        kin = torch.gather(tree, 2, at[:, None].expand(-1, s["max_new"], -1))
        pos = first + depth
        seen = ((j < first)[:, None] | (inside[:, None] & kin)) & (j < lens[:, None, None])
        key = torch.where(inside, first + torch.gather(depth, 1, at), j)
    gap = pos[..., None] - key[:, None]
    if c.get("window"):
        seen &= (gap < c["window"]) | (key < c["sink"])[:, None]
    return (seen, gap.abs()) if far else seen


def _softmax(x):
    """exp(x - max) in place, its sums (1 where nothing is seen) and the natural log of the softmax's denominator."""
    top = x.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    x = x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    return x, torch.where(total > 0, total, torch.ones_like(total)), top + total.log()


def _rows_of(y, s, rows):
    """y [b][heads][n]... -> [rows][heads]..."""
    starts = s["starts"].long()
    b = torch.repeat_interleave(torch.arange(len(starts) - 1, device="cuda"), starts[1:] - starts[:-1], output_size=rows)
    return y[b, :, torch.arange(rows, device="cuda") - starts[b]]


def _plain_tree(s):
    c = s["case"]
    batch, hq, hkv, n = c["batch"], c["hq"], c["hkv"], s["max_new"]
    t, rows = s["bt"].shape[1] * PAGE, s["q"].shape[0]
    row, news, i = _padded(s)
    page = s["bt"].clamp(min=0).long()
    k = s["k16"][page].transpose(2, 3).reshape(batch, t, hkv, D).permute(0, 2, 3, 1).float()
    q = s["q"][row].float().view(batch, n, hkv, hq // hkv, D).permute(0, 2, 3, 1, 4).reshape(batch, hkv, -1, D)
    x = torch.matmul(q, k).view(batch, hkv, hq // hkv, n, t)
    del k
    x *= 1.0 / math.sqrt(D)
    if c["cap"]:
        x = x.div_(c["cap"]).tanh_().mul_(c["cap"])
    seen, far = _seen(s, row, news, i, t, far=True)
    if s["slopes"] is not None:
        x -= s["slopes"].view(1, hkv, -1, 1, 1) * far[:, None, None].float()
    x, total, lse = _softmax(x.masked_fill_(~seen[:, None, None], -math.inf))
    v = s["v16"][page].transpose(2, 3).reshape(batch, t, hkv, D).permute(0, 2, 1, 3).float()
    y = torch.matmul(x.view(batch, hkv, -1, t), v).view(batch, hkv, -1, n, D) / total
    return {"out": _rows_of(y.reshape(batch, hq, n, D), s, rows).half(), "lse": _rows_of(lse.reshape(batch, hq, n), s, rows)}


def _plain_latent(s):
    c = s["case"]
    batch, nh, n = c["batch"], c["heads"], s["max_new"]
    t, rows = s["bt"].shape[1] * PAGE, s["q"].shape[0]
    row, news, i = _padded(s)
    k = s["pages"][s["bt"].clamp(min=0).long()].view(batch, t, ROW).float()
    q = s["q"][row].float().transpose(1, 2).reshape(batch, nh * n, ROW)
    x = torch.matmul(q, k.transpose(1, 2)).view(batch, nh, n, t)
    x *= 1.0 / math.sqrt(D + ROT)
    x, total, lse = _softmax(x.masked_fill_(~_seen(s, row, news, i, t)[:, None], -math.inf))
    y = torch.matmul(x.view(batch, nh * n, t), k[..., :LAT]).view(batch, nh, n, LAT) / total
    return {"out": _rows_of(y, s, rows).half(), "lse": _rows_of(lse[..., 0], s, rows)}


def _plain_expanded(s):
    c = s["case"]
    nh, n, t = c["heads"], s["max_new"], s["max_len"]
    rows = s["q"].shape[0]
    row, news, i = _padded(s)
    at = (s["k_starts"].long()[:-1, None] + torch.arange(t, device="cuda")).clamp(max=s["kv"].shape[0] - 1)
    kv = s["kv"][at].transpose(1, 2)                                  # [b][heads][t][2 D]
    q = s["q"][row].transpose(1, 2).float()                           # [b][heads][n][D + ROT]
    x = torch.matmul(q[..., :D], kv[..., :D].float().transpose(2, 3))
    x += torch.matmul(q[..., D:], s["lat"][at][..., LAT:].float().transpose(1, 2)[:, None])
    x *= 1.0 / math.sqrt(D + ROT)
    x, total, lse = _softmax(x.masked_fill_(~_seen(s, row, news, i, t)[:, None], -math.inf))
    y = torch.matmul(x, kv[..., D:].float()) / total
    return {"out": _rows_of(y, s, rows).half(), "lse": _rows_of(lse[..., 0], s, rows)}


def run(s):
    c = s["case"]
    if own:
        from compressed_kv_cache_quant_gb300 import kvq
        if c["op"] == "append":
            kvq.kv_rope_append(s["cache"], s["seqs"], s["rope"], s["starts"], s["q"], s["k"], s["v"], s["q_out"], s["ws"],
                               q_weight=s["wq"], k_weight=s["wk"], eps=1e-6)
            return _appended(s)
        if c["op"] == "latent_append":
            kvq.kv_latent_append(s["cache"], s["seqs"], s["rope"], s["starts"], s["c"], s["k"], s["ws"], c_weight=s["w"],
                                 eps=1e-6, q=s["q"], q_out=s["q_out"][..., LAT:])
            return {"q": s["q_out"], "pages": s["pages"]}
        if c["op"] == "tree":
            kvq.kv_tree_attn(s["cache"], s["seqs"], s["q"], s["parents"], s["starts"], s["max_new"], s["out"], s["ws"],
                             mod=s["mod"], lse=s["lse"])
        elif c["op"] == "latent":
            kvq.kv_latent_attn(s["cache"], s["seqs"], s["q"], s["starts"], s["max_new"], s["out"], s["ws"],
                               parents=s["parents"], lse=s["lse"])
        else:
            kvq.kv_latent_expanded_attn(s["q"], s["kv"][..., :D], s["lat"][:, LAT:], s["kv"][..., D:], s["starts"],
                                        s["k_starts"], s["max_new"], s["max_len"], s["out"], s["ws"], lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    if c["op"] == "append":
        return _plain_append(s)
    if c["op"] == "latent_append":
        return _plain_latent_append(s)
    return {"tree": _plain_tree, "latent": _plain_latent, "expanded": _plain_expanded}[c["op"]](s)


# ------------------------------------------------------------------ work and values

def work(case):
    c = {"name": "", **case}
    lens, news = _lens(c)
    rows = sum(news)
    if c["op"] == "append":
        size = 1 if c["cache"] == "e4m3" else 2
        kv = c["hkv"] * D
        return {"bytes": rows * (2.0 * (c["hq"] * D + 2 * kv) + 2.0 * c["hq"] * D + 2 * kv * size
                                 + (2 * kv if c["cache"] == "scored" else 0)),
                "flops": 10.0 * rows * (c["hq"] + c["hkv"]) * D}
    if c["op"] == "latent_append":
        return {"bytes": rows * (4.0 * ROW + 4.0 * c["heads"] * ROT), "flops": rows * (6.0 * ROW + 6.0 * c["heads"] * ROT)}
    pairs, read = 0.0, 0
    for t, n in zip(lens, news):
        first, tree = t - n, c["op"] == "tree" or c.get("tree")
        # a node sees the path to it, about a sixth of the nodes; a run sees half of itself
        pairs += n * first + (n * (1 + n / 6.0) if tree else n * (n + 1) / 2.0)
        if c.get("window"):
            pairs -= n * max(0, first - c["window"] - c["sink"])
            read += min(t, n + c["window"] + c["sink"])
        else:
            read += t
    if c["op"] == "tree":
        return {"bytes": read * c["hkv"] * D * 4.0 + rows * c["hq"] * (D * 4.0 + 4), "flops": 4.0 * D * c["hq"] * pairs}
    nh = c["heads"]
    if c["op"] == "latent":
        return {"bytes": 2.0 * read * ROW + rows * nh * (2.0 * ROW + 2 * LAT + 4), "flops": 2.0 * nh * pairs * (ROW + LAT)}
    return {"bytes": read * (nh * D * 4.0 + 2 * ROT) + rows * nh * (2.0 * (D + ROT) + 2 * D + 4),
            "flops": 2.0 * nh * pairs * (2 * D + ROT)}


def _exact_turn(x, pos, c, freqs):
    """x [n][heads][d] in 64 bits: its leading values as complex numbers times e^(i angle)."""
    r = 2 * len(freqs)
    turn = torch.polar(torch.ones((len(pos), r // 2), dtype=torch.float64, device="cuda"), pos.double()[:, None] * freqs)[:, None]
    z = x[..., :r]
    z = z.unflatten(-1, (r // 2, 2)) if c["interleaved"] else z.unflatten(-1, (2, r // 2)).transpose(-1, -2)
    z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * turn)
    z = z if c["interleaved"] else z.transpose(-1, -2)
    return torch.cat([z.flatten(-2), x[..., r:]], -1)


def _exact_norm(x, w):
    x = x.double()
    return x if w is None else w.double() * x / ((x ** 2).sum(-1, keepdim=True) / x.shape[-1] + 1e-6).sqrt()


def _exact_written(s, lens, news):
    c = s["case"]
    pos = torch.cat([torch.arange(t - n, t, device="cuda") for t, n in zip(lens, news)])
    seq = torch.cat([torch.full((n,), b, device="cuda") for b, n in enumerate(news)])
    page, slot = s["bt"].long()[seq, pos // PAGE], pos % PAGE
    if c["op"] == "latent_append":
        q = s["q_out"].double()
        q[..., LAT:] = _exact_turn(s["q"].double(), pos, c, s["freqs"])
        pages = s["pages"].double()
        k = _exact_turn(s["k"].double()[:, None], pos, c, s["freqs"])[:, 0]
        pages.view(-1, ROW)[page * PAGE + slot] = torch.cat([_exact_norm(s["c"], s["w"]), k], -1)
        return {"q": q, "pages": pages}
    k, v = _exact_turn(_exact_norm(s["k"], s["wk"]), pos, c, s["freqs"]), s["v"].double()
    out = {"q": _exact_turn(_exact_norm(s["q"], s["wq"]), pos, c, s["freqs"])}
    for name, x in (("k", k), ("v", v)):
        y = torch.zeros(s[name + "_pages"].shape, dtype=torch.float64, device="cuda")
        y = y.transpose(1, 2).contiguous()
        y.view(-1, c["hkv"], D)[page * PAGE + slot] = x.clamp(-448, 448) if c["cache"] == "e4m3" else x
        out[name] = y.transpose(1, 2).contiguous()
    if s["kT"] is not None:
        kT, top = s["kT"].double(), s["k_absmax"].double()
        at = 0
        for b, (t, n) in enumerate(zip(lens, news)):
            kT[b, :, :, t - n:t] = k[at:at + n].permute(1, 2, 0)
            top[b] = torch.maximum(top[b], k[at:at + n].half().double().abs().amax(0))
            at += n
        out.update(kT=kT, k_absmax=None)   # (a maximum of rounded values)
    return out


def exact(case, seed):
    """The operators from their definitions in 64 bits, one sequence and one head at a time."""
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    c = s["case"]
    lens, news = _lens(c)
    if c["op"] in ("append", "latent_append"):
        return _exact_written(s, lens, news)
    nh = c["hq"] if c["op"] == "tree" else c["heads"]
    width = LAT if c["op"] == "latent" else D
    rows = sum(news)
    out = torch.zeros((rows, nh, width), dtype=torch.float64, device="cuda")
    lse = torch.full((rows, nh), -math.inf, dtype=torch.float64, device="cuda")
    first = at = 0
    for b, (t, n) in enumerate(zip(lens, news)):
        where = torch.arange(t, device="cuda")                        # the position of every key
        seen = where[None] <= (torch.arange(n, device="cuda") + t - n)[:, None]
        if s["parents"] is not None:
            up = s["parents"][first:first + n].tolist()
            paths = []                                                # of every node, itself last
            for i, p in enumerate(up):
                paths.append((paths[p] if p >= 0 else []) + [i])
            seen[:, t - n:] = False
            for i, p in enumerate(paths):
                seen[i, [t - n + x for x in p]] = True
            where[t - n:] = torch.tensor([t - n + len(p) - 1 for p in paths], device="cuda")
        here = where[t - n:, None]
        if c.get("window"):
            seen = seen & ((here - where[None] < c["window"]) | (where[None] < c["sink"]))
        if c["op"] != "expanded":
            pages = s["bt"][b, :-(-t // PAGE)].long()
        if c["op"] == "latent":
            lat = s["pages"][pages].reshape(-1, ROW)[:t].double()
        for h in range(nh):
            q = s["q"][first:first + n, h].double()
            if c["op"] == "tree":
                g = h // (nh // c["hkv"])
                k, v = (s[a][pages, g].reshape(-1, D)[:t].double() for a in ("k16", "v16"))
            elif c["op"] == "latent":
                k, v = lat, lat[:, :LAT]
            else:
                k = torch.cat([s["kv"][at:at + t, h, :D], s["lat"][at:at + t, LAT:]], -1).double()
                v = s["kv"][at:at + t, h, D:].double()
            x = q @ k.T / math.sqrt(D if c["op"] == "tree" else D + ROT)
            if c.get("cap"):
                x = c["cap"] * torch.tanh(x / c["cap"])
            if s.get("slopes") is not None:
                x = x - float(s["slopes"][h]) * (here - where[None]).abs()
            x = x.masked_fill(~seen, -math.inf)
            z = torch.logsumexp(x, -1)
            p = torch.exp(x - torch.where(torch.isinf(z), torch.zeros_like(z), z)[:, None])
            out[first:first + n, h] = p @ v
            lse[first:first + n, h] = z
        first += n
        at += t
    return {"out": out, "lse": lse}
