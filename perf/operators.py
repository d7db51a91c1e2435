"""The paged-cache operators: what each computes, in elementary torch operations, and the cases they are timed on.

A pool holds pages of ``page`` tokens, K and V [n_pages, page, d]; every (row, KV head) has its own page list, since
compression leaves every head with its own number of tokens: table int32 [batch, heads, max_pages], lens int32
[batch, heads], refs int32 [n_pages] (lists that hold a page; 0 is free).
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
ESIZE = {"bf16": 2, "e4m3": 1}


def listed():
    return [
        # One sequence answering token by token over one layer of a half-kept 4096-token cache: latency.
        _attn("attn-decode-1x8-t2k", batch=1, heads=8, group=4, d=128, dtype="bf16", page=16, t_lo=1900, t_hi=2048,
              q_lo=1, q_hi=1),
        # A serving batch's decode step in one layer: prompts of 8K to 32K tokens, half kept.
        _attn("attn-decode-32x8-t4k-16k", batch=32, heads=8, group=4, d=128, dtype="bf16", page=32, t_lo=4096,
              t_hi=16384, q_lo=1, q_hi=1),
        # Two long 8-bit caches (131072 tokens, half kept, 10 KV heads): few rows over a long axis.
        _attn("attn-decode-e4m3-2x10-t64k", batch=2, heads=10, group=4, d=128, dtype="e4m3", page=64, t_lo=60001,
              t_hi=65537, q_lo=1, q_hi=1),
        # A mixed step: some rows decode, some bring up to 512 prompt tokens, sliding window with 64 first tokens.
        _attn("attn-mixed-8x8-window", batch=8, heads=8, group=4, d=128, dtype="bf16", page=16, t_lo=6001, t_hi=16384,
              q_lo=1, q_hi=512, window=4096, sinks=64),
        # A chunk of a long prompt over what the cache holds of it.
        _attn("attn-chunk-2048-t32k", batch=1, heads=8, group=4, d=128, dtype="bf16", page=64, t_lo=32768, t_hi=32768,
              q_lo=2048, q_hi=2048),
        # One new token of each of 16 sequences: latency.
        _rope("rope-decode-16", batch=16, heads=8, group=4, d=128, dtype="bf16", page=16, q_lo=1, q_hi=1, rot=128,
              layout="half", pos=131072),
        # Prompt chunks into an 8-bit cache, half of each head rotated, neighbouring pairs.
        _rope("rope-chunks-e4m3-part", batch=7, heads=10, group=4, d=128, dtype="e4m3", page=64, q_lo=1, q_hi=1000,
              rot=64, layout="interleaved", pos=1048576),
        # A long prompt of one sequence at once.
        _rope("rope-prompt-16k", batch=1, heads=8, group=4, d=128, dtype="bf16", page=32, q_lo=16384, q_hi=16384,
              rot=128, layout="half", pos=131072),
        # Beams of one sequence after a step: some die, some fork.
        _update("update-beams-8x8", batch=8, heads=8, d=128, dtype="bf16", page=16, t_lo=900, t_hi=2048, moved=0.9),
        # A serving step over the layers of many sequences: most go on, some end, some fork.
        _update("update-serve-512x8", batch=512, heads=8, d=128, dtype="bf16", page=16, t_lo=500, t_hi=2048,
                moved=0.25),
        # One layer's compressed prompt into fresh pages (20% removed).
        _compact("compact-fill-1x8-t4k", batch=1, heads=8, d=128, dtype="bf16", page=16, t_lo=4096, t_hi=4096, ratio=0.2,
                 source="cache"),
        # A ragged batch's paged cache halved.
        _compact("compact-pages-8x8-t8k-32k", batch=8, heads=8, d=128, dtype="bf16", page=32, t_lo=8192, t_hi=32768,
                 ratio=0.5, source="pages"),
    ]


def _attn(name=None, window=0, sinks=0, **c):
    return _case(name, op="attention", window=window, sinks=sinks, **c)


def _rope(name=None, **c):
    return _case(name, op="rope", **c)


def _update(name=None, **c):
    return _case(name, op="update", **c)


def _compact(name=None, **c):
    return _case(name, op="compact", **c)


def _case(name, **c):
    return dict(c, name=name) if name else c


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], evenly over its logarithm."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49))))))


def draw(rng):
    """One more case of the ranges that the listed ones stand for."""
    op = rng.choice(["attention", "attention", "attention", "rope", "update", "compact"])
    d = rng.choice([64, 128, 128, 128, 256])
    c = dict(heads=rng.choice([1, 2, 3, 4, 8, 8, 10]), d=d, dtype=rng.choice(["bf16", "bf16", "e4m3"]),
             page=rng.choice([16, 16, 32, 64, 128]))
    if op == "attention":
        kind = rng.choice(["decode", "decode", "mixed", "chunk"])
        c.update(group=rng.choice([1, 2, 3, 4, 4, 5, 7, 8, 16]))
        c.update(batch=_spread(rng, 1, 4 if kind == "chunk" else 32), q_lo=1)
        c["q_hi"] = 1 if kind == "decode" else _spread(rng, 2, 300 if kind == "mixed" else 2048)
        c["t_hi"] = _spread(rng, 64, 65537)
        # no more scores than the largest listed case has, nor more cached elements
        rows = c["batch"] * c["heads"]
        c["t_hi"] = min(c["t_hi"], 32 * 8 * 16384 * 128 // (rows * d),
                        2 ** 29 * 128 // (rows * c["group"] * c["q_hi"] * d))
        c["q_hi"] = min(c["q_hi"], c["t_hi"])
        c["t_lo"] = max(c["q_hi"], _spread(rng, 1, c["t_hi"]))
        c.update(rng.choice([dict(window=0, sinks=0), dict(window=0, sinks=0),
                             dict(window=_spread(rng, 16, 8192), sinks=rng.choice([0, 1, 4, 64, 100]))]))
        return _attn(**c)
    if op == "rope":
        c.update(batch=_spread(rng, 1, 32), group=rng.choice([1, 2, 3, 4, 4, 7, 8]))
        c["q_hi"] = max(1, min(_spread(rng, 1, 16384), 16384 * 40 * 128 // (c["batch"] * c["heads"] * (c["group"] + 2) * d)))
        c["q_lo"] = _spread(rng, 1, c["q_hi"])
        c.update(rot=rng.choice([r for r in (16, 32, 64, 96, 128, 256) if r <= d] + [d, d]),
                 layout=rng.choice(["half", "interleaved"]), pos=_spread(rng, 4096, 1048576))
        return _rope(**c)
    if op == "update":
        c.update(batch=_spread(rng, 1, 512), moved=rng.choice([0.0, 0.1, 0.3, 0.9]))
        c["t_hi"] = min(_spread(rng, 1, 16384), 512 * 8 * 2048 * 128 // (c["batch"] * c["heads"] * d))
        c["t_lo"] = _spread(rng, 1, c["t_hi"])
        return _update(**c)
    c.update(batch=_spread(rng, 1, 16), ratio=rng.choice([0.2, 0.25, 0.5, 0.75, 0.9]), source=rng.choice(["cache", "pages"]))
    c["t_hi"] = min(_spread(rng, 16, 65536), 8 * 8 * 32768 * 128 // (c["batch"] * c["heads"] * d))
    c["t_lo"] = _spread(rng, 1, c["t_hi"])
    return _compact(**c)


# ------------------------------------------------------------------- inputs --

def _pages(tokens, page):
    return (tokens + page - 1) // page


def _values(g, shape, dtype, sigma):
    """Normal rows with a lognormal magnitude per token, as cached keys show."""
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
    if sigma:
        x *= torch.exp(sigma * torch.randn(shape[:-1] + (1,), generator=g, device="cuda"))
    return x.clamp_(-448, 448).to(DTYPES[dtype])


def _lists(g, c, lens, max_pages, spare):
    """Page lists over a shuffled pool: table, lens, refs. `spare` pages are free; one page more is held back by the
    program (the last; no list has it). None: a pool that would hold every list at its longest."""
    lens = lens.to(torch.int32)
    count = _pages(lens.long(), c["page"]).flatten()
    used = int(count.sum())
    n = lens.numel() * max_pages if spare is None else used + spare
    perm = torch.randperm(n, generator=g, device="cuda")
    slot = torch.arange(max_pages, device="cuda")
    first = torch.cumsum(count, 0) - count
    table = torch.full((lens.numel(), max_pages), -1, dtype=torch.int32, device="cuda")
    live = slot[None] < count[:, None]
    table[live] = perm[(first[:, None] + slot[None])[live]].to(torch.int32)
    refs = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
    refs[perm[:used]] = 1
    refs[n] = 1
    return table.view(*lens.shape, max_pages), lens, refs


def _pool(g, c, n_pages):
    k = torch.empty((n_pages, c["page"], c["d"]), dtype=DTYPES[c["dtype"]], device="cuda")
    v = torch.empty_like(k)
    step = max(1, 2 ** 26 // (c["page"] * c["d"]))
    for i in range(0, n_pages, step):
        m = min(step, n_pages - i)
        k[i:i + m] = _values(g, (m, c["page"], c["d"]), c["dtype"], 0.5)
        v[i:i + m] = _values(g, (m, c["page"], c["d"]), c["dtype"], 0.0)
    return k, v


def _poison(c, k, v, table, lens):
    """Rows behind each list's last token hold whatever was there: NaN here."""
    tail = lens.flatten().long() % c["page"]
    last = table.flatten(0, 1).gather(1, (_pages(lens.flatten().long(), c["page"]) - 1).clamp(min=0)[:, None])[:, 0].long()
    rows = torch.arange(c["page"], device="cuda")
    hit = (rows[None] >= tail[:, None]) & (tail[:, None] > 0)
    where = (last[:, None] * c["page"] + rows[None])[hit]
    nan = torch.full((1,), float("nan"), device="cuda").to(k.dtype)
    for x in (k, v):
        x.view(-1, c["d"]).view(torch.uint8)[where] = nan.view(torch.uint8).repeat(c["d"])


def _draw_len(g, lo, hi, shape):
    """Numbers of [lo, hi]: the range and the shape settle which ones, the seed their order, so that every seed's tensors
    have the same sizes."""
    n = math.prod(shape)
    same = torch.Generator()
    same.manual_seed(1000003 * lo + 101 * hi + n)
    x = torch.randint(lo, hi + 1, (n,), generator=same).cuda()
    return x[torch.randperm(n, generator=g, device="cuda")].view(shape)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": c}
    B, H = c["batch"], c["heads"]
    if c["op"] in ("attention", "rope"):
        n_q = _draw_len(g, c["q_lo"], c["q_hi"], (B,))
        if c["q_hi"] > 1 and c["q_lo"] == 1 and B > 2:
            # a third of the rows answer, the others still read their prompt
            n_q = torch.where(n_q <= n_q.sort().values[(B - 1) // 3], 1, n_q)
        s["q_start"] = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), n_q.cumsum(0)]).to(torch.int32)
        n = int(n_q.sum())
        hq = H * c["group"]
    if c["op"] == "attention":
        lens = _draw_len(g, c["t_lo"], c["t_hi"], (B, H))
        s["table"], s["lens"], refs = _lists(g, c, lens, _pages(c["t_hi"], c["page"]), 8)
        s["k_pages"], s["v_pages"] = _pool(g, c, refs.numel())
        _poison(c, s["k_pages"], s["v_pages"], s["table"], s["lens"])
        s["Q"] = _values(g, (n, hq, c["d"]), "bf16", 0.0)
        s["max_q"], s["max_len"] = c["q_hi"], c["t_hi"]
        s["scale"] = 1.0 / math.sqrt(c["d"])
        s["k_scale"], s["v_scale"] = (0.75, 1.25) if c["dtype"] == "e4m3" else (1.0, 1.0)
    elif c["op"] == "rope":
        old = _draw_len(g, 0, 200, (B, H))
        lens = old + n_q[:, None]
        s["table"], s["lens"], refs = _lists(g, c, lens, _pages(c["q_hi"] + 200, c["page"]), None)
        s["k_pages"], s["v_pages"] = _pool(g, c, refs.numel())
        # the three projections of one fused product: rows of (hq + 2 H) heads
        qkv = _values(g, (n, hq + 2 * H, c["d"]), "bf16", 0.3)
        s["Q"], s["K"], s["V"] = qkv[:, :hq], qkv[:, hq:hq + H], qkv[:, hq + H:]
        first = _draw_len(g, 0, max(0, c["pos"] - c["q_hi"]), (B,))
        row = torch.repeat_interleave(torch.arange(B, device="cuda"), n_q)
        s["positions"] = (first[row] + torch.arange(n, device="cuda") - s["q_start"].long()[row]).to(torch.int32)
        i = torch.arange(c["rot"] // 2, device="cuda", dtype=torch.float64)
        s["inv_freq"] = (500000.0 ** (-2.0 * i / c["rot"])).float()
        s["factor"] = 1.0 if c["pos"] <= 131072 else 0.1 * math.log(c["pos"] / 131072) + 1.0
        s["k_scale"], s["v_scale"] = (0.0625, 0.03125) if c["dtype"] == "e4m3" else (1.0, 1.0)
        s["Q_out"] = torch.zeros((n, hq, c["d"]), dtype=torch.bfloat16, device="cuda")
    elif c["op"] == "update":
        lens = _draw_len(g, c["t_lo"], c["t_hi"], (B, H))
        max_pages = _pages(c["t_hi"] + 40, c["page"])
        parent = torch.arange(B, device="cuda")
        u = torch.rand((B,), generator=g, device="cuda")
        other = torch.randint(0, B, (B,), generator=g, device="cuda")
        parent = torch.where(u < c["moved"] / 4, torch.full_like(parent, -1), torch.where(u < c["moved"], other, parent))
        s["parent"] = parent.to(torch.int32)
        # one token each, a few rows a drafted run of them
        n_new = torch.where(torch.rand((B,), generator=g, device="cuda") < 0.05, _draw_len(g, 0, 40, (B,)), 1)
        s["n_new"] = n_new.to(torch.int32)
        s["table"], s["lens"], s["refs"] = _lists(g, c, lens, max_pages, B * H * (2 + _pages(40, c["page"])))
        s["k_pages"], s["v_pages"] = _pool(g, c, s["refs"].numel())
    else:
        T = _draw_len(g, c["t_lo"], c["t_hi"], (B, 1)).expand(B, H).contiguous()
        kept = torch.floor(T.double() * (1 - c["ratio"]) + 0.5).long()
        s["stride"] = int(math.floor(c["t_hi"] * (1 - c["ratio"]) + 0.5))
        # kept tokens ascending: the tokens of the `kept` largest of T random scores
        score = torch.rand((B, H, c["t_hi"]), generator=g, device="cuda")
        score[torch.arange(c["t_hi"], device="cuda") >= T[..., None]] = -1
        order = score.argsort(-1, descending=True)[..., :max(1, s["stride"])]
        slot = torch.arange(order.shape[-1], device="cuda")
        order = torch.where(slot < kept[..., None], order, 2 ** 30).sort(-1).values
        s["idx"] = torch.where(slot < kept[..., None], order, -7).to(torch.int32).contiguous()
        s["kept"] = kept.to(torch.int32)
        spare = int(_pages(kept, c["page"]).sum()) + 3
        lens = T if c["source"] == "pages" else torch.zeros_like(T)
        s["table"], s["lens"], s["refs"] = _lists(g, c, lens, _pages(c["t_hi"], c["page"]), spare)
        s["k_pages"], s["v_pages"] = _pool(g, c, s["refs"].numel())
        s["K"] = s["V"] = s["seq_lens"] = None
        if c["source"] == "cache":
            s["K"] = _values(g, (B, H, c["t_hi"], c["d"]), c["dtype"], 0.5)
            s["V"] = _values(g, (B, H, c["t_hi"], c["d"]), c["dtype"], 0.0)
            s["seq_lens"] = T[:, 0].to(torch.int32).contiguous()
    if c["op"] in ("update", "compact"):
        s["table_out"] = torch.full_like(s["table"], -1)
        s["lens_out"], s["refs_out"] = torch.zeros_like(s["lens"]), torch.zeros_like(s["refs"])
    if own:
        import geometric_kv_cache_gb300 as mkv
        if c["op"] == "attention":
            s["O"] = torch.empty_like(s["Q"])
            s["lse"] = torch.empty(s["Q"].shape[:2], dtype=torch.float32, device="cuda")
            s["ws"] = mkv.attention_workspace_for(s["Q"], s["k_pages"], s["table"], s["max_q"], s["max_len"])
        else:
            s["ws"] = mkv.page_workspace_for(s["k_pages"], s["table"])
    return s


# --------------------------------------------------------------- one pass --

def run(state):
    s, c = state, state["case"]
    if own:
        import geometric_kv_cache_gb300 as mkv
        if c["op"] == "attention":
            mkv.mkv_paged_attention(s["Q"], s["k_pages"], s["v_pages"], s["table"], s["lens"], s["q_start"], s["max_q"],
                                    s["max_len"], s["O"], s["ws"], scale=s["scale"], k_scale=s["k_scale"],
                                    v_scale=s["v_scale"], window=c["window"], sinks=c["sinks"], lse=s["lse"])
            return {"O": s["O"], "lse": s["lse"]}
        if c["op"] == "rope":
            mkv.mkv_rope_append(s["Q"], s["K"], s["V"], s["positions"], s["inv_freq"], s["k_pages"], s["v_pages"],
                                s["table"], s["lens"], s["q_start"], s["Q_out"], s["ws"], layout=c["layout"],
                                factor=s["factor"], k_scale=s["k_scale"], v_scale=s["v_scale"])
            return {"Q": s["Q_out"], "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
        if c["op"] == "update":
            mkv.mkv_page_update(s["k_pages"], s["v_pages"], s["table"], s["lens"], s["refs"], s["table_out"],
                                s["lens_out"], s["refs_out"], s["ws"], parent=s["parent"], n_new=s["n_new"])
        else:
            mkv.mkv_page_compact(s["k_pages"], s["v_pages"], s["table"], s["lens"], s["refs"], s["idx"], s["kept"],
                                 s["table_out"], s["lens_out"], s["refs_out"], s["ws"], K=s["K"], V=s["V"],
                                 seq_lens=s["seq_lens"])
        return {k: s[k] for k in ("table_out", "lens_out", "refs_out", "k_pages", "v_pages")}
    return {"attention": _plain_attention, "rope": _plain_rope, "update": _plain_update, "compact": _plain_compact}[c["op"]](s, c)


def _plain_attention(s, c):
    B, H, G, D, page = c["batch"], c["heads"], c["group"], c["d"], c["page"]
    dev = s["Q"].device
    slot = torch.arange(s["max_len"], device=dev)
    lens = s["lens"].long().view(B, H, 1)
    live = slot < lens
    pages = s["table"].long().view(B, H, -1)[:, :, slot // page].clamp(min=0)
    k, v = (s[x].view(torch.uint8)[pages, slot % page].view(s[x].dtype).float() for x in ("k_pages", "v_pages"))
    k, v = k * s["k_scale"], v * s["v_scale"]
    k = torch.where(live[..., None], k, 0.0)
    v = torch.where(live[..., None], v, 0.0)
    start = s["q_start"].long()
    n = start[1:] - start[:-1]
    i = torch.arange(s["max_q"], device=dev)
    there = i < n[:, None]
    token = torch.where(there, start[:-1, None] + i, 0)
    q = s["Q"][token].float().view(B, -1, H, G, D).permute(0, 2, 1, 3, 4)  # [B, H, max_q, G, D]
    sc = torch.matmul(q.reshape(B, H, -1, D), k.transpose(-1, -2)).view(B, H, -1, G, s["max_len"]) * s["scale"]
    p = lens - n.view(B, 1, 1) + i  # [B, H, max_q]: the query's own entry
    seen = slot <= p[..., None]
    if c["window"]:
        seen &= (slot > p[..., None] - c["window"]) | (slot < c["sinks"])
    seen &= live[:, :, None]
    sc = torch.where(seen[:, :, :, None], sc, -math.inf)
    m = sc.amax(-1, keepdim=True)
    e = torch.exp(sc - torch.where(m == -math.inf, 0.0, m))
    l = e.sum(-1, keepdim=True)
    o = torch.matmul(e.view(B, H, -1, s["max_len"]), v).view(B, H, -1, G, D) / torch.where(l == 0, 1.0, l)
    lse = (m + torch.log(l))[..., 0]
    # back to the packed tokens
    t = torch.arange(s["Q"].shape[0], device=dev)
    b = torch.searchsorted(start[1:], t, right=True)
    j = t - start[b]
    return {"O": o[b, :, j].reshape(-1, H * G, D).to(torch.bfloat16), "lse": lse[b, :, j].reshape(-1, H * G)}


def _rotate(x, cos, sin, c):
    """x [n, heads, d] in 32 bits, the first `rot` dims rotated by the angles of cos and sin [n, rot / 2]."""
    r = c["rot"]
    cos, sin = cos[:, None], sin[:, None]
    if c["layout"] == "half":
        a, b = x[..., :r // 2], x[..., r // 2:r]
        y = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    else:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    return torch.cat([y, x[..., r:]], -1)


def _plain_rope(s, c):
    a = s["positions"].double()[:, None] * s["inv_freq"].double()
    # the factor multiplies the rotated part alone
    cos, sin = (a.cos() * s["factor"]).float(), (a.sin() * s["factor"]).float()
    s["Q_out"].copy_(_rotate(s["Q"].float(), cos, sin, c))
    start, lens = s["q_start"].long(), s["lens"].long()
    t = torch.arange(s["Q"].shape[0], device=a.device)
    b = torch.searchsorted(start[1:], t, right=True)
    slot = lens[b] - (start[b + 1] - t)[:, None]  # [n, H]
    h = torch.arange(c["heads"], device=a.device)
    pages = s["table"].long()[b[:, None], h, slot // c["page"]]
    for name, x, scale in (("k_pages", _rotate(s["K"].float(), cos, sin, c), s["k_scale"]),
                           ("v_pages", s["V"].float(), s["v_scale"])):
        if c["dtype"] == "e4m3":
            x = (x / scale).clamp(-448, 448)
        x = x.to(DTYPES[c["dtype"]])
        s[name].view(torch.uint8)[pages, slot % c["page"]] = x.contiguous().view(torch.uint8)
    return {"Q": s["Q_out"], "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _plain_update(s, c):
    B, H, page = c["batch"], c["heads"], c["page"]
    dev = s["table"].device
    table, lens, refs = s["table"].long(), s["lens"].long(), s["refs"]
    rows = torch.arange(B, device=dev)
    parent = s["parent"].long()
    a = parent.clamp(min=0)
    gone = (parent < 0)[:, None]
    old = torch.where(gone, 0, lens[a])  # [B, H]
    new = torch.where(gone, 0, old + s["n_new"].long()[:, None])
    # who keeps a partly filled last page: the row itself, else its lowest child
    child = torch.full((B,), B, device=dev).scatter_reduce(0, a, torch.where(parent < 0, B, rows), "amin")
    keeper = torch.where(parent == rows, rows, child)
    keeps = (keeper[a] == rows)[:, None]
    shared = torch.where(keeps, _pages(old, page), old // page)
    total = _pages(new, page)
    need = (total - shared).flatten()
    first = (need.cumsum(0) - need).view(B, H, 1)
    free = torch.argsort((refs != 0).to(torch.int8), stable=True)  # free pages first, ascending
    slot = torch.arange(table.shape[-1], device=dev)
    fresh = (slot >= shared[..., None]) & (slot < total[..., None])
    took = free[torch.where(fresh, first + slot - shared[..., None], 0)]
    out = torch.where(slot < shared[..., None], table[a], took)
    held = slot < total[..., None]
    s["table_out"].copy_(torch.where(held, out, s["table_out"].long()))
    s["lens_out"].copy_(new)
    count = refs.long()
    count = count.scatter_add(0, torch.where(held, out, 0).flatten(), held.long().flatten())
    had = slot < _pages(lens, page)[..., None]
    count = count.scatter_add(0, torch.where(had, table, 0).flatten(), -had.long().flatten())
    s["refs_out"].copy_(count)
    # the partly filled last pages of the other children (the others "copy" the reserved page onto itself)
    copied = (~keeps & (old % page > 0)).flatten()
    at = (old // page).clamp(max=table.shape[-1] - 1)[..., None]
    spare = refs.numel() - 1
    src = torch.where(copied, table[a].gather(-1, at).flatten(), spare)
    dst = torch.where(copied, out.gather(-1, at).flatten(), spare)
    row = torch.arange(page, device=dev)
    real = (row < (old % page).flatten()[:, None])[..., None]
    for x in (s["k_pages"].view(torch.uint8), s["v_pages"].view(torch.uint8)):
        x[dst] = torch.where(real, x[src], x[dst])
    return {k: s[k] for k in ("table_out", "lens_out", "refs_out", "k_pages", "v_pages")}


def _plain_compact(s, c):
    B, H, page = c["batch"], c["heads"], c["page"]
    dev = s["table"].device
    table, refs, kept = s["table"].long(), s["refs"], s["kept"].long()
    total = _pages(kept, page)
    need = total.flatten()
    first = (need.cumsum(0) - need).view(B, H, 1)
    free = torch.argsort((refs != 0).to(torch.int8), stable=True)
    slot = torch.arange(table.shape[-1], device=dev)
    held = slot < total[..., None]
    out = free[torch.where(held, first + slot, 0)]
    s["table_out"].copy_(torch.where(held, out, s["table_out"].long()))
    s["lens_out"].copy_(kept)
    count = refs.long().scatter_add(0, out.flatten(), held.long().flatten())
    had = slot < _pages(s["lens"].long(), page)[..., None]
    s["refs_out"].copy_(count.scatter_add(0, torch.where(had, table, 0).flatten(), -had.long().flatten()))
    i = torch.arange(s["idx"].shape[-1], device=dev)
    real = i < kept[..., None]
    spare = (refs.numel() - 1) * page  # rows of the reserved page
    src = torch.where(real, s["idx"].long(), 0)
    dst = torch.where(real, out.gather(-1, (i // page).expand(B, H, -1)) * page + i % page, spare)
    for x, cache in ((s["k_pages"], s["K"]), (s["v_pages"], s["V"])):
        flat = x.view(torch.uint8).flatten(0, 1)
        if cache is None:
            rows = flat[torch.where(real, table.gather(-1, src // page) * page + src % page, spare)]
        else:
            rows = cache.view(torch.uint8).gather(2, src[..., None].expand(B, H, -1, flat.shape[-1]))
        flat[dst] = torch.where(real[..., None], rows, flat[spare])
    return {k: s[k] for k in ("table_out", "lens_out", "refs_out", "k_pages", "v_pages")}


# ------------------------------------------------------------------- work --

def work(case):
    """Mean bytes and operations of one pass over the case's ranges."""
    c = case
    row = c["d"] * ESIZE[c["dtype"]]
    lists = c["batch"] * c["heads"]
    if c["op"] == "attention":
        q = (c["q_lo"] + c["q_hi"]) / 2
        if c["q_hi"] > 1 and c["q_lo"] == 1 and c["batch"] > 2:
            q = (2 * q + 1) / 3
        t = max((max(c["t_lo"], q) + c["t_hi"]) / 2, q)
        seen = read = t
        if c["window"] and c["window"] + q + c["sinks"] < t:
            seen, read = c["window"] + c["sinks"], c["window"] + q + c["sinks"]
        else:
            seen = t - q / 2
        io = c["batch"] * q * c["heads"] * c["group"] * (c["d"] * 4 + 4)
        return {"bytes": lists * read * 2 * row + io, "flops": 4.0 * c["d"] * lists * c["group"] * q * seen}
    if c["op"] == "rope":
        q = (c["q_lo"] + c["q_hi"]) / 2
        if c["q_hi"] > 1 and c["q_lo"] == 1 and c["batch"] > 2:
            q = (2 * q + 1) / 3
        n = c["batch"] * q
        return {"bytes": n * (c["heads"] * (c["group"] * c["d"] * 4 + 2 * (c["d"] * 2 + row)) + 4),
                "flops": n * c["heads"] * (c["group"] + 1) * c["rot"] * 3.0}
    if c["op"] == "update":
        t = (c["t_lo"] + c["t_hi"]) / 2
        held = lists * _pages(t, c["page"])
        pool = held + lists * (2 + _pages(40, c["page"]))
        copied = lists * c["moved"] * 0.6 * c["page"] / 2
        return {"bytes": 8 * held + 8 * pool + 8 * lists + copied * 4 * row, "flops": 0}
    t = (c["t_lo"] + c["t_hi"]) / 2
    n = lists * t * (1 - c["ratio"])
    held = lists * _pages(t, c["page"]) * (2 if c["source"] == "pages" else 1)
    return {"bytes": n * (4 * row + 4) + 8 * held, "flops": 0}


# ------------------------------------------------------------------ 64 bits --

def exact(case, seed):
    """Attention and rotation from their definitions in 64 bits; the page operators return no computed numbers."""
    c = case
    if c["op"] not in ("attention", "rope"):
        return None
    s = prepare(case, seed)
    start, lens, table = s["q_start"].tolist(), s["lens"].tolist(), s["table"]
    page = c["page"]
    if c["op"] == "attention":
        O = torch.zeros(s["Q"].shape, dtype=torch.float64, device="cuda")
        lse = torch.full(s["Q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
        for b in range(c["batch"]):
            n = start[b + 1] - start[b]
            for j in range(c["heads"]):
                L = lens[b][j]
                ids = table[b, j, :_pages(L, page)].long()
                K, V = (s[x].view(torch.uint8)[ids].view(s[x].dtype).flatten(0, 1)[:L].double() for x in ("k_pages", "v_pages"))
                K, V = K * s["k_scale"], V * s["v_scale"]
                own_entry = L - n + torch.arange(n, device="cuda")
                at = torch.arange(L, device="cuda")
                back = own_entry[:, None] - at[None]
                hidden = back < 0
                if c["window"]:
                    hidden |= (back >= c["window"]) & (at >= c["sinks"])
                for h in range(j * c["group"], (j + 1) * c["group"]):
                    z = (s["Q"][start[b]:start[b + 1], h].double() * s["scale"]) @ K.T
                    z.masked_fill_(hidden, -math.inf)
                    lse[start[b]:start[b + 1], h] = torch.logsumexp(z, 1)
                    w = torch.softmax(z, 1).nan_to_num_(0.0)
                    O[start[b]:start[b + 1], h] = w @ V
        return {"O": O, "lse": lse}
    n = s["Q"].shape[0]
    i = torch.arange(c["rot"] // 2, device="cuda")
    lo, hi = (i, i + c["rot"] // 2) if c["layout"] == "half" else (2 * i, 2 * i + 1)
    angle = torch.outer(s["positions"].double(), s["inv_freq"].double())
    turn = torch.polar(torch.full_like(angle, s["factor"]), angle)[:, None]

    def turned(x):
        y = x.double().clone()
        z = torch.complex(y[..., lo], y[..., hi]) * turn
        y[..., lo], y[..., hi] = z.real, z.imag
        return y

    kp, vp = s["k_pages"].double(), s["v_pages"].double()
    K, V = turned(s["K"]), s["V"].double()
    if c["dtype"] == "e4m3":
        K, V = (K / s["k_scale"]).clamp(-448, 448), (V / s["v_scale"]).clamp(-448, 448)
    for b in range(c["batch"]):
        m = start[b + 1] - start[b]
        for j in range(c["heads"]):
            at = torch.arange(lens[b][j] - m, lens[b][j], device="cuda")
            ids = table[b, j][at // page].long()
            kp[ids, at % page] = K[start[b]:start[b + 1], j]
            vp[ids, at % page] = V[start[b]:start[b + 1], j]
    return {"Q": turned(s["Q"]), "k_pages": kp, "v_pages": vp}
