"""Caches held in 4 bits and rotary positions with several axes: what each operator computes, in elementary torch
operations, and the cases they are timed on.

A 4-bit pool holds, for every token and head, an E2M1 code per element (values 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their
negatives) and an E4M3 scale per 16 dims; an element is code * scale times the pool's k_scale or v_scale. A page of
``page`` tokens is uint8 [page * d / 2] of codes, token after token, the lower half of a byte first, then uint8
[page * d / 16] of scales; K and V are uint8 [n_pages, page, d * 9 / 16]. A group x of 16 dims is stored as

    s = e4m3(max|x| * (1 / (6 scale))),  codes e2m1(x * ((1 / scale) / s)),  all codes 0 where s is 0,

each step one fp32 operation (1 / (6 scale) and 1 / scale are rounded once), rounded to nearest, ties to the even code,
saturating at 448 and 6, zero without a sign. Keys are the exact rotated values, rounded once to fp32, before that. So the bytes of a page
are settled by the rule, and are compared as they are.

Pools, page lists and their counts are otherwise those of the 8- and 16-bit caches: table int32 [batch, heads,
max_pages], lens int32 [batch, heads], refs int32 [n_pages] (lists that hold a page; 0 is free).
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "e2m1": torch.uint8}
ESIZE = {"bf16": 2, "e4m3": 1, "e2m1": 9 / 16}  # bytes per element, scales among them


def listed():
    return [
        # One sequence answering token by token over one layer of a half-kept 4096-token cache: latency.
        _attn("attn4-decode-1x8-t2k", batch=1, heads=8, group=4, d=128, page=16, t_lo=1900, t_hi=2048, q_lo=1, q_hi=1),
        # A serving batch's decode step in one layer: prompts of 8K to 32K tokens, half kept.
        _attn("attn4-decode-64x8-t4k-16k", batch=64, heads=8, group=4, d=128, page=32, t_lo=4096, t_hi=16384, q_lo=1,
              q_hi=1),
        # Two whole 131072-token caches of 10 KV heads: few rows over a long axis.
        _attn("attn4-decode-2x10-t128k", batch=2, heads=10, group=4, d=128, page=64, t_lo=120001, t_hi=131072, q_lo=1,
              q_hi=1),
        # A mixed step: some rows decode, some bring up to 512 prompt tokens, sliding window with 64 first tokens.
        _attn("attn4-mixed-8x8-window", batch=8, heads=8, group=4, d=128, page=16, t_lo=6001, t_hi=16384, q_lo=1,
              q_hi=512, window=4096, sinks=64),
        # A chunk of a long prompt over what the cache holds of it.
        _attn("attn4-chunk-2048-t32k", batch=1, heads=8, group=4, d=128, page=64, t_lo=32768, t_hi=32768, q_lo=2048,
              q_hi=2048),
        # One new token of each of 16 sequences with images in their prompts, into a 4-bit cache: latency.
        _rope("rope-axes-decode-16-e2m1", batch=16, heads=8, group=4, d=128, dtype="e2m1", page=16, q_lo=1, q_hi=1,
              rot=128, layout="half", axes=3, dealt=True, pos=131072),
        # Prompt chunks of text and image patches into a 4-bit cache, half of each head rotated, neighbouring pairs.
        _rope("rope-axes-chunks-e2m1-part", batch=7, heads=10, group=4, d=128, dtype="e2m1", page=64, q_lo=1, q_hi=1000,
              rot=64, layout="interleaved", axes=3, dealt=False, pos=1048576),
        # A long prompt with images of one sequence at once, 16-bit cache.
        _rope("rope-axes-prompt-16k", batch=1, heads=8, group=4, d=128, dtype="bf16", page=32, q_lo=16384, q_hi=16384,
              rot=128, layout="half", axes=3, dealt=False, pos=131072),
        # One layer's compressed prompt from the 16-bit cache into fresh 4-bit pages (20% removed).
        _quantize("quantize-fill-1x8-t4k", batch=1, heads=8, d=128, dtype="e2m1", page=16, t_lo=4096, t_hi=4096,
                  ratio=0.2),
        # A ragged batch's 16-bit cache halved into 4-bit pages.
        _quantize("quantize-8x8-t8k-32k", batch=8, heads=8, d=128, dtype="e2m1", page=32, t_lo=8192, t_hi=32768,
                  ratio=0.5),
        # Beams of one sequence after a step: some die, some fork, 4-bit pages.
        _update("update4-beams-8x8", batch=8, heads=8, d=128, page=16, t_lo=900, t_hi=2048, moved=0.9),
        # A ragged batch's 4-bit paged cache halved.
        _compact("compact4-pages-8x8-t8k-32k", batch=8, heads=8, d=128, page=32, t_lo=8192, t_hi=32768, ratio=0.5),
    ]


def _attn(name=None, window=0, sinks=0, **c):
    return _case(name, op="attention", dtype="e2m1", window=window, sinks=sinks, **c)


def _rope(name=None, **c):
    return _case(name, op="rope", **c)


def _quantize(name=None, **c):
    return _case(name, op="quantize", **c)


def _update(name=None, **c):
    return _case(name, op="update", dtype="e2m1", **c)


def _compact(name=None, **c):
    return _case(name, op="compact", dtype="e2m1", **c)


def _case(name, **c):
    return dict(c, name=name) if name else c


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], evenly over its logarithm."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49))))))


def draw(rng):
    """One more case of the ranges that the listed ones stand for."""
    op = rng.choice(["attention", "attention", "attention", "rope", "rope", "quantize", "update", "compact"])
    d = rng.choice([64, 128, 128, 128, 256])
    c = dict(heads=rng.choice([1, 2, 3, 4, 8, 8, 10]), d=d, page=rng.choice([16, 16, 32, 64, 128]))
    if op == "attention":
        kind = rng.choice(["decode", "decode", "mixed", "chunk"])
        c.update(group=rng.choice([1, 2, 3, 4, 4, 5, 7, 8, 16]))
        c.update(batch=_spread(rng, 1, 4 if kind == "chunk" else 64), q_lo=1)
        c["q_hi"] = 1 if kind == "decode" else _spread(rng, 2, 300 if kind == "mixed" else 2048)
        c["t_hi"] = _spread(rng, 64, 131072)
        # no more scores than the largest listed case has, nor more cached elements
        rows = c["batch"] * c["heads"]
        c["t_hi"] = min(c["t_hi"], 64 * 8 * 10240 * 128 // (rows * d),
                        2 ** 29 * 128 // (rows * c["group"] * c["q_hi"] * d))
        c["q_hi"] = min(c["q_hi"], c["t_hi"])
        c["t_lo"] = max(c["q_hi"], _spread(rng, 1, c["t_hi"]))
        c.update(rng.choice([dict(window=0, sinks=0), dict(window=0, sinks=0),
                             dict(window=_spread(rng, 16, 8192), sinks=rng.choice([0, 1, 4, 64, 100]))]))
        return _attn(**c)
    if op == "rope":
        c.update(batch=_spread(rng, 1, 32), group=rng.choice([1, 2, 3, 4, 4, 7, 8]),
                 dtype=rng.choice(["e2m1", "e2m1", "e4m3", "bf16"]), dealt=rng.choice([True, False]))
        c["axes"] = rng.choice([1, 2, 3, 3, 4] if c["dtype"] == "e2m1" else [2, 3, 3, 4])
        c["q_hi"] = max(1, min(_spread(rng, 1, 16384), 16384 * 40 * 128 // (c["batch"] * c["heads"] * (c["group"] + 2) * d)))
        c["q_lo"] = _spread(rng, 1, c["q_hi"])
        c.update(rot=rng.choice([r for r in (16, 32, 48, 64, 96, 128, 256) if r <= d] + [d, d]),
                 layout=rng.choice(["half", "interleaved"]), pos=_spread(rng, 4096, 1048576))
        return _rope(**c)
    c["batch"] = _spread(rng, 1, 512 if op == "update" else 16)
    if op == "update":
        c["moved"] = rng.choice([0.0, 0.1, 0.3, 0.9])
        c["t_hi"] = min(_spread(rng, 1, 16384), 512 * 8 * 2048 * 128 // (c["batch"] * c["heads"] * d))
        c["t_lo"] = _spread(rng, 1, c["t_hi"])
        return _update(**c)
    c["ratio"] = rng.choice([0.2, 0.25, 0.5, 0.75, 0.9])
    c["t_hi"] = min(_spread(rng, 16, 65536), 8 * 8 * 32768 * 128 // (c["batch"] * c["heads"] * d))
    c["t_lo"] = _spread(rng, 1, c["t_hi"])
    return _compact(**c) if op == "compact" else _quantize(dtype=rng.choice(["e2m1", "e2m1", "e4m3"]), **c)


# ------------------------------------------------------------- 4-bit values --

_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _encode(x, scale):
    """x fp32 [..., d] as codes uint8 [..., d / 2] and scales uint8 [..., d / 16]."""
    g = x.unflatten(-1, (-1, 16))
    inv6 = torch.tensor(1.0 / (6.0 * scale), dtype=torch.float64).float().to(x.device)
    inv = torch.tensor(1.0 / scale, dtype=torch.float64).float().to(x.device)
    s8 = (g.abs().amax(-1) * inv6).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = s8.float()[..., None]
    t = torch.where(s == 0, 0.0, g * (inv / s))
    a = t.abs()
    # passed borders between neighbouring values, those of odd codes' lower ends included: ties go to the even code
    c = sum((a > b).to(torch.uint8) if i % 2 == 0 else (a >= b).to(torch.uint8)
            for i, b in enumerate((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)))
    c = (c | (((t < 0) & (c > 0)).to(torch.uint8) << 3)).flatten(-2)  # zero has one code
    return c[..., 0::2] | (c[..., 1::2] << 4), s8.view(torch.uint8)


def _parts(pages, c):
    """Views of a 4-bit pool: codes [n_pages, page, d / 2], scales [n_pages, page, d / 16]."""
    n, p, d = pages.shape[0], c["page"], c["d"]
    flat = pages.view(n, p * d * 9 // 16)
    return flat[:, :p * d // 2].unflatten(1, (p, d // 2)), flat[:, p * d // 2:].unflatten(1, (p, d // 16))


def _decode(codes, scales):
    """fp32 [..., d] of codes uint8 [..., d / 2] and scales uint8 [..., d / 16]."""
    lut = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), device=codes.device)
    both = torch.stack([lut.repeat(16), lut.repeat_interleave(16)], -1)  # of a byte: lower, upper
    x = both[codes.int()].flatten(-2)
    return (x.unflatten(-1, (-1, 16)) * scales.view(torch.float8_e4m3fn).float()[..., None]).flatten(-2)


def _put(pages, where, slot, x, scale, c):
    """Rows x fp32 [..., d] into rows `slot` of the pages `where`."""
    if c["dtype"] == "e2m1":
        for part, bits in zip(_parts(pages, c), _encode(x, scale)):
            part[where, slot] = bits
        return
    if c["dtype"] == "e4m3":
        x = (x * torch.tensor(1.0 / scale, dtype=torch.float64).float().to(x.device)).clamp(-448, 448)
    pages.view(torch.uint8)[where, slot] = x.to(DTYPES[c["dtype"]]).contiguous().view(torch.uint8)


# ------------------------------------------------------------------- inputs --

def _pages(tokens, page):
    return (tokens + page - 1) // page


def _values(g, shape, dtype, sigma):
    """Normal rows with a lognormal magnitude per token, as cached keys show."""
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
    if sigma:
        x *= torch.exp(sigma * torch.randn(shape[:-1] + (1,), generator=g, device="cuda"))
    return x if dtype is None else x.clamp_(-448, 448).to(DTYPES[dtype])


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
    four = c["dtype"] == "e2m1"
    k = torch.empty((n_pages, c["page"], c["d"] * 9 // 16 if four else c["d"]), dtype=DTYPES[c["dtype"]], device="cuda")
    v = torch.empty_like(k)
    step = max(1, 2 ** 26 // (c["page"] * c["d"]))
    for i in range(0, n_pages, step):
        m = min(step, n_pages - i)
        for x, sigma in ((k, 0.5), (v, 0.0)):
            rows = _values(g, (m, c["page"], c["d"]), None if four else c["dtype"], sigma)
            if four:
                for part, bits in zip(_parts(x[i:i + m], c), _encode(rows, 1.0)):
                    part.copy_(bits)
            else:
                x[i:i + m] = rows
    return k, v


def _poison(c, k, v, table, lens):
    """Rows behind each list's last token hold whatever was there: NaN scales here."""
    tail = lens.flatten().long() % c["page"]
    last = table.flatten(0, 1).gather(1, (_pages(lens.flatten().long(), c["page"]) - 1).clamp(min=0)[:, None])[:, 0].long()
    rows = torch.arange(c["page"], device="cuda")
    hit = (rows[None] >= tail[:, None]) & (tail[:, None] > 0)
    page, row = last[:, None].expand(hit.shape)[hit], rows[None].expand(hit.shape)[hit]
    for x in (k, v):
        codes, scales = _parts(x, c)
        codes[page, row], scales[page, row] = 0xFF, 0x7F


def _f32(x):
    """A host value as the 32-bit number that a call gets."""
    return float(torch.tensor(x, dtype=torch.float64).float())


def _draw_len(g, lo, hi, shape):
    """Numbers of [lo, hi]: the range and the shape settle which ones, the seed their order, so that every seed's tensors
    have the same sizes."""
    n = math.prod(shape)
    same = torch.Generator()
    same.manual_seed(1000003 * lo + 101 * hi + n)
    x = torch.randint(lo, hi + 1, (n,), generator=same).cuda()
    return x[torch.randperm(n, generator=g, device="cuda")].view(shape)


def _sections(c):
    """Pairs of each axis: the first axis (text and time) gets what is left."""
    pairs, n = c["rot"] // 2, c["axes"]
    rest = [(3 * pairs // 8) * 2 // n if n > 1 else 0] * (n - 1)
    return [pairs - sum(rest)] + rest


def _axis_of_pairs(c):
    """int32 [rot / 2]: the axis whose position turns each pair. In runs, or dealt out in turn while an axis has pairs."""
    axis = torch.repeat_interleave(torch.arange(c["axes"]), torch.tensor(_sections(c)))
    if c["dealt"]:
        nth = torch.cat([torch.arange(m) for m in _sections(c)])
        axis = axis[torch.argsort(nth * c["axes"] + axis)]
    return axis.to(torch.int32)


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
        s["k_scale"], s["v_scale"] = 0.75, 1.25
    elif c["op"] == "rope":
        old = _draw_len(g, 0, 200, (B, H))
        lens = old + n_q[:, None]
        s["table"], s["lens"], refs = _lists(g, c, lens, _pages(c["q_hi"] + 200, c["page"]), None)
        s["k_pages"], s["v_pages"] = _pool(g, c, refs.numel())
        # the three projections of one fused product: rows of (hq + 2 H) heads
        qkv = _values(g, (n, hq + 2 * H, c["d"]), "bf16", 0.3)
        s["Q"], s["K"], s["V"] = qkv[:, :hq], qkv[:, hq:hq + H], qkv[:, hq + H:]
        first = _draw_len(g, 0, max(0, c["pos"] - c["q_hi"] - 64), (B,))
        row = torch.repeat_interleave(torch.arange(B, device="cuda"), n_q)
        i = torch.arange(n, device="cuda") - s["q_start"].long()[row]
        # runs of 256 text tokens (one place on every axis) and images of 16 x 16 patches (one time, rows, columns, ...)
        run, at = i // 256, i % 256
        places = torch.stack([torch.where(run % 2 == 0, i, run * 256 + (0 if k == 0 else at // 16 if k == 1 else at % 16 // (k - 1)))
                              for k in range(c["axes"])])
        s["positions"] = (first[row] + places).to(torch.int32).contiguous()
        s["axes"] = _axis_of_pairs(c).cuda()
        i = torch.arange(c["rot"] // 2, device="cuda", dtype=torch.float64)
        s["inv_freq"] = (500000.0 ** (-2.0 * i / c["rot"])).float()
        s["factor"] = 1.0 if c["pos"] <= 131072 else _f32(0.1 * math.log(c["pos"] / 131072) + 1.0)
        s["k_scale"], s["v_scale"] = {"bf16": (1.0, 1.0), "e4m3": (0.0625, 0.03125), "e2m1": (_f32(0.011), 0.0625)}[c["dtype"]]
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
        stride = int(math.floor(c["t_hi"] * (1 - c["ratio"]) + 0.5))
        # kept tokens ascending: the tokens of the `kept` largest of T random scores
        score = torch.rand((B, H, c["t_hi"]), generator=g, device="cuda")
        score[torch.arange(c["t_hi"], device="cuda") >= T[..., None]] = -1
        order = score.argsort(-1, descending=True)[..., :max(1, stride)]
        slot = torch.arange(order.shape[-1], device="cuda")
        order = torch.where(slot < kept[..., None], order, 2 ** 30).sort(-1).values
        s["idx"] = torch.where(slot < kept[..., None], order, -7).to(torch.int32).contiguous()
        s["kept"] = kept.to(torch.int32)
        spare = int(_pages(kept, c["page"]).sum()) + 3
        lens = T if c["op"] == "compact" else torch.zeros_like(T)
        s["table"], s["lens"], s["refs"] = _lists(g, c, lens, _pages(c["t_hi"], c["page"]), spare)
        s["k_pages"], s["v_pages"] = _pool(g, c, s["refs"].numel())
        if c["op"] == "quantize":
            s["K"] = _values(g, (B, H, c["t_hi"], c["d"]), "bf16", 0.5)
            s["V"] = _values(g, (B, H, c["t_hi"], c["d"]), "bf16", 0.0)
            s["seq_lens"] = T[:, 0].to(torch.int32).contiguous()
            s["k_scale"], s["v_scale"] = 0.0625, _f32(0.03)
    if c["op"] not in ("attention", "rope"):
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
            if c["axes"] == 1:
                mkv.mkv_rope_append(s["Q"], s["K"], s["V"], s["positions"][0], s["inv_freq"], s["k_pages"], s["v_pages"],
                                    s["table"], s["lens"], s["q_start"], s["Q_out"], s["ws"], layout=c["layout"],
                                    factor=s["factor"], k_scale=s["k_scale"], v_scale=s["v_scale"])
            else:
                mkv.mkv_rope_append_axes(s["Q"], s["K"], s["V"], s["positions"], s["axes"], s["inv_freq"], s["k_pages"],
                                         s["v_pages"], s["table"], s["lens"], s["q_start"], s["Q_out"], s["ws"],
                                         layout=c["layout"], factor=s["factor"], k_scale=s["k_scale"],
                                         v_scale=s["v_scale"])
            return {"Q": s["Q_out"], "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
        if c["op"] == "update":
            mkv.mkv_page_update(s["k_pages"], s["v_pages"], s["table"], s["lens"], s["refs"], s["table_out"],
                                s["lens_out"], s["refs_out"], s["ws"], parent=s["parent"], n_new=s["n_new"])
        elif c["op"] == "compact":
            mkv.mkv_page_compact(s["k_pages"], s["v_pages"], s["table"], s["lens"], s["refs"], s["idx"], s["kept"],
                                 s["table_out"], s["lens_out"], s["refs_out"], s["ws"])
        else:
            mkv.mkv_page_quantize(s["k_pages"], s["v_pages"], s["table"], s["lens"], s["refs"], s["idx"], s["kept"],
                                  s["K"], s["V"], s["table_out"], s["lens_out"], s["refs_out"], s["ws"],
                                  k_scale=s["k_scale"], v_scale=s["v_scale"], seq_lens=s["seq_lens"])
        return {k: s[k] for k in ("table_out", "lens_out", "refs_out", "k_pages", "v_pages")}
    return {"attention": _plain_attention, "rope": _plain_rope, "update": _plain_update, "compact": _plain_compact,
            "quantize": _plain_compact}[c["op"]](s, c)


def _plain_attention(s, c):
    B, H, G, D, page = c["batch"], c["heads"], c["group"], c["d"], c["page"]
    dev = s["Q"].device
    slot = torch.arange(s["max_len"], device=dev)
    lens = s["lens"].long().view(B, H, 1)
    live = slot < lens
    pages = s["table"].long().view(B, H, -1)[:, :, slot // page].clamp(min=0)
    k, v = (_decode(*(part[pages, slot % page] for part in _parts(s[x], c))) for x in ("k_pages", "v_pages"))
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
    """x [n, heads, d], the first `rot` dims rotated by the angles of cos and sin [n, rot / 2]."""
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
    # 64 bits: far positions' angles, and rotated keys next to the border of two codes
    a = s["positions"].double()[s["axes"].long()].T * s["inv_freq"].double()
    # the factor multiplies the rotated part alone
    cos, sin = a.cos() * s["factor"], a.sin() * s["factor"]
    s["Q_out"].copy_(_rotate(s["Q"].float(), cos.float(), sin.float(), c))
    start, lens = s["q_start"].long(), s["lens"].long()
    t = torch.arange(s["Q"].shape[0], device=a.device)
    b = torch.searchsorted(start[1:], t, right=True)
    slot = lens[b] - (start[b + 1] - t)[:, None]  # [n, H]
    h = torch.arange(c["heads"], device=a.device)
    pages = s["table"].long()[b[:, None], h, slot // c["page"]]
    _put(s["k_pages"], pages, slot % c["page"], _rotate(s["K"].double(), cos, sin, c).float(), s["k_scale"], c)
    _put(s["v_pages"], pages, slot % c["page"], s["V"].float(), s["v_scale"], c)
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
    for x in (*_parts(s["k_pages"], c), *_parts(s["v_pages"], c)):
        x[dst] = torch.where(real, x[src], x[dst])
    return {k: s[k] for k in ("table_out", "lens_out", "refs_out", "k_pages", "v_pages")}


def _plain_compact(s, c):
    """Kept tokens into new pages: of 4-bit pages their codes and scales as they are, of a 16-bit cache rounded."""
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
    src = torch.where(real, s["idx"].long(), 0)[real]
    to, row = out.gather(-1, (i // page).expand(B, H, -1))[real], (i % page).expand(B, H, -1)[real]
    if c["op"] == "quantize":
        b, h = torch.nonzero(real, as_tuple=True)[:2]
        for x, cache, scale in ((s["k_pages"], s["K"], s["k_scale"]), (s["v_pages"], s["V"], s["v_scale"])):
            _put(x, to, row, cache[b, h, src].float(), scale, c)
    else:
        at = table.gather(-1, torch.where(real, s["idx"].long(), 0) // page)[real]
        for x in (*_parts(s["k_pages"], c), *_parts(s["v_pages"], c)):
            x[to, row] = x[at, src % page]
    return {k: s[k] for k in ("table_out", "lens_out", "refs_out", "k_pages", "v_pages")}


# ------------------------------------------------------------------- work --

def work(case):
    """Mean bytes and operations of one pass over the case's ranges."""
    c = case
    row = c["d"] * ESIZE[c["dtype"]]
    lists = c["batch"] * c["heads"]
    if c["op"] in ("attention", "rope"):
        q = (c["q_lo"] + c["q_hi"]) / 2
        if c["q_hi"] > 1 and c["q_lo"] == 1 and c["batch"] > 2:
            q = (2 * q + 1) / 3
    if c["op"] == "attention":
        t = max((max(c["t_lo"], q) + c["t_hi"]) / 2, q)
        seen = read = t
        if c["window"] and c["window"] + q + c["sinks"] < t:
            seen, read = c["window"] + c["sinks"], c["window"] + q + c["sinks"]
        else:
            seen = t - q / 2
        io = c["batch"] * q * c["heads"] * c["group"] * (c["d"] * 4 + 4)
        return {"bytes": lists * read * 2 * row + io, "flops": 4.0 * c["d"] * lists * c["group"] * q * seen}
    if c["op"] == "rope":
        n = c["batch"] * q
        return {"bytes": n * (c["heads"] * (c["group"] * c["d"] * 4 + 2 * (c["d"] * 2 + row)) + 4 * c["axes"]),
                "flops": n * c["heads"] * (c["group"] + 1) * c["rot"] * 3.0}
    t = (c["t_lo"] + c["t_hi"]) / 2
    held = lists * _pages(t, c["page"])
    if c["op"] == "update":
        pool = held + lists * (2 + _pages(40, c["page"]))
        copied = lists * c["moved"] * 0.6 * c["page"] / 2
        return {"bytes": 8 * held + 8 * pool + 8 * lists + copied * 4 * row, "flops": 0}
    n = lists * t * (1 - c["ratio"])
    if c["op"] == "compact":
        return {"bytes": n * (4 * row + 4) + 16 * held, "flops": 0}
    return {"bytes": n * (2 * (row + 2 * c["d"]) + 4) + 8 * held, "flops": n * c["d"] * 4.0}


# ------------------------------------------------------------------ 64 bits --

def _stored(x, ids, page, d):
    """The rows of a list's pages in 64 bits, from the definition of the codes."""
    flat = x[ids].flatten(1).int()
    codes, scales = flat[:, :page * d // 2].reshape(-1, d // 2), flat[:, page * d // 2:].reshape(-1, d // 16)
    nib = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).double()
    sign, e, m = 1 - 2 * (nib // 8), nib % 8 // 2, nib % 2
    val = sign * torch.where(e == 0, m / 2, (1 + m / 2) * 2 ** (e - 1))
    f, t = (scales // 8 % 16).double(), (scales % 8).double()
    s = torch.where(f == 0, t / 8 * 2.0 ** -6, (1 + t / 8) * 2 ** (f - 7))
    return val * s.repeat_interleave(16, -1)


def exact(case, seed):
    """Attention, rotation and 8-bit rounding (of the values before it) from their definitions in 64 bits; the moves
    return no computed numbers, and the bytes of 4-bit pages are whole numbers."""
    c = case
    if c["op"] not in ("attention", "rope") and (c["op"] != "quantize" or c["dtype"] != "e4m3"):
        return None
    s = prepare(case, seed)
    page = c["page"]
    if c["op"] == "quantize":
        free = [i for i, n in enumerate(s["refs"].tolist()) if n == 0]
        kp, vp = s["k_pages"].double().flatten(0, 1), s["v_pages"].double().flatten(0, 1)
        for b in range(c["batch"]):
            for j in range(c["heads"]):
                ids = s["idx"][b, j, :int(s["kept"][b, j])].long()
                mine, free = free[:-(-len(ids) // page)], free[-(-len(ids) // page):]
                rows = (torch.tensor(mine, dtype=torch.int64)[:, None] * page + torch.arange(page)).flatten()[:len(ids)].cuda()
                kp[rows] = (s["K"][b, j, ids].double() / s["k_scale"]).clamp(-448, 448)
                vp[rows] = (s["V"][b, j, ids].double() / s["v_scale"]).clamp(-448, 448)
        return {"table_out": None, "lens_out": None, "refs_out": None, "k_pages": kp.view(s["k_pages"].shape),
                "v_pages": vp.view(s["v_pages"].shape)}
    start, lens, table = s["q_start"].tolist(), s["lens"].tolist(), s["table"]
    if c["op"] == "attention":
        O = torch.zeros(s["Q"].shape, dtype=torch.float64, device="cuda")
        lse = torch.full(s["Q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
        for b in range(c["batch"]):
            n = start[b + 1] - start[b]
            for j in range(c["heads"]):
                L = lens[b][j]
                ids = table[b, j, :_pages(L, page)].long()
                K, V = (_stored(s[x], ids, page, c["d"])[:L] * s[y] for x, y in (("k_pages", "k_scale"), ("v_pages", "v_scale")))
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
    i = torch.arange(c["rot"] // 2, device="cuda")
    lo, hi = (i, i + c["rot"] // 2) if c["layout"] == "half" else (2 * i, 2 * i + 1)
    place = torch.stack([s["positions"][a] for a in s["axes"].tolist()], 1).double()
    angle = place * s["inv_freq"].double()
    turn = torch.polar(torch.full_like(angle, s["factor"]), angle)[:, None]

    def turned(x):
        y = x.double().clone()
        z = torch.complex(y[..., lo], y[..., hi]) * turn
        y[..., lo], y[..., hi] = z.real, z.imag
        return y

    if c["dtype"] == "e2m1":
        return {"Q": turned(s["Q"]), "k_pages": None, "v_pages": None}
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
