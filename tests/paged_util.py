"""Plain references of the paged-cache calls in 64 bits (torch on the CPU and Python integers), and random page
lists for their tests. Written from the definitions in include/mkv.h; no code of the library is used."""
import math
import random

import torch

CODES = {torch.bfloat16: torch.int16, torch.float8_e4m3fn: torch.uint8}


def pages_of(n, page):
    return -(-n // page)


def raw(x):
    """The bits of a cache tensor."""
    return x.view(CODES[x.dtype])


def random_lists(rng, lens, page, n_pages, max_pages):
    """Page lists of the given lengths (nested lists [batch][heads]) over shuffled pages: table, lens, refs tensors.
    Unused table entries hold a page number far outside every pool: they may not be read."""
    ids = list(range(n_pages))
    rng.shuffle(ids)
    B, H = len(lens), len(lens[0]) if lens else 0
    table = torch.full((B, H, max_pages), 2 ** 30, dtype=torch.int32)
    refs = torch.zeros(n_pages, dtype=torch.int32)
    for b in range(B):
        for j in range(H):
            for p in range(pages_of(lens[b][j], page)):
                i = ids.pop()
                table[b, j, p] = i
                refs[i] += 1
    return table, torch.tensor(lens, dtype=torch.int32).view(B, H), refs


def random_pool(seed, n_pages, page, d, dtype, sigma=0.5):
    g = torch.Generator().manual_seed(seed)
    k = torch.randn((n_pages, page, d), generator=g) * torch.exp(sigma * torch.randn((n_pages, page, 1), generator=g))
    v = torch.randn((n_pages, page, d), generator=g)
    return k.clamp(-440, 440).to(dtype), v.clamp(-440, 440).to(dtype)


def poison_unused(k, v, table, lens, page):
    """NaN (all ones) in every row that no list reaches."""
    used = torch.zeros(k.shape[:2], dtype=torch.bool)
    for b in range(lens.shape[0]):
        for j in range(lens.shape[1]):
            for s in range(int(lens[b, j])):
                used[int(table[b, j, s // page]), s % page] = True
    for x in (k, v):
        raw(x)[~used] = -1 if x.dtype == torch.bfloat16 else 255


def rows_of(pool, table, n, page):
    """The first n tokens of one list, fp64."""
    ids = table[:pages_of(n, page)].long()
    return raw(pool)[ids].reshape(-1, pool.shape[-1])[:n].view(pool.dtype).double()


def attention(Q, k, v, table, lens, q_start, page, scale, k_scale=1.0, v_scale=1.0, window=0, sinks=0):
    """O, lse, and per output element A = sum of weights times |v| and per row E, the largest sum of |scale q_i k_i|
    over the visible keys, and W = sum |v| / l: what the bounds are made of."""
    n_tok, hq, d = Q.shape
    H = lens.shape[1]
    G = hq // H
    O = torch.zeros((n_tok, hq, d), dtype=torch.float64)
    lse = torch.full((n_tok, hq), -math.inf, dtype=torch.float64)
    A, W, E = torch.zeros_like(O), torch.zeros_like(O), torch.zeros((n_tok, hq), dtype=torch.float64)
    for b in range(lens.shape[0]):
        t0, t1 = int(q_start[b]), int(q_start[b + 1])
        for j in range(H):
            L = int(lens[b, j])
            K, V = rows_of(k, table[b, j], L, page) * k_scale, rows_of(v, table[b, j], L, page) * v_scale
            for t in range(t0, t1):
                p = L - (t1 - t)
                keys = [s for s in range(max(0, min(p + 1, L))) if window == 0 or s > p - window or s < sinks]
                if not keys:
                    continue
                Ks, Vs = K[keys], V[keys]
                for h in range(j * G, (j + 1) * G):
                    q = Q[t, h].double()
                    x = scale * (Ks @ q)
                    m = x.max()
                    w = torch.exp(x - m)
                    l = w.sum()
                    O[t, h], A[t, h], W[t, h] = (w @ Vs) / l, (w @ Vs.abs()) / l, Vs.abs().sum(0) / l
                    lse[t, h] = m + torch.log(l)
                    E[t, h] = (abs(scale) * (Ks.abs() @ q.abs())).max()
    return O, lse, A, W, E


def attention_bounds(O, lse, A, W, E, d, dtype):
    """Elementwise bounds of |O - exact| and |lse - exact|.

    A score is a sum of d products of exact factors in fp32: off by at most d 2^-24 E, doubled for the tensor cores'
    truncation of aligned addends; scaling to log2 units and the differences to the maximum round four times more on
    numbers up to 2 E log2(e); 2^x is off by 2^-22 relative and the running factors multiply it a few times over. So a
    weight is off by eps = 2 d 2^-24 E + 16 2^-24 E + 2^-18 relative, and so is the sum l. A weight is then rounded to 16
    bits: half a step, 2^-8 (bf16) or 2^-11 (fp16, next to E4M3 values; below 2^-14 half a step is 2^-25 absolute).
    (Queries next to E4M3 keys run as fp16 scaled to a largest element of 1 to 2: an element is off by at most 2^-25 of the
    largest, a score by 2^-25 max|q| sum|scale k|, which for the normal queries here, max|q| < 10 mean|q|, is below a
    twentieth of the 2 d 2^-24 E.) The
    sum's fp32 error adds at most (keys / 8) 2^-24, inside the 2^-18 for the sizes here. The output is rounded to bf16:
    2^-8 relative to what is rounded."""
    eps = (2 * d + 16) * 2.0 ** -24 * E + 2.0 ** -18
    half = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -11
    tiny = 0.0 if dtype == torch.bfloat16 else 2.0 ** -25
    err = (2 * eps[..., None] + half) * A * (1 + 2.0 ** -6) + tiny * W
    return err * (1 + 2.0 ** -8) + 2.0 ** -8 * O.abs() + 1e-30, eps + 2.0 ** -22 * lse.abs().nan_to_num(0, 0, 0) + 2.0 ** -20


def rotate(x, positions, inv_freq, rot, layout, factor):
    """x [n, heads, d] in fp64."""
    y = x.double().clone()
    a = (positions.double()[:, None] * inv_freq.double())[:, None]
    i = torch.arange(rot // 2)
    lo, hi = (i, i + rot // 2) if layout == "half" else (2 * i, 2 * i + 1)
    p, q = x.double()[..., lo], x.double()[..., hi]
    y[..., lo], y[..., hi] = factor * (p * a.cos() - q * a.sin()), factor * (p * a.sin() + q * a.cos())
    return y


def page_update(k, v, table, lens, refs, parent, n_new, page):
    """In Python integers; returns table_out (unused entries as in `table`), lens_out, refs_out, k, v."""
    B, H, M = table.shape
    parent = list(range(B)) if parent is None else [int(x) for x in parent]
    n_new = [0] * B if n_new is None else [int(x) for x in n_new]
    free = [p for p in range(refs.numel()) if int(refs[p]) == 0]
    out, lens_out, refs_out, k, v = table.clone(), lens.clone(), refs.clone(), k.clone(), v.clone()
    keeper = {}
    for a in set(parent) - {-1}:
        keeper[a] = a if parent[a] == a else min(b for b in range(B) if parent[b] == a)
    held_before = [[table[b, j, :pages_of(int(lens[b, j]), page)].tolist() for j in range(H)] for b in range(B)]
    at = 0
    new_lists = {}
    copies = []
    for b in range(B):
        for j in range(H):
            a = parent[b]
            if a < 0:
                new_lists[b, j] = ([], 0)
                continue
            L = int(lens[a, j])
            shared = held_before[a][j] if keeper[a] == b else held_before[a][j][:L // page]
            total = pages_of(L + n_new[b], page)
            fresh = free[at:at + total - len(shared)]
            at += total - len(shared)
            assert len(fresh) == total - len(shared), "the test's pool is too small"
            if keeper[a] != b and L % page:
                copies.append((held_before[a][j][L // page], fresh[0], L % page))
            new_lists[b, j] = (shared + fresh, L + n_new[b])
    for s, e, n in copies:
        for x in (k, v):
            raw(x)[e, :n] = raw(x)[s, :n]
    for b in range(B):
        for j in range(H):
            pages, n = new_lists[b, j]
            out[b, j, :len(pages)] = torch.tensor(pages, dtype=torch.int32)
            lens_out[b, j] = n
            for p in pages:
                refs_out[p] += 1
            for p in held_before[b][j]:
                refs_out[p] -= 1
    return out, lens_out, refs_out, k, v


def page_compact(k, v, table, lens, refs, idx, kept, page, K=None, V=None):
    B, H, M = table.shape
    free = [p for p in range(refs.numel()) if int(refs[p]) == 0]
    out, lens_out, refs_out = table.clone(), kept.clone(), refs.clone()
    k0, v0, k, v = k, v, k.clone(), v.clone()
    at = 0
    for b in range(B):
        for j in range(H):
            n = int(kept[b, j])
            fresh = free[at:at + pages_of(n, page)]
            at += len(fresh)
            assert len(fresh) == pages_of(n, page), "the test's pool is too small"
            for i in range(n):
                s = i if idx is None else int(idx[b, j, i])
                for src, cache, dst in ((k0, K, k), (v0, V, v)):
                    row = raw(src)[int(table[b, j, s // page]), s % page] if cache is None else raw(cache)[b, j, s]
                    raw(dst)[fresh[i // page], i % page] = row
            out[b, j, :len(fresh)] = torch.tensor(fresh, dtype=torch.int32)
            for p in fresh:
                refs_out[p] += 1
            for p in table[b, j, :pages_of(int(lens[b, j]), page)].tolist():
                refs_out[p] -= 1
    return out, lens_out, refs_out, k, v
