"""4-bit pages and several axes where they could go wrong without a sign: pools beyond 4 GB, long segments, many heads,
numbers that are not finite, queries in place, two calls at once."""
import math
import random

import pytest
import torch

import e2m1_util as eu
import geometric_kv_cache_gb300 as mkv
import paged_util as pu
from test_gpu_paged_rope import _close
from test_gpu_rope_axes import Step

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F8, U8 = torch.bfloat16, torch.float8_e4m3fn, torch.uint8


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mkv.load()
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _decoded(pages, table, L):
    """A list's first L tokens in fp64, on the GPU."""
    n, page, b = pages.shape
    d, flat = b * 16 // 9, pages.view(n, page * b)[table.long()]
    codes = flat[:, :page * d // 2].reshape(-1, d // 2)[:L].int()
    scales = flat[:, page * d // 2:].reshape(-1, d // 16)[:L]
    values = torch.tensor(list(eu.E2M1) + [-x for x in eu.E2M1], dtype=torch.float64, device=DEV)
    x = torch.stack([values[codes & 15], values[codes >> 4]], -1).flatten(-2)
    return x * scales.view(F8).double().repeat_interleave(16, -1)


@pytest.mark.parametrize("d,page,G", [(64, 16, 1), (128, 64, 4), (128, 16, 12), (256, 32, 2)])
def test_segments_of_many_steps(d, page, G):
    # 170 lists whose CTAs have whole tiles: a CTA walks far more blocks of keys than it looks pages up for at once
    B, L0 = 85, 9000 if d < 256 else 7000
    g = torch.Generator(device=DEV).manual_seed(d + G)
    lens = L0 + torch.randint(0, 700, (B, 2), generator=g, device=DEV).to(torch.int32)
    M = pu.pages_of(L0 + 700, page)
    perm = torch.randperm(2 * B * M, generator=g, device=DEV).to(torch.int32)
    table = perm.view(B, 2, M).contiguous()
    k, v = (torch.randint(0, 256, (2 * B * M, page, d * 9 // 16), generator=g, device=DEV, dtype=U8) for _ in range(2))
    for x in (k, v):  # scales below 2
        x.view(-1, page * d * 9 // 16)[:, page * d // 2:].bitwise_and_(0x3F)
    Q = torch.randn((B, 2 * G, d), generator=g, device=DEV).to(BF)
    O, lse = torch.empty_like(Q), torch.empty((B, 2 * G), device=DEV)
    start = torch.arange(B + 1, dtype=torch.int32, device=DEV)
    ws = mkv.attention_workspace_for(Q, k, table, 1, M * page)
    mkv.mkv_paged_attention(Q, k, v, table, lens, start, 1, M * page, O, ws, k_scale=0.05, v_scale=0.5, lse=lse)
    assert mkv.mkv_device_status(ws) == 0
    for b in random.Random(1).sample(range(B), 12):
        for j in range(2):
            L, h = int(lens[b, j]), slice(j * G, (j + 1) * G)
            K, V = _decoded(k, table[b, j], L) * 0.05, _decoded(v, table[b, j], L) * 0.5
            q = Q[b, h].double()
            x = q @ K.T * d ** -0.5
            m = x.amax(-1, keepdim=True)
            w = torch.exp(x - m)
            l = w.sum(-1, keepdim=True)
            E = (q.abs() @ K.abs().T * d ** -0.5).amax(-1)
            args = (w @ V / l, (m + l.log())[..., 0], w @ V.abs() / l, V.abs().sum(0) / l, E)
            tol, tol_lse = pu.attention_bounds(*(y.cpu() for y in args), d, F8)
            # (the bound's 2^-18 holds 64 roundings of the sum l: a lane adds up at most 26 steps of four weights here)
            assert ((O[b, h].double() - args[0]).abs().cpu() <= tol).all()
            assert ((lse[b, h].double() - args[1]).abs().cpu() <= tol_lse).all()


@pytest.mark.parametrize("rows", [2, 80])
def test_pools_beyond_4_gb(rows):
    """The same calls in a small pool and in one whose only free pages lie beyond 2^32 bytes: the same bits."""
    d, page, H, G = 128, 128, 2, 4 if rows == 2 else 16
    big = 2 ** 32 // (page * 72) + 40
    K, V = (torch.randn((1, H, 700, d), device=DEV).to(BF) for _ in range(2))
    qkv = torch.randn((rows, H * (G + 2), d), device=DEV).to(BF)
    pos = torch.randint(0, 10 ** 6, (3, rows), device=DEV).to(torch.int32)
    axes, freq = mkv.mkv_rope_axes([32, 16, 16]).to(DEV), mkv.mkv_rope_frequencies(d, 10000.0).to(DEV)
    results = []
    for n_pages in (40, big):
        k, v = (torch.zeros((n_pages, page, 72), dtype=U8, device=DEV) for _ in range(2))
        refs = torch.ones(n_pages, dtype=torch.int32, device=DEV)
        refs[-40:] = 0
        z = lambda *s: torch.zeros(s, dtype=torch.int32, device=DEV)  # noqa: E731
        bufs = [(z(1, H, 8), z(1, H)) for _ in range(3)]
        ws = mkv.page_workspace_for(k, bufs[0][0])
        mkv.mkv_page_quantize(k, v, *bufs[0], refs, None, _i32([[700, 333]]), K, V, *bufs[1], refs, ws, 0.1, 0.2)
        keep = torch.arange(0, 700, 2, device=DEV).to(torch.int32).expand(1, H, 350).contiguous()
        mkv.mkv_page_compact(k, v, *bufs[1], refs, keep, _i32([[350, 160]]), *bufs[2], refs, ws)
        table, lens = bufs[2]
        mkv.mkv_page_update(k, v, table, lens, refs, table, lens, refs, ws, n_new=_i32([rows]))
        start, Q = _i32([0, rows]), torch.empty((rows, H * G, d), dtype=BF, device=DEV)
        hq = H * G
        mkv.mkv_rope_append_axes(qkv[:, :hq], qkv[:, hq:hq + H], qkv[:, hq + H:], pos, axes, freq, k, v, table, lens, start,
                                 Q, ws, k_scale=0.1, v_scale=0.2)
        O, lse = torch.empty_like(Q), torch.empty((rows, hq), device=DEV)
        wa = mkv.attention_workspace_for(Q, k, table, rows, 8 * page)
        mkv.mkv_paged_attention(Q, k, v, table, lens, start, rows, 8 * page, O, wa, k_scale=0.1, v_scale=0.2, lse=lse)
        assert mkv.mkv_device_status(ws) == 0 and mkv.mkv_device_status(wa) == 0
        assert int(table[0, 0, 0]) >= n_pages - 40
        ids = torch.arange(n_pages - 40, n_pages, device=DEV)
        results.append((Q.cpu(), O.cpu(), lse.cpu(), k[ids].cpu(), v[ids].cpu(), lens.cpu()))
        del k, v
        torch.cuda.empty_cache()
    for a, b in zip(*results):
        assert torch.equal(a.view(U8) if a.dtype == BF else a, b.view(U8) if b.dtype == BF else b)
    assert torch.isfinite(results[0][2]).all() and results[0][5].tolist() == [[350 + rows, 160 + rows]]


@pytest.mark.parametrize("dtype", [BF, F8, U8])
@pytest.mark.parametrize("d,H,n", [(64, 40, 3), (128, 70, 2), (256, 33, 200), (64, 64, 1500)])
def test_more_than_32_heads_of_keys(dtype, d, H, n):
    p = Step(H, [n, 1] if n < 1000 else [n], H, 1, d, 16, dtype, 2, pad_back=1)
    inv_freq, axes = mkv.mkv_rope_frequencies(d, 10000.0), mkv.mkv_rope_axes([d // 4, d // 4], True)
    scales = {BF: (1.0, 1.0), F8: (0.02, 0.3), U8: (0.013, 0.3)}[dtype]
    if n >= 1000:  # (a warp per token: its own heads of all kinds)
        p.qkv = p.qkv.clone()
        p.table[0, H - 1, :] = p.k.shape[0]  # one list's pages are not there
        res = p.run(inv_freq, axes, "half", 1.0, scales)
        assert p.status == mkv.MKV_DEV_BAD_PAGE
        y, _ = p.rotated(inv_freq, axes, "half", 1.0)
        if dtype is U8:
            got = eu.rows_of(res[1]).view(U8)
            for j in (0, 31, 32, H - 2):
                t = torch.arange(n)
                s = p.lens[0, j] - n + t
                want = torch.cat(eu.encode(y[:n, H + j].float(), scales[0]), -1)
                assert torch.equal(got[p.table[0, j, s // 16].long(), s % 16], want)
        return
    res = p.run(inv_freq, axes, "half", 1.0, scales)
    assert p.status == 0
    p.check(res, inv_freq, axes, "half", 1.0, scales)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_new_keys_and_values_that_are_not_finite(layout):
    p = Step(4, [20, 3], 2, 2, 128, 16, U8)
    x = p.qkv.clone()
    p.qkv[2, 4, 70] = math.nan      # a key
    p.qkv[5, 5, 3] = math.inf
    p.qkv[7, 6, 17] = math.nan      # a value
    p.qkv[8, 7, 127] = -math.inf
    inv_freq = mkv.mkv_rope_frequencies(64, 10000.0)
    bad = p.run(inv_freq, None, layout, 1.0, (0.013, 0.3))
    p.qkv = x
    good = p.run(inv_freq, None, layout, 1.0, (0.013, 0.3))
    assert p.status == 0

    def row(pages, b, j, t):
        s = int(p.lens[b, j]) - (int(p.start[b + 1]) - t)
        c, sc = (y[int(p.table[b, j, s // 16]), s % 16][None] for y in eu.from_pages(pages))
        return eu.decode(c.contiguous(), sc.contiguous())[0]

    for t in range(23):
        b = 0 if t < 20 else 1
        for j in range(2):
            for i, kv in enumerate(("k", "v")):
                got, want = row(bad[1 + i], b, j, t), row(good[1 + i], b, j, t)
                if (t, kv, j) == (2, "k", 0):    # dims 64 and on do not turn
                    assert got[64:80].isnan().all() and torch.equal(got[:64], want[:64]) and torch.equal(got[80:], want[80:])
                elif (t, kv, j) == (7, "v", 0):
                    assert got[16:32].isnan().all() and int(got.isnan().sum()) == 16
                elif (t, kv, j) == (8, "v", 1):
                    assert float(got[127]) == -6 * 448 and torch.equal(got[:112], want[:112])
                elif (t, kv, j) == (5, "k", 1):  # its pair's groups saturate or are NaN, the others are as they were
                    partner = 35 if layout == "half" else 2
                    hit = {3 // 16, partner // 16}
                    for g in range(8):
                        assert g in hit or torch.equal(got[16 * g:16 * g + 16], want[16 * g:16 * g + 16])
                else:
                    assert torch.equal(got, want), (t, j, kv)


@pytest.mark.parametrize("dtype", [BF, U8])
def test_queries_in_place(dtype):
    p = Step(6, [3, 200], 2, 4, 128, 16, dtype, 3)
    inv_freq, axes = mkv.mkv_rope_frequencies(128, 10000.0), mkv.mkv_rope_axes([32, 16, 16], True)
    scales = (1.0, 1.0) if dtype is BF else (0.013, 0.3)
    apart = p.run(inv_freq, axes, "half", 1.0, scales)
    k, v, qkv, pos, table, lens, start = (x.to(DEV) for x in (p.k, p.v, p.qkv, p.positions, p.table, p.lens, p.start))
    Q, ws = qkv[:, :8].contiguous(), mkv.page_workspace_for(k, table)
    mkv.mkv_rope_append_axes(Q, qkv[:, 8:10], qkv[:, 10:], pos, axes.to(DEV), inv_freq.to(DEV), k, v, table, lens, start, Q, ws,
                             k_scale=scales[0], v_scale=scales[1])
    assert mkv.mkv_device_status(ws) == 0
    assert torch.equal(Q.cpu().view(U8), apart[0].view(U8)) and torch.equal(k.cpu().view(U8), apart[1].view(U8))


def test_appended_at_position_zero_and_quantized_are_the_same_bytes():
    # nothing turns at position 0: the two ways into 4-bit pages have to agree on every border
    H, d, n = 3, 128, 64
    g = torch.Generator().manual_seed(2)
    grid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 0.0, -0.0, -0.25, -5.0, 1.1, -0.3])
    K, V = (grid[torch.randint(0, len(grid), (1, H, n, d), generator=g)].to(BF) for _ in range(2))
    Q = torch.zeros((n, H, d), dtype=BF, device=DEV)
    for ks, vs in ((1.0, 1.0), (0.3, 7.0)):
        got = []
        for way in (0, 1):
            k, v = (torch.zeros((20, 16, 72), dtype=U8, device=DEV) for _ in range(2))
            z = lambda *s: torch.zeros(s, dtype=torch.int32, device=DEV)  # noqa: E731
            refs, old, new = z(20), (z(1, H, 4), z(1, H)), (z(1, H, 4), z(1, H))
            ws = mkv.page_workspace_for(k, old[0])
            if way == 0:
                mkv.mkv_page_quantize(k, v, *old, refs, None, _i32([[n] * H]), K.to(DEV), V.to(DEV), *new, refs, ws, ks, vs)
            else:
                mkv.mkv_page_update(k, v, *old, refs, *new, refs, ws, n_new=_i32([n]))
                tokens = [x[0].transpose(0, 1).contiguous().to(DEV) for x in (K, V)]
                mkv.mkv_rope_append(Q, *tokens, z(n), mkv.mkv_rope_frequencies(d, 10000.0).to(DEV), k, v, *new, _i32([0, n]),
                                    torch.empty_like(Q), ws, k_scale=ks, v_scale=vs)
            assert mkv.mkv_device_status(ws) == 0
            got.append((k.cpu(), v.cpu(), new[0].cpu()))
        assert all(torch.equal(a, b) for a, b in zip(*got))


def test_two_calls_at_once_on_their_own_workspaces():
    problems = [eu.Four(30 + i, [1, 1], [[5000, 300], [40, 2000]], 4, 128, 16) for i in range(2)]
    sets = [p.on_device() for p in problems]
    streams = [torch.cuda.Stream() for _ in sets]
    spaces = [mkv.attention_workspace_for(s[0], s[1], s[3], 1, 5000) for s in sets]
    torch.cuda.synchronize()
    for _ in range(20):
        for (Q, k, v, table, lens, start, O, lse), st, ws in zip(sets, streams, spaces):
            mkv.mkv_paged_attention(Q, k, v, table, lens, start, 1, 5000, O, ws, k_scale=0.75, v_scale=1.25, lse=lse, stream=st)
    torch.cuda.synchronize()
    for p, s, ws in zip(problems, sets, spaces):
        assert mkv.mkv_device_status(ws) == 0
        p.check(s[6].cpu(), s[7].cpu())


@pytest.mark.parametrize("dtype", [BF, U8])
@pytest.mark.parametrize("start", [[0, 5, 3, 9], [-2, 1, 3, 9], [0, 3, 6, 1000], [9, 6, 3, 0]])
def test_bad_row_starts_write_inside_the_lists_only(dtype, start):
    p = Step(9, [3, 3, 3], 1, 2, 64, 16, dtype, 2)
    p.start = torch.tensor(start, dtype=torch.int32)
    p.lens.clamp_(min=9)
    axes, inv_freq = mkv.mkv_rope_axes([16, 16]), mkv.mkv_rope_frequencies(64, 10000.0)
    _, k, v = p.run(inv_freq, axes, "half", 1.0, (1.0, 1.0) if dtype is BF else (0.013, 0.3))
    assert p.status & mkv.MKV_DEV_BAD_TOKENS
    assert p.status & ~(mkv.MKV_DEV_BAD_TOKENS | mkv.MKV_DEV_BAD_SEQ_LEN | mkv.MKV_DEV_BAD_PAGE) == 0
    held = torch.zeros(k.shape[0], dtype=torch.bool)
    for b in range(3):
        for q in p.table[b, 0, :pu.pages_of(int(p.lens[b, 0]), 16)].tolist():
            if 0 <= q < len(held):
                held[q] = True
    raw = lambda x: x.view(torch.int16) if x.dtype is BF else x  # noqa: E731
    for got, old in ((k, p.k), (v, p.v)):
        assert torch.equal(raw(got)[~held], raw(old)[~held])


@pytest.mark.parametrize("rows", [33, 1100])
def test_many_rows(rows):
    rng = random.Random(rows)
    counts = [rng.choice([0, 0, 1, 2]) for _ in range(rows)]
    p = Step(10, counts, 1, 1, 64, 16, U8, 2, pad_front=2, pad_back=3)
    axes, inv_freq = mkv.mkv_rope_axes([16, 16]), mkv.mkv_rope_frequencies(64, 10000.0)
    res = p.run(inv_freq, axes, "half", 1.0, (0.013, 0.3))
    assert p.status == 0
    p.check(res, inv_freq, axes, "half", 1.0, (0.013, 0.3))


def test_no_tokens_no_lists_and_empty_lists():
    d, z = 128, lambda *s: torch.zeros(s, dtype=torch.int32, device=DEV)  # noqa: E731
    k, v = mkv.e2m1_pages(4, 16, d), mkv.e2m1_pages(4, 16, d)
    none = torch.empty((0, 8, d), dtype=BF, device=DEV)
    ws = mkv.page_workspace_for(k, z(2, 2, 1))
    freq, axes = mkv.mkv_rope_frequencies(d, 10000.0).to(DEV), mkv.mkv_rope_axes([32, 32]).to(DEV)
    mkv.mkv_rope_append_axes(none, none[:, :2], none[:, :2], z(2, 0), axes, freq, k, v, z(2, 2, 1), z(2, 2), z(3), none, ws)
    K = torch.empty((2, 2, 0, d), dtype=BF, device=DEV)
    refs, out, lens_out = z(4), z(2, 2, 1) + 9, z(2, 2) + 9
    mkv.mkv_page_quantize(k, v, z(2, 2, 1), z(2, 2), refs, None, z(2, 2), K, K, out, lens_out, refs, ws)
    assert mkv.mkv_device_status(ws) == 0 and int(lens_out.sum()) == 0 and int(refs.sum()) == 0 and (out == 9).all()
    # rows with one new token each in lists that are empty: they see nothing
    Q = torch.randn((2, 8, d), device=DEV).to(BF)
    O, lse = torch.full_like(Q, 7.0), torch.full((2, 8), 7.0, device=DEV)
    wa = mkv.attention_workspace_for(Q, k, z(2, 2, 1), 1, 16)
    mkv.mkv_paged_attention(Q, k, v, z(2, 2, 1), z(2, 2), torch.arange(3, dtype=torch.int32, device=DEV), 1, 16, O, wa, lse=lse)
    assert mkv.mkv_device_status(wa) == 0 and int((O != 0).sum()) == 0 and bool((lse == -math.inf).all())


@pytest.mark.parametrize("dtype", [BF, F8, U8])
@pytest.mark.parametrize("layout,sections", [("half", [16, 16]), ("interleaved", [12, 4])])
def test_every_row_of_more_than_32_heads_with_a_warp_per_token(dtype, layout, sections):
    # 1300 tokens: a warp has all heads of a token, and looks places up for 32 lists at a time, keys' and then values'
    H, G, d, page = 70, 2, 64, 16
    p = Step(H + sum(sections), [900, 400], H, G, d, page, dtype, 2, pad_back=3)
    n_pages = p.k.shape[0]
    p.table[0, H - 1, :] = n_pages  # one list's pages are not there
    inv_freq, axes = mkv.mkv_rope_frequencies(2 * sum(sections), 10000.0), mkv.mkv_rope_axes(sections, True)
    scales = {BF: (1.0, 1.0), F8: (0.02, 0.3), U8: (0.013, 0.3)}[dtype]
    Q, *pages = p.run(inv_freq, axes, layout, 1.25, scales)
    assert p.status == mkv.MKV_DEV_BAD_PAGE
    y, size = p.rotated(inv_freq, axes, layout, 1.25)
    hq, n = H * G, int(p.start[-1])
    _close(Q[:n], y[:n, :hq], size[:n, :hq], BF, "Q")
    assert (Q[n:] == 7.0).all()
    t = torch.arange(n)
    b = (t >= p.start[1]).long()
    s = p.lens[b] - (p.start[b + 1] - t)[:, None]                     # [n, H]
    at = p.table[b[:, None], torch.arange(H), (s // page).long()].long()
    there = at < n_pages
    assert int((~there).sum()) == 900
    at, row = at[there], (s % page).long()[there]
    for got, old, x, sz, scale in ((pages[0], p.k, y[:n, hq:hq + H][there], size[:n, hq:hq + H][there], scales[0]),
                                   (pages[1], p.v, p.qkv[:n, hq + H:].double()[there], 0 * size[:n, hq:hq + H][there], scales[1])):
        if dtype is U8:
            want = eu.rows_of(old).view(U8).clone()
            want[at, row] = torch.cat(eu.encode(x.float(), scale), -1)
            assert torch.equal(eu.rows_of(got).view(U8), want)
            continue
        ref = x / scale
        _close(pu.raw(got)[at, row].view(dtype), ref.clamp(-448, 448) if dtype is F8 else ref, sz / scale, dtype, "pages")
        got, want = pu.raw(got).clone(), pu.raw(old).clone()
        got[at, row] = want[at, row] = 0
        assert torch.equal(got, want)
