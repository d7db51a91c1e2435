"""mkv_paged_attention over 4-bit pages against the definition in 64 bits, in both forms: head dims, page sizes, groups,
lists of 0, 1 and many tokens, windows, rows that see nothing, NaN scales behind every list's end, bad pages, queries that
are not finite; and the whole path compress -> 4-bit pages -> grow -> append -> attend."""
import math
import random

import pytest
import torch

import e2m1_util as eu
import geometric_kv_cache_gb300 as mkv
import paged_util as pu
from e2m1_util import Four, wide
from test_gpu_paged_edges import _check, _spoil

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F8 = torch.bfloat16, torch.float8_e4m3fn
SHAPES = [(64, 16), (64, 128), (128, 16), (128, 64), (256, 16), (256, 128)]


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mkv.load()
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


@pytest.mark.parametrize("d,page", SHAPES)
@pytest.mark.parametrize("G", [1, 4, 7, 8, 9, 16, 40])
def test_decode(d, page, G):
    lens = [[0, 1], [page, page + 1], [2, page - 1], [300, 17], [1025, 640]]
    p = Four(G, [1] * 5, lens, G, d, page, pad=2, spare_len=37)
    O, lse = p.run()
    assert p.status == 0
    p.check(O, lse)


@pytest.mark.parametrize("d,page", SHAPES)
@pytest.mark.parametrize("counts", [[3, 0, 1, 40], [130, 1, 2, 64]])
def test_few_new_tokens_and_chunks(d, page, counts):
    lens = [[c + x for x in (0, 5)] for c in counts]
    lens[0] = [counts[0] + 150, max(counts[0] - 2, 0)]  # a list shorter than its new tokens: the first see nothing
    p = Four(5, counts, lens, 3, d, page, pad=1)
    O, lse = p.run()
    assert p.status == 0
    p.check(O, lse)


@pytest.mark.parametrize("d,page", SHAPES)
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 4), (16, 0), (33, 1), (100, 64), (100, 300), (5000, 4),
                                          (2 ** 31 - 1, 2 ** 31 - 1)])
def test_window_and_first_tokens(d, page, window, sinks):
    for counts in ([1, 1, 1], [20, 1, 5]):
        lens = [[c + x for x in (0, 333)] for c in counts]
        p = Four(window, counts, lens, 4, d, page)
        O, lse = p.run(window, sinks)
        assert p.status == 0
        p.check(O, lse, window, sinks)


@pytest.mark.parametrize("d,page", SHAPES)
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 4), (33, 0), (130, 64)])
def test_chunk_form_windows_and_short_lists(d, page, window, sinks):
    p = wide(window + 1, [36, 0, 1, 2, 40], [0, 1, -3, 200, 430, -40], 8, d, page, pad=2, spare_len=300)
    O, lse = p.run(window, sinks)
    assert p.status == 0
    p.check(O, lse, window, sinks)


@pytest.mark.parametrize("d,page", SHAPES)
@pytest.mark.parametrize("extra", [[0, 128, 256, 900, 1500], [1900]])
def test_chunk_form_cut_and_whole_tiles(d, page, extra):
    p = wide(3, [66, 20, 33, 1], extra, 4, d, page)
    a, b = p.run(strided=True), p.run()
    assert p.status == 0
    p.check(*a)
    assert torch.equal(a[0].view(torch.int16), b[0].view(torch.int16)) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("q_scale,scale", [(0.0, None), (30.0, None), (1.0, -0.3), (1.0, 0.0), (1.0, -1e-37)])
@pytest.mark.parametrize("form", ["few", "chunk"])
def test_flat_sharp_tiny_and_negative(form, q_scale, scale):
    p = Four(3, [1, 3], [[500, 64], [700, 33]], 4, 128, 16, q_scale=q_scale) if form == "few" else \
        wide(4, [40, 3, 10], [0, 7, 300], 8, 128, 16, q_scale=q_scale, spare_len=200)
    p.Q[0] = 0
    for t, e in ((1, -120), (2, -70), (3, -30)):
        p.Q[t] = (p.Q[t].double() * 2.0 ** e).to(BF)
    O, lse = p.run(scale=scale)
    assert p.status == 0
    p.check(O, lse, scale=scale)


def test_scales_from_the_smallest_to_the_largest():
    """Groups under every E4M3 scale, zero and the largest among them, next to values of the largest codes."""
    for form in ("few", "chunk"):
        p = Four(8, [1, 2], [[200, 64], [130, 33]], 4, 128, 16, q_scale=0.01) if form == "few" else \
            wide(8, [40, 3, 10], [0, 7, 300], 8, 128, 16, q_scale=0.01, spare_len=200)
        for name, pages in (("k", p.kp), ("v", p.vp)):
            codes, scales = (x.clone() for x in eu.from_pages(pages))
            g = torch.Generator().manual_seed(1)
            used = scales != 0x7F
            scales[used] = torch.randint(0, 0x7F, scales.shape, generator=g).to(torch.uint8)[used]
            pages.copy_(eu.to_pages(codes, scales))
            setattr(p, name, eu.decode(codes, scales).to(BF))
        O, lse = p.run()
        assert p.status == 0
        p.check(O, lse)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("form", ["few", "chunk"])
def test_queries_that_are_not_finite(d, form):
    if form == "few":
        p = Four(21, [2, 1, 1], [[6000, 50], [70, 3000], [60, 60]], 5, d, 16)
        _spoil(p, [0, 2])
    else:
        p = wide(22, [66, 20, 33, 1], [2500, 900], 4, d, 16)
        _spoil(p, [0, 40, 70, 119])
    O, lse = p.run()
    assert p.status == 0
    _check(p, O, lse, nans=True)


@pytest.mark.parametrize("d,page", [(64, 16), (128, 16), (128, 128), (256, 32)])
@pytest.mark.parametrize("form", ["few", "chunk"])
def test_pages_outside_the_pool_count_as_zeros(form, d, page):
    if form == "few":
        p = Four(23, [1, 2], [[600, 200], [290, 9]], 4, d, page)
        bad = [(0, 0, 0), (0, 0, 3), (0, 1, 0), (1, 0, 2)]
    else:
        p = wide(23, [70, 9, 30], [500], 8, d, page)
        bad = [(0, 0, 2), (0, 0, 3), (0, 5, 0), (2, 7, 3)]
    zero = torch.zeros((1, *p.k.shape[1:]), dtype=BF)
    k, v, table = torch.cat([p.k, zero]), torch.cat([p.v, zero]), p.table.clone()
    for i, at in enumerate(bad):
        table[at] = p.k.shape[0]
        p.table[at] = [p.k.shape[0], -1, 2 ** 31 - 1, -2 ** 31][i]
    O, lse = p.run()
    assert p.status == mkv.MKV_DEV_BAD_PAGE
    p.k, p.v, p.table = k, v, table
    p.check(O, lse)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_long_lists_cut_in_parts_and_joined(d):
    p = Four(12, [2, 1, 1], [[9000, 3], [1, 0], [64, 4097]], 4, d, 16)
    O, lse = p.run()
    _check(p, O, lse)
    p = Four(13, [1], [[30000]], 12, d, 64)
    a, b = p.run(), p.run()
    _check(p, *a)
    assert torch.equal(a[0].view(torch.int16), b[0].view(torch.int16)) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("extra", [[255], [700, 29], [-1, 59, 3899]])
def test_many_short_lists_and_a_few_long_ones(extra):
    p = Four(18, [1] * 70, [[1 + extra[b % len(extra)], 1 + extra[(b + 1) % len(extra)]] for b in range(70)], 2, 128, 16, pad=1)
    a, b = p.run(), p.run()
    assert p.status == 0
    p.check(*a)
    assert torch.equal(a[0].view(torch.int16), b[0].view(torch.int16)) and torch.equal(a[1], b[1])


def test_more_lists_than_threads():
    rng = random.Random(1)
    counts = [rng.choice([0, 1, 1]) for _ in range(400)]
    lens = [[c + rng.choice([0, 1, 30]) for _ in range(3)] for c in counts]
    lens[90][1] = lens[251][2] = 900
    p = Four(16, counts, lens, 2, 64, 16, pad=3)
    O, lse = p.run()
    assert p.status == 0
    p.check(O, lse)


def test_invalid_rows_and_lengths_are_reported():
    p = Four(7, [2, 9], [[60, 200], [50, 9]], 2, 128, 16)
    first = p.run()[0]
    O, lse = p.run(max_q=8)  # row 1 brings 9
    assert p.status == mkv.MKV_DEV_BAD_TOKENS
    p.check(O, lse, rows=slice(0, 2))
    assert torch.equal(O[2:], torch.full_like(O[2:], 7.0))
    p.max_len = 199
    p.table = p.table[..., :13].contiguous()
    O, lse = p.run()
    assert p.status == mkv.MKV_DEV_BAD_SEQ_LEN
    assert torch.equal(O[:2, :2], first[:2, :2])
    assert torch.equal(O[:2, 2:], torch.full_like(O[:2, 2:], 7.0))


@pytest.mark.parametrize("counts", [[1, 1], [50, 3]])
def test_strided_queries_and_outputs_on_another_stream(counts):
    p = Four(6, counts, [[60, 200], [5, 9]], 2, 128, 16)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        O, lse = p.run(strided=True)
    p.check(O, lse)


@pytest.mark.parametrize("G,n", [(4, 1), (16, 1), (8, 100)])
def test_captured_call_replays_on_longer_lists(G, n):
    heads = 2 if n == 1 else 12
    p = Four(10, [n, 1, 1, 1], [[n + 700] * heads] * 4, G, 128, 16)
    Q, k, v, table, lens, start, O, lse = p.on_device()
    ws = mkv.attention_workspace_for(Q, k, table, n, p.max_len)
    call = lambda: mkv.mkv_paged_attention(Q, k, v, table, lens, start, n, p.max_len, O, ws, k_scale=0.75,  # noqa: E731
                                           v_scale=1.25, lse=lse)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.synchronize()
    p.check(O.cpu(), lse.cpu())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for new in ([[n + 650, 1] * (heads // 2)] * 4, [[n, 130] * (heads // 2), [5, 600] * (heads // 2), [16, 17] * (heads // 2),
                                                    [699, 400] * (heads // 2)]):
        p.lens = torch.tensor(new, dtype=torch.int32)
        lens.copy_(p.lens)
        O.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        p.check(O.cpu(), lse.cpu())
    assert mkv.mkv_device_status(ws) == 0


def test_compress_then_4_bit_pages_then_steps():
    """A bf16 prompt is compressed with per-head counts, its kept rows become 4-bit pages, the sequence forks, and rounds of
    new tokens with positions on three axes are appended and attended; the reference rebuilds every list as plain rows."""
    torch.manual_seed(0)
    B, H, G, T, d, page = 2, 3, 2, 300, 128, 16
    K, V = (torch.randn(B, H, T, d) * 2).to(BF), torch.randn(B, H, T, d).to(BF)
    Kd, Vd = K.to(DEV), V.to(DEV)
    n_keep = torch.tensor([[150, 20, 33], [299, 16, 1]], dtype=torch.int32, device=DEV)
    ks = 299
    idx = torch.full((B, H, ks), -1, dtype=torch.int32, device=DEV)
    kept = torch.zeros((B, H), dtype=torch.int32, device=DEV)
    Ko, Vo = (torch.empty((B, H, ks, d), dtype=BF, device=DEV) for _ in range(2))
    mkv.mkv_compress(Kd, Vd, 0.5, "l2", 0, ks, Ko, Vo, idx, kept, mkv.workspace_for(Kd), n_keep=n_keep)
    n_pages, max_pages = 200, 24
    k = torch.full((n_pages, page, 72), 255, dtype=torch.uint8, device=DEV)
    v = k.clone()
    bufs = [[torch.zeros((B + 1, H, max_pages), dtype=torch.int32, device=DEV),
             torch.zeros((B + 1, H), dtype=torch.int32, device=DEV)] for _ in range(2)]
    refs = torch.zeros(n_pages, dtype=torch.int32, device=DEV)
    part = [[t[:B] for t in x] for x in bufs]
    wsp = mkv.page_workspace_for(k, bufs[0][0])
    scales = (0.125, 0.0625)
    mkv.mkv_page_quantize(k, v, *part[0], refs, idx, kept, Kd, Vd, *part[1], refs, wsp, *scales)
    kept_c, idx_c = kept.cpu(), idx.cpu()
    enc = lambda x, s: torch.cat(eu.encode(x.float(), s), -1)  # noqa: E731
    plain = {(b, j): [enc(x[b, j][idx_c[b, j, :kept_c[b, j]].long()], s) for x, s in ((K, scales[0]), (V, scales[1]))]
             for b in range(B) for j in range(H)}
    none = torch.zeros((0, 72), dtype=torch.uint8)
    plain.update({(2, j): [none, none] for j in range(H)})
    inv_freq, axes = mkv.mkv_rope_frequencies(64, 10000.0), mkv.mkv_rope_axes([12, 10, 10], True)
    cur = 1
    for parent, counts in (([0, 1, 0], [5, 1, 1]), ([2, 1, 2], [1, 1, 1]), (None, [1, 30, 1])):
        src, dst = bufs[cur], bufs[1 - cur]
        n_new = torch.tensor(counts, dtype=torch.int32, device=DEV)
        if parent is None:
            mkv.mkv_page_update(k, v, *src, refs, *src, refs, wsp, n_new=n_new)
        else:
            mkv.mkv_page_update(k, v, *src, refs, *dst, refs, wsp, n_new=n_new,
                                parent=torch.tensor(parent, dtype=torch.int32, device=DEV))
            cur = 1 - cur
            plain = {(b, j): plain[parent[b], j] for b in range(B + 1) for j in range(H)}
        table, lens = bufs[cur]
        start = torch.tensor([0] + list(torch.tensor(counts).cumsum(0)), dtype=torch.int32)
        n = int(start[-1])
        qkv = torch.randn(n, H * (G + 2), d).to(BF)
        pos = torch.randint(0, 5000, (3, n), dtype=torch.int32)
        Q, x = torch.empty((n, H * G, d), dtype=BF, device=DEV), qkv.to(DEV)
        mkv.mkv_rope_append_axes(x[:, :H * G], x[:, H * G:H * (G + 1)], x[:, H * (G + 1):], pos.to(DEV), axes.to(DEV),
                                 inv_freq.to(DEV), k, v, table, lens, start.to(DEV), Q, wsp, k_scale=scales[0],
                                 v_scale=scales[1])
        a = (pos[axes.long()].T.double() * inv_freq.double())[:, None]
        y = qkv.double()
        y = torch.cat([y[..., :32] * a.cos() - y[..., 32:64] * a.sin(), y[..., :32] * a.sin() + y[..., 32:64] * a.cos(),
                       y[..., 64:]], -1)
        rk, rv = (eu.rows_of(x.cpu()).view(torch.uint8) for x in (k, v))
        tc, lc = table.cpu(), lens.cpu()
        for (b, j), old in list(plain.items()):
            t0, t1 = int(start[b]), int(start[b + 1])
            new = (enc(y[t0:t1, H * G + j], scales[0]), enc(qkv[t0:t1, H * (G + 1) + j], scales[1]))
            rows = [torch.cat([o, w]) for o, w in zip(old, new)]
            L, ids = int(lc[b, j]), tc[b, j, :pu.pages_of(int(lc[b, j]), page)].long()
            assert L == len(rows[0])
            for got, want in zip((rk, rv), rows):
                assert torch.equal(got[ids].reshape(-1, 72)[:L], want)
            plain[b, j] = rows
        max_q, max_len = max(counts), max_pages * page
        wsa = mkv.attention_workspace_for(Q, k, table, max_q, max_len)
        O, lse = torch.empty_like(Q), torch.empty((n, H * G), device=DEV)
        mkv.mkv_paged_attention(Q, k, v, table, lens, start.to(DEV), max_q, max_len, O, wsa, k_scale=scales[0],
                                v_scale=scales[1], window=64, sinks=4, lse=lse)
        kc, vc = (eu.decode(r[..., :64].contiguous(), r[..., 64:].contiguous()).to(BF) for r in (rk, rv))
        ref = pu.attention(Q.cpu(), kc, vc, tc, lc, start, page, d ** -0.5, *scales, 64, 4)
        tol, tol_lse = pu.attention_bounds(*ref, d, F8)
        assert ((O.cpu().double() - ref[0]).abs() <= tol).all()
        assert ((lse.cpu().double() - ref[1]).abs() <= tol_lse).all()
        assert mkv.mkv_device_status(wsa) == 0
    assert mkv.mkv_device_status(wsp) == 0
    held = torch.zeros(n_pages, dtype=torch.int32)
    for b in range(B + 1):
        for j in range(H):
            for q in tc[b, j, :pu.pages_of(int(lc[b, j]), page)].tolist():
                held[q] += 1
    assert torch.equal(held, refs.cpu())
