"""mkv_paged_attention against the definition in 64 bits: head dims, cache types, page sizes, groups of query heads,
lists of 0, 1 and many tokens, decode and chunks, windows with first tokens, rows that see nothing, NaN behind every
list's end; and the whole path compress -> pages -> grow -> append -> attend."""
import math
import random

import pytest
import torch

import geometric_kv_cache_gb300 as mkv
import paged_util as pu

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F8 = torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mkv.load()
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


class Problem:
    def __init__(self, seed, counts, lens, G, d, page, dtype, q_scale=1.0, pad=0, spare_len=0):
        rng = random.Random(seed)
        H = len(lens[0])
        self.page, self.dtype, self.G, self.d = page, dtype, G, d
        self.max_len = max(max(r) for r in lens) + spare_len
        max_pages = pu.pages_of(self.max_len, page)
        need = sum(pu.pages_of(x, page) for r in lens for x in r)
        self.table, self.lens, _ = pu.random_lists(rng, lens, page, need + 2, max_pages)
        self.k, self.v = pu.random_pool(seed, need + 2, page, d, dtype)
        pu.poison_unused(self.k, self.v, self.table, self.lens, page)
        start = [0]
        for n in counts:
            start.append(start[-1] + n)
        self.start = torch.tensor(start, dtype=torch.int32)
        self.max_q = max(counts)
        self.n = start[-1] + pad
        g = torch.Generator().manual_seed(seed + 1)
        self.Q = (torch.randn((self.n, H * G, d), generator=g) * q_scale).to(BF)
        self.scales = (0.75, 1.25) if dtype == F8 else (1.0, 1.0)

    def run(self, window=0, sinks=0, scale=None, max_q=None, strided=False, stream=None):
        dev = lambda x: pu.raw(x).to(DEV).view(x.dtype) if x.dtype in pu.CODES else x.to(DEV)  # noqa: E731
        k, v, table, lens, start = (dev(x) for x in (self.k, self.v, self.table, self.lens, self.start))
        Q = dev(self.Q)
        O = torch.full_like(Q, 7.0)
        if strided:  # slices of wider rows
            wide = torch.full((self.n, Q.shape[1] + 3, self.d), 3.0, dtype=BF, device=DEV)
            wide[:, 1:-2] = Q
            Q, O = wide[:, 1:-2], torch.full_like(wide, 7.0)[:, 2:-1]
        lse = torch.full(Q.shape[:2], 7.0, device=DEV)
        max_q = self.max_q if max_q is None else max_q
        ws = mkv.attention_workspace_for(Q, k, table, max_q, self.max_len)
        ws[256:] = 255  # (what a call leaves in the workspace is NaN to the next)
        mkv.mkv_paged_attention(Q, k, v, table, lens, start, max_q, self.max_len, O, ws, scale=scale,
                                k_scale=self.scales[0], v_scale=self.scales[1], window=window, sinks=sinks, lse=lse)
        self.status = mkv.mkv_device_status(ws)
        return O.cpu(), lse.cpu()

    def check(self, O, lse, window=0, sinks=0, scale=None, rows=None):
        scale = self.d ** -0.5 if scale is None else scale
        ref, ref_lse, A, W, E = pu.attention(self.Q, self.k, self.v, self.table, self.lens, self.start, self.page, scale,
                                             *self.scales, window, sinks)
        tol, tol_lse = pu.attention_bounds(ref, ref_lse, A, W, E, self.d, self.dtype)
        n = int(self.start[-1])
        rows = slice(0, n) if rows is None else rows
        err = (O.double() - ref).abs()
        bad = ~(err <= tol)
        assert not bad[rows].any(), (int(bad[rows].sum()), float((err / tol)[rows].max()))
        assert torch.equal(torch.isinf(lse)[rows], torch.isinf(ref_lse)[rows])
        off = (lse.double() - ref_lse).abs()
        assert not (off > tol_lse)[rows][torch.isfinite(ref_lse[rows])].any(), float(off[rows].nan_to_num(0).max())
        assert torch.equal(O[n:], torch.full_like(O[n:], 7.0)) and torch.equal(lse[n:], torch.full_like(lse[n:], 7.0))


SHAPES = [(64, BF, 16), (64, F8, 32), (128, BF, 16), (128, BF, 128), (128, F8, 16), (128, F8, 64), (256, BF, 32),
          (256, F8, 16)]


@pytest.mark.parametrize("d,dtype,page", SHAPES)
@pytest.mark.parametrize("G", [1, 4, 7, 16, 40])
def test_decode(d, dtype, page, G):
    lens = [[0, 1], [page, page + 1], [2, page - 1], [300, 17], [1025, 640]]
    p = Problem(G, [1] * 5, lens, G, d, page, dtype, pad=2, spare_len=37)
    O, lse = p.run()
    assert p.status == 0
    p.check(O, lse)


@pytest.mark.parametrize("d,dtype,page", SHAPES)
@pytest.mark.parametrize("counts", [[3, 0, 1, 40], [130, 1, 2, 64], [200, 0, 0, 129]])
def test_chunks(d, dtype, page, counts):
    lens = [[c + x for x in (0, 5)] for c in counts]
    lens[0] = [counts[0] + 150, max(counts[0] - 2, 0)]  # a list shorter than its new tokens: the first see nothing
    p = Problem(5, counts, lens, 3, d, page, dtype, pad=1)
    O, lse = p.run()
    assert p.status == 0
    p.check(O, lse)


@pytest.mark.parametrize("d,dtype,page", SHAPES)
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 4), (16, 0), (33, 1), (100, 64), (100, 300), (5000, 4)])
def test_window_and_first_tokens(d, dtype, page, window, sinks):
    for counts in ([1, 1, 1], [70, 1, 5]):
        lens = [[c + x for x in (0, 333)] for c in counts]
        p = Problem(window, counts, lens, 4, d, page, dtype)
        O, lse = p.run(window, sinks)
        assert p.status == 0
        p.check(O, lse, window, sinks)


@pytest.mark.parametrize("counts", [[1, 1], [70, 3]])
@pytest.mark.parametrize("window,sinks", [(2 ** 31 - 1, 0), (2 ** 31 - 1, 2 ** 31 - 1), (3, 2 ** 31 - 1), (400, 0)])
def test_largest_window_and_first_tokens(counts, window, sinks):
    # row 1's second list is shorter than its new tokens: places below zero
    p = Problem(14, counts, [[counts[0] + 300, counts[0]], [40, counts[1] - 1]], 4, 128, 16, BF)
    O, lse = p.run(window, sinks)
    assert p.status == 0
    p.check(O, lse, window, sinks)


@pytest.mark.parametrize("dtype", [BF, F8])
@pytest.mark.parametrize("q_scale", [0.0, 30.0])
def test_flat_and_sharp_softmax(dtype, q_scale):
    p = Problem(3, [1, 33], [[500, 64], [700, 33]], 4, 128, 16, dtype, q_scale=q_scale)
    O, lse = p.run()
    p.check(O, lse)
    O, lse = p.run(scale=-0.3)
    p.check(O, lse, scale=-0.3)


@pytest.mark.parametrize("d,dtype", [(128, BF), (128, F8), (64, BF)])
@pytest.mark.parametrize("most", [1, 600])
def test_more_lists_than_threads(d, dtype, most):
    # decode and chunk forms over hundreds to thousands of tiles, most of them without rows or with few keys
    rng = random.Random(most)
    counts = [rng.choice([0, 1, 1]) for _ in range(260)]
    counts[37] = most
    counts[200] = min(most, 40)
    lens = [[c + rng.choice([0, 1, 30]) for _ in range(3)] for c in counts]
    lens[90][1] = lens[251][2] = 900
    p = Problem(16, counts, lens, 2, d, 16, dtype, pad=3)
    O, lse = p.run()
    assert p.status == 0
    p.check(O, lse)


@pytest.mark.parametrize("dtype", [BF, F8])
@pytest.mark.parametrize("counts", [[1, 1], [70, 2]])
def test_queries_of_zero_and_tiny_and_large_ones(dtype, counts):
    p = Problem(17, counts, [[counts[0] + 100, counts[0]], [40, 300]], 4, 128, 16, dtype)
    p.Q[0] = 0
    p.Q[-1] = 0
    if counts[0] > 1:
        for t, e in ((1, -120), (2, -70), (3, -30), (4, 8)):
            p.Q[t] = (p.Q[t].double() * 2.0 ** e).to(BF)
    for scale in (None, 0.0, 1e-30, -1e-37):
        O, lse = p.run(scale=scale)
        p.check(O, lse, scale=scale)


def test_one_long_list_among_short_ones():
    p = Problem(4, [1, 1, 1], [[9000, 3], [1, 0], [64, 4097]], 4, 128, 16, BF)
    O, lse = p.run()
    p.check(O, lse)


@pytest.mark.parametrize("counts", [[1, 1], [50, 3]])
def test_strided_queries_and_outputs(counts):
    p = Problem(6, counts, [[60, 200], [5, 9]], 2, 128, 16, BF)
    O, lse = p.run(strided=True)
    p.check(O, lse)


def test_larger_bounds_change_little_and_smaller_ones_are_reported():
    p = Problem(7, [2, 9], [[60, 200], [50, 9]], 2, 128, 16, BF)
    p.check(*p.run(max_q=300))
    first = p.run()[0]
    O, lse = p.run(max_q=8)  # row 1 brings 9
    assert p.status == mkv.MKV_DEV_BAD_TOKENS
    p.check(O, lse, rows=slice(0, 2))
    assert torch.equal(O[2:], torch.full_like(O[2:], 7.0))
    p.max_len = 199
    p.table = p.table[..., :13].contiguous()
    O, lse = p.run()
    assert p.status == mkv.MKV_DEV_BAD_SEQ_LEN
    assert torch.equal(O[:2, :2], first[:2, :2])  # the other head's list is in bounds
    assert torch.equal(O[:2, 2:], torch.full_like(O[:2, 2:], 7.0))
    p.check(O, lse, rows=slice(2, 11))


@pytest.mark.parametrize("start", [[0, 3, 1], [-1, 2, 4], [0, 2, 500]])
def test_bad_row_starts_are_reported(start):
    p = Problem(8, [2, 2], [[60, 20], [50, 9]], 2, 128, 16, BF)
    p.start = torch.tensor(start, dtype=torch.int32)
    p.max_q = 8
    p.run()
    assert p.status == mkv.MKV_DEV_BAD_TOKENS


@pytest.mark.parametrize("counts", [[1, 1], [140, 3]])
def test_pages_outside_the_pool_are_reported(counts):
    p = Problem(9, counts, [[600, 200], [50, 9]], 2, 128, 16, BF)
    p.table[0, 0, 2] = p.k.shape[0]
    p.table[0, 0, 3] = -1
    O, lse = p.run()
    assert p.status == mkv.MKV_DEV_BAD_PAGE
    p.table[0, 0, 2:4] = p.table[0, 0, 0]
    n = counts[0]
    O[:n, :2], lse[:n, :2] = 0, 0
    ref = pu.attention(p.Q, p.k, p.v, p.table, p.lens, p.start, 16, 128 ** -0.5)
    tol, _ = pu.attention_bounds(*ref, 128, BF)
    assert ((O.double() - ref[0]).abs() <= tol)[:, 2:].all()


def test_captured_call_replays_on_longer_lists():
    p = Problem(10, [1, 1, 1, 1], [[700, 800]] * 4, 4, 128, 16, BF)
    dev = lambda x: pu.raw(x).to(DEV).view(x.dtype) if x.dtype in pu.CODES else x.to(DEV)  # noqa: E731
    Q, k, v, table, lens, start = (dev(x) for x in (p.Q, p.k, p.v, p.table, p.lens, p.start))
    O, lse = torch.zeros_like(Q), torch.zeros(Q.shape[:2], device=DEV)
    ws = mkv.attention_workspace_for(Q, k, table, 1, 800)
    call = lambda: mkv.mkv_paged_attention(Q, k, v, table, lens, start, 1, 800, O, ws, lse=lse)  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.synchronize()
    p.check(O.cpu(), lse.cpu())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for new in ([[700, 1]] * 4, [[0, 130], [5, 800], [16, 17], [699, 400]]):
        p.lens = torch.tensor(new, dtype=torch.int32)
        lens.copy_(p.lens)
        O.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        p.check(O.cpu(), lse.cpu())
    assert mkv.mkv_device_status(ws) == 0


@pytest.mark.parametrize("d,dtype,page", [(64, BF, 16), (128, BF, 64), (256, BF, 16), (128, F8, 32)])
def test_long_lists_of_full_and_nearly_empty_tiles(d, dtype, page):
    # tiles of many blocks of keys, of which some have all their rows and some a few, cut in several parts
    p = Problem(12, [70, 1, 130, 3, 1], [[5000, 900], [4000, 2500], [300, 6000], [5200, 33], [1, 3000]], 2, d, page, dtype)
    O, lse = p.run()
    assert p.status == 0
    p.check(O, lse)


@pytest.mark.parametrize("d,dtype,page", [(64, BF, 16), (128, BF, 64), (128, F8, 32), (256, BF, 32)])
@pytest.mark.parametrize("extra", [[255], [700, 29], [-1, 59, 3899], [1999]])
def test_many_short_lists_and_a_few_long_ones(d, dtype, page, extra):
    # 140 tiles over 152 CTAs: cuts move to the ends of short tiles, long ones among them are cut all the same
    p = Problem(18, [1] * 70, [[1 + extra[b % len(extra)], 1 + extra[(b + 1) % len(extra)]] for b in range(70)], 2, d,
                page, dtype, pad=1)
    a, b = p.run(), p.run()
    assert p.status == 0
    p.check(*a)
    assert torch.equal(a[0].view(torch.int16), b[0].view(torch.int16)) and torch.equal(a[1], b[1])


def wide(seed, counts, extra, G, d, page, dtype, heads=16, **kw):
    """A problem of enough query rows for the form for chunks: its parts in the workspace are 128 or 256 rows, not 16."""
    p = Problem(seed, counts, [[max(0, c + extra[(b + j) % len(extra)]) for j in range(heads)]
                               for b, c in enumerate(counts)], G, d, page, dtype, **kw)
    pool = torch.empty(p.k.shape, dtype=dtype, device=DEV)
    ws = mkv.attention_workspace_for(torch.empty((p.n, heads * G, d), dtype=BF, device=DEV), pool,
                                     torch.empty(p.table.shape, dtype=torch.int32, device=DEV), p.max_q, p.max_len)
    assert ws.numel() > 152 * 2 * 100 * (4 * d + 8)
    return p


@pytest.mark.parametrize("d,dtype,page", SHAPES)
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 4), (33, 0), (130, 64), (5000, 4)])
def test_chunk_form_windows_and_short_lists(d, dtype, page, window, sinks):
    # lists shorter than their new tokens (the first see nothing), empty ones, rows without tokens and of one token
    p = wide(window + 1, [36, 0, 1, 2, 20], [0, 1, -3, 200, 430, -40], 8, d, page, dtype, pad=2)
    O, lse = p.run(window, sinks)
    assert p.status == 0
    p.check(O, lse, window, sinks)


@pytest.mark.parametrize("d,dtype,page", SHAPES)
def test_chunk_form_one_token_per_row(d, dtype, page):
    p = wide(2, [1] * 80, [-1, 0, 5, 129, page, 700], 40, d, page, dtype, heads=2)
    O, lse = p.run()
    assert p.status == 0
    p.check(O, lse)


@pytest.mark.parametrize("d,dtype,page", SHAPES)
@pytest.mark.parametrize("extra", [[0, 128, 256, 900, 1500], [1900], [0, 60]])
def test_chunk_form_cut_and_whole_tiles(d, dtype, page, extra):
    # 96 to 160 tiles of 1 to 32 blocks: some lines are cut at tiles' ends, some inside tiles
    p = wide(3, [66, 20, 33, 1], extra, 4, d, page, dtype)
    a, b = p.run(strided=True), p.run()
    assert p.status == 0
    p.check(*a)
    assert torch.equal(a[0].view(torch.int16), b[0].view(torch.int16)) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("d,dtype,page", [(64, F8, 32), (128, BF, 16), (128, F8, 64), (256, BF, 32)])
@pytest.mark.parametrize("q_scale,scale", [(0.0, None), (30.0, None), (1.0, -0.3), (1.0, 0.0), (1.0, -1e-37)])
def test_chunk_form_flat_sharp_and_negative_scales(d, dtype, page, q_scale, scale):
    p = wide(4, [36, 3, 10], [0, 7, 300], 8, d, page, dtype, q_scale=q_scale)
    p.Q[0] = 0
    for t, e in ((1, -120), (2, -70), (3, -30), (4, 8)):
        p.Q[t] = (p.Q[t].double() * 2.0 ** e).to(BF)
    O, lse = p.run(scale=scale)
    assert p.status == 0
    p.check(O, lse, scale=scale)


@pytest.mark.parametrize("dtype", [BF, F8])
def test_chunk_form_reports_bad_pages_rows_and_lengths(dtype):
    p = wide(5, [70, 9, 30], [300], 8, 128, 16, dtype)
    good, _ = p.run()
    table, lens, start = p.table.clone(), p.lens.clone(), p.start.clone()
    p.table[0, 0, 2], p.table[0, 5, 3] = p.k.shape[0], -1
    O, _ = p.run()
    assert p.status == mkv.MKV_DEV_BAD_PAGE
    assert torch.equal(O[70:], good[70:]) and torch.equal(O[:, 8:40], good[:, 8:40])
    p.table = table.clone()
    p.lens[1, 3] = p.max_len + 1
    O, _ = p.run()
    assert p.status == mkv.MKV_DEV_BAD_SEQ_LEN
    untouched = torch.full_like(O[70:79, 24:32], 7.0)
    assert torch.equal(O[70:79, 24:32], untouched) and torch.equal(O[:70], good[:70])
    p.lens = lens.clone()
    p.start = start.clone()
    p.start[2] = p.start[3] + 1  # row 2 ends before it begins
    p.run(max_q=70)
    assert p.status == mkv.MKV_DEV_BAD_TOKENS


def test_workspace_of_any_contents_after_one_status_call():
    p = Problem(15, [1, 1], [[3000, 200], [50, 4000]], 4, 128, 16, BF)
    dev = lambda x: pu.raw(x).to(DEV).view(x.dtype) if x.dtype in pu.CODES else x.to(DEV)  # noqa: E731
    Q, k, v, table, lens, start = (dev(x) for x in (p.Q, p.k, p.v, p.table, p.lens, p.start))
    O, lse = torch.zeros_like(Q), torch.zeros(Q.shape[:2], device=DEV)
    ws = torch.full_like(mkv.attention_workspace_for(Q, k, table, 1, 4000), 0xA7)
    assert mkv.mkv_device_status(ws) == 0xA7A7A7A7
    for _ in range(3):
        O.fill_(7.0)
        mkv.mkv_paged_attention(Q, k, v, table, lens, start, 1, 4000, O, ws, lse=lse)
        assert int(ws[:256].sum()) == 0
        p.check(O.cpu(), lse.cpu())
    assert mkv.mkv_device_status(ws) == 0


@pytest.mark.parametrize("counts", [[1, 1], [90, 1]])
def test_same_bits_on_every_call(counts):
    p = Problem(11, counts, [[2000, 200], [50, 1500]], 4, 128, 16, BF)
    a, b = p.run(), p.run()
    assert torch.equal(a[0].view(torch.int16), b[0].view(torch.int16)) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("dtype", [BF, F8])
def test_compress_then_pages_then_steps(dtype):
    """A prompt is compressed with per-head counts, its kept rows go into pages, the sequence forks, and two rounds of new
    tokens are appended and attended; the reference rebuilds every list as a plain sequence of rows."""
    torch.manual_seed(0)
    B, H, G, T, d, page, rot = 2, 3, 2, 300, 128, 16, 64
    K = (torch.randn(B, H, T, d) * 2).to(dtype)
    V = torch.randn(B, H, T, d).to(dtype)
    dev = lambda x: pu.raw(x).to(DEV).view(x.dtype)  # noqa: E731
    Kd, Vd = dev(K), dev(V)
    n_keep = torch.tensor([[150, 20, 33], [299, 16, 1]], dtype=torch.int32, device=DEV)
    ks = 299
    idx = torch.full((B, H, ks), -1, dtype=torch.int32, device=DEV)
    kept = torch.zeros((B, H), dtype=torch.int32, device=DEV)
    Ko, Vo = (torch.empty((B, H, ks, d), dtype=dtype, device=DEV) for _ in range(2))
    ws0 = mkv.workspace_for(Kd)
    mkv.mkv_compress(Kd, Vd, 0.5, "l2", 0, ks, Ko, Vo, idx, kept, ws0, n_keep=n_keep)
    n_pages, max_pages = 200, 24
    k = torch.full((n_pages, page, d), float("nan")).to(dtype).to(DEV)
    v = k.clone()
    bufs = [[torch.zeros((B + 1, H, max_pages), dtype=torch.int32, device=DEV),
             torch.zeros((B + 1, H), dtype=torch.int32, device=DEV)] for _ in range(2)]
    refs = torch.zeros(n_pages, dtype=torch.int32, device=DEV)
    # rows 0 and 1 hold the prompts, row 2 is free; the fill call sees the first two rows alone
    part = [[t[:B] for t in x] for x in bufs]
    wsp = mkv.page_workspace_for(k, bufs[0][0])
    mkv.mkv_page_compact(k, v, *part[0], refs, idx, kept, *part[1], refs, wsp, K=Kd, V=Vd)
    kept_c, idx_c = kept.cpu(), idx.cpu()
    plain = {(b, j): tuple(x[b, j].double()[idx_c[b, j, :kept_c[b, j]].long()] for x in (K, V))
             for b in range(B) for j in range(H)}
    plain.update({(2, j): (torch.zeros(0, d).double(), torch.zeros(0, d).double()) for j in range(H)})
    scales = (1.0, 1.0) if dtype == BF else (0.125, 0.0625)
    inv_freq = mkv.mkv_rope_frequencies(rot, 10000.0)
    cur = 1
    wsa = None
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
        pos = torch.arange(n, dtype=torch.int32) + 300
        Q = torch.empty((n, H * G, d), dtype=BF, device=DEV)
        x = qkv.to(DEV)
        mkv.mkv_rope_append(x[:, :H * G], x[:, H * G:H * (G + 1)], x[:, H * (G + 1):], pos.to(DEV), inv_freq.to(DEV), k, v,
                            table, lens, start.to(DEV), Q, wsp, k_scale=scales[0], v_scale=scales[1])
        # what the pages hold now, against the plain rows: the old ones bit for bit, the new ones rotated once
        y = pu.rotate(qkv, pos, inv_freq, rot, "half", 1.0)
        kc, vc, tc, lc = pu.raw(k).cpu().view(dtype), pu.raw(v).cpu().view(dtype), table.cpu(), lens.cpu()
        half = 2.0 ** -8 if dtype == BF else 2.0 ** -4
        for (b, j), (pk, pv) in list(plain.items()):
            L = int(lc[b, j])
            assert L == len(pk) + counts[b]
            rk, rv = pu.rows_of(kc, tc[b, j], L, page), pu.rows_of(vc, tc[b, j], L, page)
            assert torch.equal(rk[:len(pk)], pk) and torch.equal(rv[:len(pv)], pv)
            t0 = int(start[b])
            for rows, want in ((rk[len(pk):], y[t0:t0 + counts[b], H * G + j] / scales[0]),
                               (rv[len(pv):], qkv[t0:t0 + counts[b], H * (G + 1) + j].double() / scales[1])):
                assert ((rows - want).abs() <= half * 1.01 * want.abs() + 2.0 ** -10 + 2.0 ** -18).all()
            plain[b, j] = (rk, rv)
        max_q, max_len = max(counts), max_pages * page
        wsa = mkv.attention_workspace_for(Q, k, table, max_q, max_len)
        O, lse = torch.empty_like(Q), torch.empty((n, H * G), device=DEV)
        mkv.mkv_paged_attention(Q, k, v, table, lens, start.to(DEV), max_q, max_len, O, wsa, k_scale=scales[0],
                                v_scale=scales[1], window=64, sinks=4, lse=lse)
        ref = pu.attention(Q.cpu(), kc, vc, tc, lc, start, page, d ** -0.5, *scales, 64, 4)
        tol, tol_lse = pu.attention_bounds(*ref, d, dtype)
        assert ((O.cpu().double() - ref[0]).abs() <= tol).all()
        assert ((lse.cpu().double() - ref[1]).abs() <= tol_lse).all()
    assert mkv.mkv_device_status(wsp) == 0 and mkv.mkv_device_status(wsa) == 0
    # every list's pages and no others are held
    held = torch.zeros(n_pages, dtype=torch.int32)
    for b in range(B + 1):
        for j in range(H):
            for p in tc[b, j, :pu.pages_of(int(lc[b, j]), page)].tolist():
                held[p] += 1
    assert torch.equal(held, refs.cpu())
