"""The paged calls where they could go wrong without a sign, against the definitions in 64 bits."""
import math
import random

import pytest
import torch

import geometric_kv_cache_gb300 as mkv
import paged_util as pu
from test_gpu_paged_attention import Problem, wide

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


def _definition(p):
    """pu.attention without windows, list by list in matrices: O, lse and their bounds."""
    n, hq, d = p.Q.shape
    O, A, W = (torch.zeros((n, hq, d), dtype=torch.float64) for _ in range(3))
    lse, E = torch.full((n, hq), -math.inf, dtype=torch.float64), torch.zeros((n, hq), dtype=torch.float64)
    for b in range(p.lens.shape[0]):
        t0, t1 = int(p.start[b]), int(p.start[b + 1])
        for j in range(p.lens.shape[1]):
            L, h = int(p.lens[b, j]), slice(j * p.G, (j + 1) * p.G)
            K, V = (pu.rows_of(x, p.table[b, j], L, p.page) * s for x, s in zip((p.k, p.v), p.scales))
            hidden = torch.arange(L)[None] > (L - (t1 - t0) + torch.arange(t1 - t0))[:, None]  # [tokens, keys]
            some = ~hidden.all(1)
            if not some.any():
                continue
            hidden, q = hidden[some][:, None], p.Q[t0:t1, h].double()[some]
            x = (q @ K.T * d ** -0.5).masked_fill(hidden, -math.inf)
            w = torch.exp(x - x.amax(-1, keepdim=True)).masked_fill(hidden, 0.0)
            l = w.sum(-1, keepdim=True)
            at = torch.arange(t0, t1)[some]
            O[at, h], A[at, h], W[at, h] = w @ V / l, w @ V.abs() / l, (~hidden).double() @ V.abs() / l
            lse[at, h] = x.amax(-1) + torch.log(l[..., 0])
            E[at, h] = (q.abs() @ K.abs().T * d ** -0.5).masked_fill(hidden, 0.0).amax(-1)
    return O, lse, *pu.attention_bounds(O, lse, A, W, E, d, p.dtype)


def _check(p, O, lse, nans=False):
    """NaN exactly where the definition has it, the rest within the bounds, tokens of no row as they were."""
    ref, ref_lse, tol, tol_lse = _definition(p)
    n = int(p.start[-1])
    assert torch.equal(O[n:], torch.full_like(O[n:], 7.0)) and torch.equal(lse[n:], torch.full_like(lse[n:], 7.0))
    O, lse, ref, ref_lse, tol, tol_lse = (x[:n] for x in (O, lse, ref, ref_lse, tol, tol_lse))
    assert bool(ref_lse.isnan().any()) == nans and not bool(ref_lse.isnan().all())
    assert torch.equal(lse.isnan(), ref_lse.isnan()) and torch.equal(O.isnan(), ref.isnan())
    assert torch.equal(torch.isinf(lse), torch.isinf(ref_lse))
    fine = ~ref_lse.isnan()
    assert ((O.double() - ref).abs() <= tol)[fine].all()
    assert ((lse.double() - ref_lse).abs() <= tol_lse)[torch.isfinite(ref_lse)].all()


def _spoil(p, tokens):
    """In each of these tokens: a query of NaN, one with a single NaN, with +inf and with -inf, for every KV head."""
    for t in tokens:
        for j in range(p.lens.shape[1]):
            h = j * p.G
            p.Q[t, h] = math.nan
            p.Q[t, h + 1, p.d // 2 + 1] = math.nan
            p.Q[t, h + 2, 3] = math.inf
            p.Q[t, h + 3, p.d - 1] = -math.inf


@pytest.mark.parametrize("d,dtype", [(64, BF), (64, F8), (128, BF), (128, F8), (256, BF), (256, F8)])
@pytest.mark.parametrize("counts", [[1, 1, 1], [3, 1, 1]])
def test_queries_that_are_not_finite(d, dtype, counts):
    # lists cut into many parts, and lists of one block that one CTA has whole
    p = Problem(21, counts, [[6000, 50], [70, 3000], [60, 60]], 5, d, 16, dtype)
    _spoil(p, [0, counts[0]])
    O, lse = p.run()
    assert p.status == 0
    _check(p, O, lse, nans=True)


@pytest.mark.parametrize("d,dtype", [(64, BF), (64, F8), (128, BF), (128, F8), (256, BF), (256, F8)])
@pytest.mark.parametrize("extra", [[2500, 900], [50, 60]])
def test_chunk_form_queries_that_are_not_finite(d, dtype, extra):
    p = wide(22, [66, 20, 33, 1], extra, 4, d, 16, dtype)
    _spoil(p, [0, 40, 70, 119])
    O, lse = p.run()
    assert p.status == 0
    _check(p, O, lse, nans=True)


def _with_zero_page(p, bad):
    """The same problem with a page of zeros more, which the table entries `bad` name."""
    zero = torch.zeros((1,) + tuple(p.k.shape[1:]), dtype=torch.uint8).to(p.dtype)
    k, v = (torch.cat([pu.raw(x), pu.raw(zero)]).view(p.dtype) for x in (p.k, p.v))
    table = p.table.clone()
    for at in bad:
        table[at] = p.k.shape[0]
    return k, v, table


@pytest.mark.parametrize("dtype", [BF, F8])
@pytest.mark.parametrize("form", ["few", "chunk"])
def test_tokens_of_pages_outside_the_pool_count_as_zeros(form, dtype):
    if form == "few":
        p = Problem(23, [1, 3], [[600, 200], [90, 9]], 4, 128, 16, dtype)
        bad = [(0, 0, 2), (0, 0, 3), (0, 1, 0), (1, 0, 5)]
    else:
        p = wide(23, [70, 9, 30], [300], 8, 128, 16, dtype)
        bad = [(0, 0, 2), (0, 0, 3), (0, 5, 0), (2, 7, 20)]
    k, v, table = _with_zero_page(p, bad)
    for i, at in enumerate(bad):
        p.table[at] = [p.k.shape[0], -1, 2 ** 31 - 1, -2 ** 31][i]
    O, lse = p.run()
    assert p.status == mkv.MKV_DEV_BAD_PAGE
    p.k, p.v, p.table = k, v, table
    _check(p, O, lse)


@pytest.mark.parametrize("rows,start", [(3, [0, 5, 3, 9]), (3, [-2, 1, 3, 9]), (3, [0, 3, 6, 1000]), (3, [9, 6, 3, 0]),
                                        (3, [0, 3, 2 ** 31 - 1, -2 ** 31]), (300, None), (40, None)])
def test_rope_reports_every_bad_row_start(rows, start):
    # what is written stays within the queries and the places of the lists' new tokens
    n, H, G, d, page = 9 if start else 2 * rows, 1, 2, 64, 16
    rng = random.Random(rows)
    if start is None:  # one step back among many rows
        start = [2 * b for b in range(rows + 1)]
        start[rows - 7] = start[rows - 8] - 1
    lens = [[rng.randint(n, n + 40)] for _ in range(rows)]
    need = sum(pu.pages_of(r[0], page) for r in lens)
    table, lens, _ = pu.random_lists(rng, lens, page, need + 3, pu.pages_of(n + 40, page))
    k, v = pu.random_pool(rows, need + 3, page, d, BF)
    qkv = torch.randn((n, H * (G + 2), d), generator=torch.Generator().manual_seed(rows)).to(BF)
    positions, inv_freq = torch.arange(n, dtype=torch.int32) * 7, mkv.mkv_rope_frequencies(d, 10000.0)
    kd, vd, x = k.to(DEV), v.to(DEV), qkv.to(DEV)
    Q_out = torch.full((n, H * G, d), 7.0, dtype=BF, device=DEV)
    ws = mkv.page_workspace_for(kd, table.to(DEV))
    mkv.mkv_rope_append(x[:, :H * G], x[:, H * G:H * (G + 1)], x[:, H * (G + 1):], positions.to(DEV), inv_freq.to(DEV), kd,
                        vd, table.to(DEV), lens.to(DEV), torch.tensor(start, dtype=torch.int32, device=DEV), Q_out, ws)
    assert mkv.mkv_device_status(ws) == mkv.MKV_DEV_BAD_TOKENS
    y = pu.rotate(qkv, positions, inv_freq, d, "half", 1.0)[:, :H * G]
    near = (Q_out.cpu().double() - y).abs() <= 2.0 ** -8 * y.abs() * (1 + 2.0 ** -7) + 2.0 ** -18
    turned, left = near.all(-1).all(-1), (Q_out.cpu() == 7.0).all(-1).all(-1)
    assert (turned | left).all()
    # a token inside the range of exactly one row has its query turned, also where that range leaves [0, n]
    inside = torch.tensor([sum(start[b] <= t < start[b + 1] for b in range(rows)) for t in range(n)])
    steady = all(start[b] <= start[b + 1] for b in range(rows))
    if steady:
        assert torch.equal(turned, inside == 1)
    assert left[inside == 0].all()
    # the lists' last places, and of rows with an invalid range none
    may = torch.zeros(k.shape[:2], dtype=torch.bool)
    for b in range(rows):
        if 0 <= start[b] <= start[b + 1] <= n:
            L = int(lens[b, 0])
            for s in range(L - (start[b + 1] - start[b]), L):
                may[int(table[b, 0, s // page]), s % page] = True
    for pool, old in ((kd.cpu(), k), (vd.cpu(), v)):
        assert torch.equal(pu.raw(pool)[~may], pu.raw(old)[~may])
        if steady:  # the tokens of the valid rows are there
            assert (pu.raw(pool)[may] != pu.raw(old)[may]).any(-1).all()


def test_failed_update_without_capacity_gives_the_lists_as_they_were():
    # lists of no pages: both tables may be the same (no) memory, the lengths are not
    i32 = lambda *shape: torch.zeros(shape, dtype=torch.int32, device=DEV)  # noqa: E731
    k = torch.zeros((4, 16, 64), dtype=BF, device=DEV)
    ws = mkv.page_workspace_for(k, i32(2, 3, 0))
    for n_new, status in ((1, mkv.MKV_DEV_BAD_PARENT), (0, 0)):
        lens_out, refs_out = i32(2, 3) + 9, i32(4) + 9
        mkv.mkv_page_update(k, k.clone(), i32(2, 3, 0), i32(2, 3), i32(4) + 3, i32(2, 3, 0), lens_out, refs_out, ws,
                            n_new=i32(2) + n_new)
        assert mkv.mkv_device_status(ws) == status
        assert lens_out.tolist() == [[0] * 3] * 2 and refs_out.tolist() == [3] * 4


def test_compaction_of_no_indices_and_of_an_empty_cache_is_not_that_of_the_lists():
    # an index tensor without columns, or a cache without tokens, holds nothing to keep
    i32 = lambda *shape: torch.zeros(shape, dtype=torch.int32, device=DEV)  # noqa: E731
    k = torch.zeros((9, 16, 64), dtype=BF, device=DEV)
    v = k.clone()
    table, lens, refs = i32(1, 2, 2), i32(1, 2) + 20, i32(9)
    table.view(-1).copy_(torch.arange(4))
    refs[:4] = 1
    ws = mkv.page_workspace_for(k, table)
    empty = torch.zeros((1, 2, 0, 64), dtype=BF, device=DEV)
    for extra in (dict(idx=i32(1, 2, 0)), dict(idx=i32(1, 2, 0), K=empty, V=empty), dict(idx=None, K=empty, V=empty)):
        for kept in (1, 0):
            out = i32(1, 2, 2) - 1, i32(1, 2) - 1, i32(9) - 1
            mkv.mkv_page_compact(k, v, table, lens, refs, kept=i32(1, 2) + kept, table_out=out[0], lens_out=out[1],
                                 refs_out=out[2], workspace=ws, **extra)
            if kept:  # refused: the lists as they were
                assert mkv.mkv_device_status(ws) == mkv.MKV_DEV_BAD_N_KEEP
                assert torch.equal(out[0], table) and torch.equal(out[1], lens) and torch.equal(out[2], refs)
            else:
                assert mkv.mkv_device_status(ws) == 0
                assert int(out[1].abs().sum()) == 0 and int(out[2].abs().sum()) == 0


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("new", [1, 48])
def test_weights_far_below_the_largest_add_up_next_to_e4m3_values(d, new):
    # 12 keys (one for every warp of a CTA) score 26 powers of two above the 2^18 others, whose values are 1 where theirs
    # are 0: the others together weigh 2^-8, although each alone is below fp16's smallest number relative to the largest.
    # (152 lists, a CTA each, that share their pages.)
    n, page, lists, top = 2 ** 18, 128, 152, 12
    k = torch.zeros((n // page, page, d), dtype=torch.uint8).to(F8)
    v = torch.ones((n // page, page, d)).to(F8)
    for i in range(top):
        k[16 * i // page, 16 * i % page, 0] = 1.0
        pu.raw(v)[16 * i // page, 16 * i % page] = 0
    Q = torch.zeros((new * lists, 1, d), dtype=BF)
    Q[:, 0, 0] = 1.0
    dev = lambda x: pu.raw(x).to(DEV).view(x.dtype) if x.dtype in pu.CODES else x.to(DEV)  # noqa: E731
    kd, vd, Qd = dev(k), dev(v), dev(Q)
    table = torch.arange(n // page, dtype=torch.int32, device=DEV).expand(lists, 1, -1).contiguous()
    lens = torch.full((lists, 1), n, dtype=torch.int32, device=DEV)
    start = torch.arange(lists + 1, dtype=torch.int32, device=DEV) * new
    O, lse = torch.empty_like(Qd), torch.empty((new * lists, 1), device=DEV)
    ws = mkv.attention_workspace_for(Qd, kd, table, new, n)
    assert (ws.numel() > 152 * 2 * 100 * (4 * d + 8)) == (new > 1)  # the form for chunks, the one for few rows
    scale = 26 * math.log(2)
    mkv.mkv_paged_attention(Qd, kd, vd, table, lens, start, new, n, O, ws, scale=scale, lse=lse)
    assert mkv.mkv_device_status(ws) == 0
    small = (n - top - new + 1 + torch.arange(new, dtype=torch.float64)) * 2.0 ** -26  # visible keys but the large ones
    want = (small / (top + small)).repeat(lists)
    # scale * log2(e) is an fp32 number: 26 is off by at most 26 x 2^-23, a weight by 2^-18.7 relative, 2^x by 2^-22.
    # Such a weight times 2^7 lies next to 2^-19, a multiple of fp16's smallest step 2^-24, and rounds to it. At most
    # 2^18 / 16 additions of equal positive numbers in fp32: 2^-10. The sum of weights may lose all the small ones, each
    # below half a step of it: small / top. Then bf16's half step.
    off = 2.0 ** -18 + 2.0 ** -10 + (small / top).repeat(lists)
    tol = want * (off + 2.0 ** -8 * (1 + 2.0 ** -8))
    err = (O[:, 0].double().cpu() - want[:, None]).abs()
    assert (err <= tol[:, None]).all(), (float(O[0, 0, 0]), float(want[0]))
    exact = scale + torch.log(top + small).repeat(lists)
    assert ((lse[:, 0].double().cpu() - exact).abs() <= off + 2.0 ** -18).all()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("new", [1, 48])
def test_scores_of_many_powers_of_two_stay_finite_next_to_e4m3_values(d, new):
    # Scores up to 2^28 and beyond, of which fp32 holds no fractions: the weights mean little then, but nothing turns into
    # NaN, and up to 2^28 O stays inside the range of the values.
    n, page = 3000, 16
    k, v = pu.random_pool(d + new, pu.pages_of(n, page), page, d, F8)
    dev = lambda x: pu.raw(x).to(DEV).view(x.dtype) if x.dtype in pu.CODES else x.to(DEV)  # noqa: E731
    kd, vd = dev(k), dev(v)
    table = torch.arange(len(k), dtype=torch.int32, device=DEV).expand(16, 1, -1).contiguous()
    lens, start = torch.full((16, 1), n, dtype=torch.int32, device=DEV), torch.arange(17, dtype=torch.int32, device=DEV) * new
    top = v.double().flatten(0, 1)[:n].abs().amax(0)
    for e in (12, 16, 18, 20):
        Q = (torch.randn((16 * new, 32, d), generator=torch.Generator().manual_seed(e)) * 2.0 ** e).to(BF)
        O, lse = torch.empty_like(dev(Q)), torch.empty(Q.shape[:2], device=DEV)
        ws = mkv.attention_workspace_for(O, kd, table, new, n)
        assert (ws.numel() > 152 * 2 * 100 * (4 * d + 8)) == (new > 1)
        mkv.mkv_paged_attention(dev(Q), kd, vd, table, lens, start, new, n, O, ws, scale=1.0, lse=lse)
        assert mkv.mkv_device_status(ws) == 0
        assert bool(lse.isfinite().all()) and bool(O.isfinite().all())
        # Below 2^28 a score in log2 units is below 2^28.53, where an fp32 step is 32, so the reference point is off by at
        # most 16 and the largest weight, 2^7 to 2^15 above it, lies in [2^-9, 2^31]: it saturates, which only makes O
        # smaller, or is a normal fp16 number. O is then an average of the values with weights off by 2^-11 relative, or
        # 2^-25 absolute against a sum of at least 2^-9, and is rounded to bf16.
        K = kd.double().flatten(0, 1)[:n]
        most = torch.cat([(x.double() @ K.T).abs().amax(1) for x in dev(Q).flatten(0, 1).split(4096)])
        inside = (most < 2.0 ** 28).cpu()
        assert e > 16 or bool(inside.all())
        slack = 2.0 ** -8 + 2.0 ** -10 + n * 2.0 ** -16
        assert (O.flatten(0, 1).double().cpu().abs() <= top * (1 + slack))[inside].all()


def test_update_over_pages_outside_the_pool():
    # what the header promises: such an entry is carried over and not counted, and a tail that would have been copied from
    # it has a new page whose contents stay
    rng = random.Random(61)
    page, M, P = 16, 5, 40
    table, lens, refs = pu.random_lists(rng, [[33, 20], [33, 20], [40, 5]], page, P, M)
    k, v = pu.random_pool(61, P, page, 64, BF)
    bad = {(1, 0, 0): P, (1, 0, 2): -3, (2, 1, 0): 2 ** 31 - 1}
    # the same lists with three pages more in the bad ones' place
    more, n = table.clone(), P
    for at in bad:
        more[at] = n
        n += 1
    pad = lambda x: torch.cat([x, torch.zeros((3,) + tuple(x.shape[1:]), dtype=x.dtype)])  # noqa: E731
    refs_more = pad(refs)
    refs_more[P:] = 9
    want = pu.page_update(pad(k), pad(v), more, lens, refs_more, [0, 1, 1], [1, 1, 1], page)
    for at, x in bad.items():
        table[at] = x
    g = [x.to(DEV) for x in (k, v, table, lens, refs)]
    out = [g[2].clone(), torch.zeros_like(g[3]), torch.zeros_like(g[4])]
    ws = mkv.page_workspace_for(g[0], g[2])
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    mkv.mkv_page_update(*g, *out, ws, parent=i32([0, 1, 1]), n_new=i32([1, 1, 1]))
    assert mkv.mkv_device_status(ws) == mkv.MKV_DEV_BAD_PAGE
    carried = want[0].clone()
    for i, x in enumerate(bad.values()):
        carried[want[0] == P + i] = x
    live = torch.arange(M)[None, None] < ((want[1] + page - 1) // page)[..., None]
    assert torch.equal(out[0].cpu()[live], carried[live])
    assert torch.equal(out[1].cpu(), want[1]) and torch.equal(out[2].cpu(), want[2][:P])
    new = int(want[0][2, 0, 2])  # the tail of row 1's first list, which row 2 could not copy
    assert new < P
    for pool, old, w in ((g[0], k, want[3]), (g[1], v, want[4])):
        expect = w[:P].clone()
        expect[new] = old[new]
        assert torch.equal(pu.raw(pool).cpu(), pu.raw(expect))


def test_compaction_over_pages_outside_the_pool():
    rng = random.Random(67)
    page, M, P = 16, 4, 30
    table, lens, refs = pu.random_lists(rng, [[50, 17], [33, 64]], page, P, M)
    k, v = pu.random_pool(67, P, page, 64, BF)
    kept = torch.tensor([[20, 17], [33, 7]], dtype=torch.int32)
    idx = torch.stack([torch.stack([torch.randperm(max(int(lens[b, j]), 33), generator=torch.Generator().manual_seed(b))[:33]
                                    for j in range(2)]) for b in range(2)]).to(torch.int32)
    for b in range(2):
        for j in range(2):
            idx[b, j, :kept[b, j]] %= int(lens[b, j])
    bad = {(0, 0, 1): P, (1, 1, 3): -1}
    more, n = table.clone(), P
    for at in bad:
        more[at] = n
        n += 1
    mark = torch.full((2, page, 64), 77.0, dtype=BF)
    refs_more = torch.cat([refs, torch.full((2,), 9, dtype=torch.int32)])
    want = pu.page_compact(torch.cat([k, mark]), torch.cat([v, mark]), more, lens, refs_more, idx, kept, page)
    for at, x in bad.items():
        table[at] = x
    g = [x.to(DEV) for x in (k, v, table, lens, refs)]
    out = [g[2].clone(), torch.zeros_like(g[3]), torch.zeros_like(g[4])]
    ws = mkv.page_workspace_for(g[0], g[2])
    mkv.mkv_page_compact(*g, idx.to(DEV), kept.to(DEV), *out, ws)
    assert mkv.mkv_device_status(ws) == mkv.MKV_DEV_BAD_PAGE
    live = torch.arange(M)[None, None] < ((kept + page - 1) // page)[..., None]
    assert torch.equal(out[0].cpu()[live], want[0][live])
    assert torch.equal(out[1].cpu(), kept) and torch.equal(out[2].cpu(), want[2][:P])
    skipped = 0
    for pool, old, w in ((g[0], k, want[3]), (g[1], v, want[4])):
        expect = torch.where(w[:P] == 77.0, old, w[:P])  # rows that have no source stay
        skipped += int((w[:P] == 77.0).any(-1).sum())
        assert torch.equal(pu.raw(pool).cpu(), pu.raw(expect))
    assert skipped > 0


@pytest.mark.parametrize("d,dtype", [(64, BF), (64, F8), (256, BF), (256, F8)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (70, 5)])
def test_chunk_form_pages_of_128_tokens(d, dtype, window, sinks):
    # at 256 dims a page spans two blocks of keys
    p = wide(24, [40, 20, 33, 1], [0, 64, 129, 700], 4, d, 128, dtype)
    O, lse = p.run(window, sinks)
    assert p.status == 0
    p.check(O, lse, window, sinks)


@pytest.mark.parametrize("dtype", [BF, F8])
@pytest.mark.parametrize("rows", [19, 38])
def test_ragged_lists_as_many_as_the_sms(rows, dtype):
    # 152 and 304 lists whose lengths differ fourfold: cuts at tiles' ends would make parts of uneven length
    rng = random.Random(rows)
    p = Problem(25, [1] * rows, [[rng.randint(300, 1300) for _ in range(8)] for _ in range(rows)], 2, 64, 16, dtype)
    a, b = p.run(), p.run()
    assert p.status == 0
    _check(p, *a)
    assert torch.equal(a[0].view(torch.int16), b[0].view(torch.int16)) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("d,dtype", [(64, BF), (128, BF), (128, F8), (256, BF)])
@pytest.mark.parametrize("counts,heads", [([608], 8), ([40, 300, 1, 77, 210], 9)])
def test_fresh_prompts(counts, heads, d, dtype):
    # lists of the new tokens alone: the tiles of a list see ever more keys
    p = wide(26, counts, [0], 8, d, 16, dtype, heads=heads)
    a, b = p.run(), p.run()
    assert p.status == 0
    _check(p, *a)
    assert torch.equal(a[0].view(torch.int16), b[0].view(torch.int16)) and torch.equal(a[1], b[1])


def test_two_streams_with_a_workspace_each():
    ps = [Problem(27, [1, 1, 1], [[5000, 50], [70, 3000], [60, 900]], 4, 128, 16, BF),
          wide(28, [66, 20, 33, 1], [2500, 900], 4, 128, 16, BF),
          Problem(29, [3, 1], [[9000, 50], [70, 7000]], 4, 128, 16, F8)]
    dev = lambda x: pu.raw(x).to(DEV).view(x.dtype) if x.dtype in pu.CODES else x.to(DEV)  # noqa: E731
    runs = []
    for p in ps:
        Q, k, v, table, lens, start = (dev(x) for x in (p.Q, p.k, p.v, p.table, p.lens, p.start))
        runs.append((p, (Q, k, v, table, lens, start, p.max_q, p.max_len), torch.empty_like(Q),
                     torch.empty(Q.shape[:2], device=DEV), mkv.attention_workspace_for(Q, k, table, p.max_q, p.max_len),
                     torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(8):
        for p, args, O, lse, ws, stream in runs:
            mkv.mkv_paged_attention(*args, O, ws, k_scale=p.scales[0], v_scale=p.scales[1], lse=lse, stream=stream)
    torch.cuda.synchronize()
    for p, args, O, lse, ws, stream in runs:
        alone = p.run()
        assert mkv.mkv_device_status(ws) == 0
        assert torch.equal(O.cpu().view(torch.int16), alone[0].view(torch.int16)) and torch.equal(lse.cpu(), alone[1])
        _check(p, *alone)


@pytest.mark.parametrize("dtype,new", [(BF, 1), (F8, 1), (BF, 48), (F8, 48)])
def test_lists_beyond_64k_tokens(dtype, new):
    # (the reference in fp64 on the GPU: the lists are long, the rows few)
    n, d, page, G = 140001, 64, 64, 2
    rng = random.Random(new)
    pages = pu.pages_of(n, page)
    g = torch.Generator().manual_seed(new)
    ids = torch.randperm(pages, generator=g).to(torch.int32)
    k, v = pu.random_pool(new, pages, page, d, dtype)
    pu.raw(k)[int(ids[-1]), n % page:] = pu.raw(v)[int(ids[-1]), n % page:] = -1 if dtype == BF else 255
    Q = torch.randn((new, G, d), generator=g).to(BF)
    dev = lambda x: pu.raw(x).to(DEV).view(x.dtype) if x.dtype in pu.CODES else x.to(DEV)  # noqa: E731
    kd, vd, Qd, table = dev(k), dev(v), dev(Q), ids.view(1, 1, -1).to(DEV)
    lens, start = torch.tensor([[n]], dtype=torch.int32, device=DEV), torch.tensor([0, new], dtype=torch.int32, device=DEV)
    O, lse = torch.empty_like(Qd), torch.empty((new, G), device=DEV)
    ws = mkv.attention_workspace_for(Qd, kd, table, new, n)
    mkv.mkv_paged_attention(Qd, kd, vd, table, lens, start, new, n, O, ws, lse=lse)
    assert mkv.mkv_device_status(ws) == 0
    K, V = (x[table[0, 0].long()].view(-1, d)[:n].view(dtype).double() for x in (pu.raw(kd), pu.raw(vd)))
    at, E = torch.arange(n, device=DEV), torch.zeros((new, G), dtype=torch.float64)
    ref, A, W = (torch.zeros((new, G, d), dtype=torch.float64) for _ in range(3))
    ref_lse = torch.zeros((new, G), dtype=torch.float64)
    for t in range(new):
        q = Qd[t].double()
        x = (q @ K.T * d ** -0.5).masked_fill(at > n - new + t, -math.inf)
        w = torch.exp(x - x.amax(1, keepdim=True))
        l = w.sum(1, keepdim=True)
        seen = (at <= n - new + t).double()
        ref[t], A[t], W[t] = (w @ V / l).cpu(), (w @ V.abs() / l).cpu(), ((seen @ V.abs())[None] / l).cpu()
        ref_lse[t] = torch.logsumexp(x, 1).cpu()
        E[t] = ((q.abs() @ K.abs().T) * d ** -0.5).amax(1).cpu()
    tol, tol_lse = pu.attention_bounds(ref, ref_lse, A, W, E, d, dtype)
    # beyond 2^13 keys the sum's fp32 error grows past the bound's 2^-18: (keys / 8) 2^-24 for both sums
    tol = tol + 2 * (n / 8) * 2.0 ** -24 * A
    assert ((O.cpu().double() - ref).abs() <= tol).all()
    assert ((lse.cpu().double() - ref_lse).abs() <= tol_lse + (n / 8) * 2.0 ** -24).all()
