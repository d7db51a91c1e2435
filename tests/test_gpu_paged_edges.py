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


def _check_with_nans(p, O, lse):
    """NaN exactly where the definition has it, the rest within the bounds."""
    ref, ref_lse, A, W, E = pu.attention(p.Q, p.k, p.v, p.table, p.lens, p.start, p.page, p.d ** -0.5, *p.scales)
    n = int(p.start[-1])
    assert bool(ref_lse[:n].isnan().any()) and not bool(ref_lse[:n].isnan().all())
    assert torch.equal(lse[:n].isnan(), ref_lse[:n].isnan())
    assert torch.equal(O[:n].isnan(), ref[:n].isnan())
    tol, tol_lse = pu.attention_bounds(ref, ref_lse, A, W, E, p.d, p.dtype)
    fine = ~ref_lse[:n].isnan()
    assert ((O[:n].double() - ref[:n]).abs() <= tol[:n])[fine].all()
    assert torch.equal(torch.isinf(lse[:n]), torch.isinf(ref_lse[:n]))
    some = fine & torch.isfinite(ref_lse[:n])
    assert ((lse[:n].double() - ref_lse[:n]).abs() <= tol_lse[:n])[some].all()


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
    _check_with_nans(p, O, lse)


@pytest.mark.parametrize("d,dtype", [(64, BF), (64, F8), (128, BF), (128, F8), (256, BF), (256, F8)])
@pytest.mark.parametrize("extra", [[2500, 900], [50, 60]])
def test_chunk_form_queries_that_are_not_finite(d, dtype, extra):
    p = wide(22, [66, 20, 33, 1], extra, 4, d, 16, dtype)
    _spoil(p, [0, 40, 70, 119])
    O, lse = p.run()
    assert p.status == 0
    _check_with_nans(p, O, lse)


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
