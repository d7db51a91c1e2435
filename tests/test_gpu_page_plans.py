"""The plan of page calls over its shapes: lists of more pages than a warp reads at once, updates in one launch and in
several, more heads than lanes, compactions whose plan has a list, a few or more than 32 lists per warp."""
import random

import pytest
import torch

import e2m1_util as eu
import geometric_kv_cache_gb300 as mkv
import paged_util as pu

pytestmark = pytest.mark.gpu
DEV, BF = "cuda", torch.bfloat16


# 1 list, 64 (as many as one launch takes), 65, and 120 of 40 heads
@pytest.mark.parametrize("rows,heads", [(1, 1), (8, 8), (13, 5), (3, 40)])
@pytest.mark.parametrize("kind", ["beams", "in place"])
def test_update_of_long_lists(rows, heads, kind):
    rng, page, d = random.Random(rows * heads), 16, 64
    lens = [[rng.choice([0, 5, 31 * 16 + 3, 2047, 2048, 2049, 4096, 4111]) for _ in range(heads)] for _ in range(rows)]
    lens[0][0] = 9001
    n_new = [rng.choice([0, 1, 16, 700]) for _ in range(rows)]
    parent = None if kind == "in place" else [rng.randrange(-1, rows) for _ in range(rows)]
    need = sum(pu.pages_of(x, page) for r in lens for x in r)
    n_pages, M = need + rows * heads * 47, pu.pages_of(9001 + 700, page)
    table, ln, refs = pu.random_lists(rng, lens, page, n_pages, M)
    k, v = eu.random_pages(7, n_pages, page, d)
    dev = [x.to(DEV) for x in (k, v, table, ln, refs)]
    out = dev[2:] if kind == "in place" else [torch.full_like(dev[2], 2 ** 30), torch.zeros_like(dev[3]), torch.zeros_like(dev[4])]
    ws = mkv.page_workspace_for(dev[0], dev[2])
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    mkv.mkv_page_update(*dev, *out, ws, parent=None if parent is None else i32(parent), n_new=i32(n_new))
    assert mkv.mkv_device_status(ws) == 0
    want = pu.page_update(eu.rows_of(k), eu.rows_of(v), table, ln, refs, parent, n_new, page)
    assert torch.equal(out[1].cpu(), want[1]) and torch.equal(out[2].cpu(), want[2])
    held = torch.arange(M).view(1, 1, M) < ((want[1] + page - 1) // page).unsqueeze(2)
    assert torch.equal(out[0].cpu()[held], want[0][held])
    for got, ref in ((dev[0], want[3]), (dev[1], want[4])):
        assert torch.equal(got.cpu(), eu.rows_to_pages(ref))


# lists per warp of the plan: 1 (one launch), 6 (one launch), 1 (two launches), 2, 35
@pytest.mark.parametrize("batch,heads", [(3, 1), (40, 8), (300, 8), (1025, 4), (35000, 4)])
@pytest.mark.parametrize("four", [False, True])
def test_compaction_of_any_number_of_lists(batch, heads, four):
    g = torch.Generator(device=DEV).manual_seed(batch)
    page, d, T, n = 16, 64, 35, batch * heads
    few = torch.rand((batch, heads), generator=g, device=DEV) < 0.5
    kept = torch.randint(0, T + 1, (batch, heads), generator=g, device=DEV).masked_fill(few, 0).to(torch.int32)
    lens = torch.randint(0, 40, (batch, heads), generator=g, device=DEV).to(torch.int32)
    M = 3
    pages, old = (kept + page - 1) // page, (lens + page - 1) // page
    taken, given = int(pages.sum()), int(old.sum())
    held = torch.randperm(2 * (taken + given) + 8, generator=g, device=DEV)[:given].sort().values  # the lists' old pages
    refs = torch.zeros(2 * (taken + given) + 8, dtype=torch.int32, device=DEV)
    refs[held] = 1
    at = torch.arange(M, device=DEV).view(1, 1, M)
    table = torch.full((batch, heads, M), 2 ** 30, dtype=torch.int32, device=DEV)
    table[at < old.unsqueeze(2)] = held.to(torch.int32)
    K = torch.randn((n * T, d), generator=g, device=DEV).to(BF).view(batch, heads, T, d)
    V = (K * 0.5).contiguous()
    if four:
        k, v = mkv.e2m1_pages(len(refs), page, d), mkv.e2m1_pages(len(refs), page, d)
    else:
        k, v = (torch.zeros((len(refs), page, d), dtype=BF, device=DEV) for _ in range(2))
    out, lens_out, refs_out = torch.full_like(table, 2 ** 30), torch.zeros_like(lens), torch.zeros_like(refs)
    ws = mkv.page_workspace_for(k, table)
    if four:
        mkv.mkv_page_quantize(k, v, table, lens, refs, None, kept, K, V, out, lens_out, refs_out, ws)
    else:
        mkv.mkv_page_compact(k, v, table, lens, refs, None, kept, out, lens_out, refs_out, ws, K=K, V=V)
    assert mkv.mkv_device_status(ws) == 0
    fresh = torch.nonzero(refs == 0).view(-1)[:taken]  # list after list, the lowest free pages
    want = torch.full_like(table, 2 ** 30)
    want[at < pages.unsqueeze(2)] = fresh.to(torch.int32)
    assert torch.equal(out, want) and torch.equal(lens_out, kept)
    assert int(refs_out.sum()) == taken and bool((refs_out[fresh] == 1).all())
    owner = torch.nonzero(at < pages.unsqueeze(2))  # list and place of each new page
    tok = owner[:, 2:] * page + torch.arange(page, device=DEV)
    there = tok < kept[owner[:, 0], owner[:, 1]].unsqueeze(1)
    for got, src in ((k, K), (v, V)):
        rows = src[owner[:, :1], owner[:, 1:2], tok.clamp(max=T - 1)]
        if not four:
            assert torch.equal(got[fresh][there].view(torch.int16), rows[there].view(torch.int16))
            continue
        # a row's bytes are its own: those of one list holding all of them
        m = int(there.sum())
        one = rows[there].view(1, 1, m, d).contiguous()
        p1 = mkv.e2m1_pages(pu.pages_of(m, page) + 1, page, d)
        t1 = torch.zeros((1, 1, len(p1)), dtype=torch.int32, device=DEV)
        l1, r1 = torch.zeros((1, 1), dtype=torch.int32, device=DEV), torch.zeros(len(p1), dtype=torch.int32, device=DEV)
        o1, lo1, ro1 = torch.zeros_like(t1), torch.zeros_like(l1), torch.zeros_like(r1)
        w1 = mkv.page_workspace_for(p1, t1)
        mkv.mkv_page_quantize(p1, p1.clone(), t1, l1, r1, None, torch.full_like(l1, m), one, one, o1, lo1, ro1, w1)
        assert mkv.mkv_device_status(w1) == 0
        split = lambda x: (x.view(len(x), -1)[:, :page * d // 2].view(len(x), page, d // 2),  # noqa: E731
                           x.view(len(x), -1)[:, page * d // 2:].view(len(x), page, d // 16))
        for a, b in zip(split(got[fresh]), split(p1[o1.view(-1)[:pu.pages_of(m, page)].long()])):
            assert torch.equal(a[there], b.reshape(-1, b.shape[-1])[:m])
