"""4-bit pages written and moved: codes and scales are those of the definition, byte for byte -- from a contiguous cache
(mkv_page_quantize, into E4M3 pages too), from new tokens (mkv_rope_append) -- and pages are forked, copied and compacted
as others are."""
import math
import random

import pytest
import torch

import e2m1_util as eu
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


def _bytes(x):
    return x.view(torch.uint8)


def _quantize(K, V, idx, kept, page, k_scale, v_scale, dtype=torch.uint8, seq_lens=None, spare=3, old=None):
    """Runs mkv_page_quantize into a pool of all ones; the pool's rows (as paged_util takes them), lists and status."""
    B, H, T, d = K.shape
    M = max(1, max(pu.pages_of(int(x), page) for x in kept.flatten()), 0 if old is None else old[0].shape[-1])
    need = sum(pu.pages_of(int(x), page) for x in kept.flatten())
    table, lens, refs = old if old is not None else (torch.zeros((B, H, M), dtype=torch.int32),
                                                     torch.zeros((B, H), dtype=torch.int32),
                                                     torch.zeros(need + spare, dtype=torch.int32))
    width = d * 9 // 16 if dtype is torch.uint8 else d
    k = torch.full((refs.numel(), page, width), 255, dtype=torch.uint8, device=DEV).view(dtype)
    v = k.clone()
    out, lens_out, refs_out = (torch.full(x.shape, 77, dtype=torch.int32, device=DEV) for x in (table, lens, refs))
    ws = mkv.page_workspace_for(k, out)
    mkv.mkv_page_quantize(k, v, table.to(DEV), lens.to(DEV), refs.to(DEV), None if idx is None else idx.to(DEV), kept.to(DEV),
                          K.to(DEV), V.to(DEV), out, lens_out, refs_out, ws, k_scale=k_scale, v_scale=v_scale,
                          seq_lens=None if seq_lens is None else seq_lens.to(DEV))
    status = mkv.mkv_device_status(ws)
    rows = [eu.rows_of(x.cpu()) if dtype is torch.uint8 else _bytes(x).cpu().view(F8) for x in (k, v)]
    return rows, out.cpu(), lens_out.cpu(), refs_out.cpu(), status, (table, lens, refs)


def _rounded(X, scale, dtype):
    """The contiguous cache as rows of the pool."""
    if dtype is F8:
        inv = torch.tensor(1.0 / float(torch.tensor(scale)), dtype=torch.float64).float()
        return (X.float() * inv).clamp(-448, 448).to(F8)
    return torch.cat(eu.encode(X.float(), scale), -1).view(F8)


def _check_quantize(K, V, idx, kept, page, k_scale, v_scale, dtype=torch.uint8, seq_lens=None, old=None):
    (k, v), table, lens, refs, status, lists = _quantize(K, V, idx, kept, page, k_scale, v_scale, dtype, seq_lens, old=old)
    assert status == 0
    ones = torch.full(k.shape, 255, dtype=torch.uint8).view(F8)
    want = pu.page_compact(ones, ones, *lists, idx, kept, page, _rounded(K, k_scale, dtype), _rounded(V, v_scale, dtype))
    for b in range(K.shape[0]):
        for j in range(K.shape[1]):
            n = pu.pages_of(int(kept[b, j]), page)
            assert torch.equal(table[b, j, :n], want[0][b, j, :n])
            assert (table[b, j, n:] == 77).all()
    assert torch.equal(lens, want[1]) and torch.equal(refs, want[2])
    for got, ref in ((k, want[3]), (v, want[4])):
        assert torch.equal(_bytes(got), _bytes(ref)), int((_bytes(got) != _bytes(ref)).sum())


def _cache(seed, B, H, T, d, sigma=0.7):
    k, v = pu.random_pool(seed, B * H, T, d, BF, sigma)
    return k.view(B, H, T, d), v.view(B, H, T, d)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("dtype", [torch.uint8, F8])
@pytest.mark.parametrize("page,T,kept", [(16, 70, [[70, 0, 1], [16, 17, 33]]), (128, 300, [[299, 128, 129], [5, 300, 0]]),
                                         (32, 1, [[1, 0, 1], [1, 1, 1]])])
def test_quantize(d, dtype, page, T, kept):
    K, V = _cache(d + T, 2, 3, T, d)
    kept = torch.tensor(kept, dtype=torch.int32)
    n = int(kept.max()) + 2
    g = torch.Generator().manual_seed(T)
    idx = torch.randint(0, T, (2, 3, n), generator=g).to(torch.int32)  # any order, the same one twice
    _check_quantize(K, V, idx, kept, page, 0.013, 0.3, dtype)
    _check_quantize(K, V, None, kept, page, 1.0, 7.0, dtype)


def test_quantize_ragged_rows_and_old_lists():
    K, V = _cache(3, 3, 2, 90, 128)
    rng = random.Random(1)
    old = pu.random_lists(rng, [[20, 0], [33, 16], [0, 1]], 16, 40, 6)
    lens = torch.tensor([90, 7, 0], dtype=torch.int32)
    kept = torch.tensor([[45, 90], [7, 3], [0, 0]], dtype=torch.int32)
    idx = torch.stack([torch.stack([torch.randperm(max(int(x), 1))[:1].repeat(90) for _ in range(2)]) for x in lens]).to(torch.int32)
    _check_quantize(K, V, idx, kept, 16, 0.02, 0.02, seq_lens=lens, old=old)


def test_quantize_borders_zeros_and_extremes():
    """Every border between codes and between scales met exactly, groups of zeros, numbers that vanish or saturate."""
    d = 128
    rows = []
    for s in (1.0, 1.125, 1.875, 0.0625, 2.0 ** -6, 448.0):  # group maxima 6 s: the scale is s
        ties = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0]
        rows.append([x * s for x in ties] + [-x * s for x in ties[:7]] + [6 * s])
    for a, b in ((1.0, 1.125), (1.125, 1.25), (15 * 2.0 ** -9, 2.0 ** -5), (2.0 ** -9, 2.0 ** -8), (0.0, 2.0 ** -9)):
        rows.append([3 * (a + b)] + [0.0, -0.0] * 7 + [-(a + b)])  # a maximum of 6 times the middle of two scales
    rows += [[0.0] * 16, [-0.0] * 16, [1e-30] * 16, [2.0 ** -133] * 16, [3e38] * 8 + [-3e38] * 8, [1e5, -1.0] * 8]
    x = torch.tensor(rows + [[0.0] * 16] * (-len(rows) % 8)).reshape(-1, d).to(BF)
    x = x.view(1, 1, -1, d)
    kept = torch.tensor([[x.shape[2]]], dtype=torch.int32)
    for k_scale, v_scale in ((1.0, 1.0), (0.3, 4.0), (2.0 ** -100, 2.0 ** 100)):
        _check_quantize(x, -x.flip(2), None, kept, 16, k_scale, v_scale)


def test_quantize_nan_makes_its_group_nan_and_infinity_saturates():
    K, V = _cache(5, 1, 1, 16, 64)
    K[0, 0, 3, 20] = math.nan
    V[0, 0, 5, 63] = math.inf
    V[0, 0, 6, 0] = -math.inf
    kept = torch.tensor([[16]], dtype=torch.int32)
    (k, v), table, *_, status, _ = _quantize(K, V, None, kept, 16, 1.0, 1.0)
    assert status == 0
    at = int(table[0, 0, 0])
    split = lambda rows: (_bytes(rows)[at][:, :32].contiguous(), _bytes(rows)[at][:, 32:].contiguous())  # noqa: E731
    x, want = eu.decode(*split(k)), eu.decode(*eu.encode(K[0, 0].float().nan_to_num(0.0), 1.0))
    assert x[3, 16:32].isnan().all() and int(x.isnan().sum()) == 16
    assert torch.equal(x[~x.isnan()], want[~x.isnan()])
    x = eu.decode(*split(v))
    assert float(x[5, 63]) == 6 * 448 and float(x[6, 0]) == -6 * 448 and torch.isfinite(x).all()


def test_quantize_reports_what_compaction_reports():
    K, V = _cache(7, 1, 2, 40, 64)
    kept = torch.tensor([[20, 41]], dtype=torch.int32)
    _, out, lens, refs, status, lists = _quantize(K, V, None, kept, 16, 1.0, 1.0)
    assert status == mkv.MKV_DEV_BAD_N_KEEP and torch.equal(refs, lists[2]) and torch.equal(lens, lists[1])
    kept = torch.tensor([[20, 40]], dtype=torch.int32)
    _, _, _, refs, status, lists = _quantize(K, V, None, kept, 16, 1.0, 1.0, spare=-1)
    assert status == mkv.MKV_DEV_NO_PAGES and torch.equal(refs, lists[2])
    idx = torch.zeros((1, 2, 40), dtype=torch.int32)
    idx[0, 1, 3] = 40
    (k, _), table, *_, status, _ = _quantize(K, V, idx, kept, 16, 1.0, 1.0)
    assert status == mkv.MKV_DEV_BAD_INDEX
    assert (_bytes(k)[int(table[0, 1, 0]), 3] == 255).all()  # its place stays what it was


# ------------------------------------------------------------- moves of pages --

@pytest.mark.parametrize("d,page", [(64, 16), (64, 128), (128, 16), (128, 64), (256, 32), (256, 16)])
def test_update_of_4_bit_pages(d, page):
    rng = random.Random(d + page)
    lens = [[rng.choice([0, 1, page - 1, page, page + 1, 3 * page + 5]) for _ in range(3)] for _ in range(9)]
    parent = [0, 0, 1, -1, 4, 1, 8, 8, 8]
    n_new = [1, 5, 0, 9, page, 1, 2, page + 3, 0]
    need = sum(pu.pages_of(x, page) for r in lens for x in r)
    n_pages, M = need + 9 * 3 * 4, 8
    table, ln, refs = pu.random_lists(rng, lens, page, n_pages, M)
    k, v = eu.random_pages(d, n_pages, page, d)
    dev = [x.to(DEV) for x in (k, v, table, ln, refs)]
    out, lens_out, refs_out = torch.full_like(dev[2], 2 ** 30), torch.zeros_like(dev[3]), torch.zeros_like(dev[4])
    ws = mkv.page_workspace_for(dev[0], dev[2])
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    mkv.mkv_page_update(*dev, out, lens_out, refs_out, ws, parent=i32(parent), n_new=i32(n_new))
    assert mkv.mkv_device_status(ws) == 0
    want = pu.page_update(eu.rows_of(k), eu.rows_of(v), table, ln, refs, parent, n_new, page)
    assert torch.equal(lens_out.cpu(), want[1]) and torch.equal(refs_out.cpu(), want[2])
    for b in range(9):
        for j in range(3):
            n = pu.pages_of(int(want[1][b, j]), page)
            assert torch.equal(out.cpu()[b, j, :n], want[0][b, j, :n])
    for got, ref in ((dev[0], want[3]), (dev[1], want[4])):
        assert torch.equal(got.cpu(), eu.rows_to_pages(ref))


@pytest.mark.parametrize("d,page", [(64, 16), (64, 128), (128, 16), (128, 32), (256, 64), (256, 16)])
@pytest.mark.parametrize("indices", [True, False])
def test_compaction_of_4_bit_pages(d, page, indices):
    rng = random.Random(d + page)
    lens = [[rng.choice([0, 1, 16, page + 1, 3 * page + 5, 400]) for _ in range(3)] for _ in range(4)]
    kept = torch.tensor([[rng.randint(0, x) for x in r] for r in lens], dtype=torch.int32)
    M = pu.pages_of(400, page) + 1
    n_pages = 2 * sum(pu.pages_of(x, page) for r in lens for x in r) + 2
    table, ln, refs = pu.random_lists(rng, lens, page, n_pages, M)
    idx = torch.full((4, 3, 400), -5, dtype=torch.int32)
    for b in range(4):
        for j in range(3):
            n = int(kept[b, j])
            idx[b, j, :n] = torch.tensor([rng.randrange(lens[b][j]) for _ in range(n)], dtype=torch.int32)
    idx = idx if indices else None
    k, v = eu.random_pages(d, n_pages, page, d)
    dev = [x.to(DEV) for x in (k, v, table, ln, refs)]
    out, lens_out, refs_out = torch.full_like(dev[2], 2 ** 30), torch.zeros_like(dev[3]), torch.zeros_like(dev[4])
    ws = mkv.page_workspace_for(dev[0], dev[2])
    mkv.mkv_page_compact(*dev, None if idx is None else idx.to(DEV), kept.to(DEV), out, lens_out, refs_out, ws)
    assert mkv.mkv_device_status(ws) == 0
    want = pu.page_compact(eu.rows_of(k), eu.rows_of(v), table, ln, refs, idx, kept, page)
    assert torch.equal(lens_out.cpu(), want[1]) and torch.equal(refs_out.cpu(), want[2])
    for got, ref in ((dev[0], want[3]), (dev[1], want[4])):
        assert torch.equal(got.cpu(), eu.rows_to_pages(ref))
