"""mkv_rope_append against the rotation in 64 bits: both pair layouts, part of the head, far positions, bf16 and E4M3
pages, fused projections, padding and rows without new tokens."""
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


def _problem(seed, counts, H, G, d, page, dtype, pad_front=0, pad_back=0, pos_max=200000):
    rng = random.Random(seed)
    B = len(counts)
    start = [pad_front]
    for n in counts:
        start.append(start[-1] + n)
    n = start[-1] + pad_back
    lens = [[c + rng.choice([0, 1, page - 1, page, 3 * page + 5]) for _ in range(H)] for c in counts]
    max_pages = pu.pages_of(max(max(r) for r in lens), page) + 1
    need = sum(pu.pages_of(x, page) for r in lens for x in r)
    table, lens, _ = pu.random_lists(rng, lens, page, need + 3, max_pages)
    k, v = pu.random_pool(seed, need + 3, page, d, dtype)
    g = torch.Generator().manual_seed(seed)
    qkv = (torch.randn((n, H * (G + 2), d), generator=g) * 2).to(BF)
    positions = torch.randint(0, pos_max, (n,), generator=g).to(torch.int32)
    return dict(start=torch.tensor(start, dtype=torch.int32), table=table, lens=lens, k=k, v=v, qkv=qkv, n=n,
                positions=positions)


def _run(p, H, G, rot, layout, factor=1.0, scales=(1.0, 1.0), inv_freq=None, in_place=False):
    d = p["k"].shape[-1]
    dev = lambda x: pu.raw(x).to(DEV).view(x.dtype) if x.dtype in pu.CODES else x.to(DEV)  # noqa: E731
    qkv, k, v = dev(p["qkv"]), dev(p["k"]), dev(p["v"])
    Q, K, V = qkv[:, :H * G], qkv[:, H * G:H * (G + 1)], qkv[:, H * (G + 1):]
    if in_place:
        Q = Q.contiguous()
    Q_out = Q if in_place else torch.full((p["n"], H * G, d), 7.0, dtype=BF, device=DEV)
    inv_freq = mkv.mkv_rope_frequencies(rot, 10000.0) if inv_freq is None else inv_freq
    ws = mkv.page_workspace_for(k, dev(p["table"]))
    mkv.mkv_rope_append(Q, K, V, dev(p["positions"]), inv_freq.to(DEV), k, v, dev(p["table"]), dev(p["lens"]),
                        dev(p["start"]), Q_out, ws, layout=layout, factor=factor, k_scale=scales[0], v_scale=scales[1])
    return Q_out.cpu(), pu.raw(k).cpu().view(k.dtype), pu.raw(v).cpu().view(v.dtype), mkv.mkv_device_status(ws), inv_freq


def _close(got, want, size, dtype, what):
    """One rounding of a value that is off by the fp32 arithmetic: sine, cosine and their products with x and y, each
    2^-23 of |factor| (|x| + |y|) (`size`), times four; half a step of the type relative to the value (bf16 2^-8, E4M3
    2^-4), E4M3 at least half its smallest step, 2^-10."""
    half = 2.0 ** -8 if dtype == BF else 2.0 ** -4
    tol = half * want.abs() * (1 + 2.0 ** -7) + 4 * 2.0 ** -23 * size + (0 if dtype == BF else 2.0 ** -10) + 1e-38
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), (what, int(bad.sum()), got.double()[bad][:4], want[bad][:4])


def _check(p, res, H, G, rot, layout, factor, scales, skip_rows=()):
    Q_out, k, v, status, inv_freq = res
    page, d, n = p["k"].shape[1], p["k"].shape[2], p["n"]
    x = p["qkv"].double()
    y = pu.rotate(x, p["positions"], inv_freq, rot, layout, factor)
    r2 = rot // 2
    size = x.abs().clone()
    i = torch.arange(r2)
    lo, hi = (i, i + r2) if layout == "half" else (2 * i, 2 * i + 1)
    size[..., lo] = size[..., hi] = abs(factor) * (x[..., lo].abs() + x[..., hi].abs())
    k_want, v_want = pu.raw(p["k"]).clone(), pu.raw(p["v"]).clone()
    for b in range(len(p["start"]) - 1):
        t0, t1 = int(p["start"][b]), int(p["start"][b + 1])
        _close(Q_out[t0:t1], y[t0:t1, :H * G], size[t0:t1, :H * G], BF, "Q")
        for j in range(H):
            for t in range(t0, t1):
                if (b, j) in skip_rows:
                    continue
                s = int(p["lens"][b, j]) - (t1 - t)
                at = (int(p["table"][b, j, s // page]), s % page)
                for pool, want, src, sz, sc in ((k, k_want, y[t, H * G + j], size[t, H * G + j], scales[0]),
                                                (v, v_want, x[t, H * (G + 1) + j], 0 * size[t, 0], scales[1])):
                    ref = src / sc
                    if pool.dtype == F8:
                        ref = ref.clamp(-448, 448)
                    _close(pool[at], ref, sz / sc, pool.dtype, ("pages", b, j, t))
                    pu.raw(pool)[at] = 0
                    want[at] = 0
    # every other row, and the tokens that belong to no row, as they were
    assert torch.equal(pu.raw(k), k_want) and torch.equal(pu.raw(v), v_want)
    outside = torch.ones(n, dtype=torch.bool)
    outside[int(p["start"][0]):int(p["start"][-1])] = False
    return Q_out[outside]


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("d,rot,H,G,page,dtype", [(64, 64, 1, 1, 16, BF), (64, 16, 3, 5, 16, F8), (128, 128, 8, 4, 16, BF),
                                                  (128, 64, 2, 7, 64, F8), (128, 48, 10, 4, 32, BF), (256, 256, 2, 3, 128, BF),
                                                  (256, 96, 1, 16, 64, F8)])
def test_rope_append(layout, d, rot, H, G, page, dtype):
    scales = (1.0, 1.0) if dtype == BF else (0.02, 0.3)  # 0.02: keys beyond 448 saturate
    for seed, counts in enumerate([[1], [0, 3, 1, 0, 37], [1, 1, 1, 1, 1], [page + 1, 0]]):
        p = _problem(seed, counts, H, G, d, page, dtype, pad_front=seed % 2, pad_back=2 * (seed % 2))
        res = _run(p, H, G, rot, layout, 1.25, scales)
        assert res[3] == 0
        rest = _check(p, res, H, G, rot, layout, 1.25, scales)
        assert torch.equal(rest, torch.full_like(rest, 7.0))


def test_far_positions_and_fast_pairs():
    p = _problem(5, [64, 64], 2, 2, 128, 16, BF, pos_max=2 ** 31 - 1)
    p["positions"][:4] = torch.tensor([0, 1, 2 ** 31 - 1, 2 ** 24 + 1], dtype=torch.int32)
    freqs = torch.exp2(torch.linspace(3, -45, 64))  # faster than a radian per position down to almost none
    for layout in ("half", "interleaved"):
        res = _run(p, 2, 2, 128, layout, 1.0, inv_freq=freqs)
        assert res[3] == 0
        _check(p, res, 2, 2, 128, layout, 1.0, (1.0, 1.0))


@pytest.mark.parametrize("rows", [33, 1100])
def test_many_rows(rows):
    rng = random.Random(rows)
    counts = [rng.choice([0, 0, 1, 2]) for _ in range(rows)]
    p = _problem(10, counts, 1, 1, 64, 16, BF, pad_front=2, pad_back=3)
    res = _run(p, 1, 1, 64, "half")
    assert res[3] == 0
    _check(p, res, 1, 1, 64, "half", 1.0, (1.0, 1.0))


def test_queries_in_place():
    p = _problem(6, [3, 20], 2, 4, 128, 16, BF)
    res = _run(p, 2, 4, 64, "half", 1.0, in_place=True)
    assert res[3] == 0
    _check(p, res, 2, 4, 64, "half", 1.0, (1.0, 1.0))


def test_invalid_lists_are_reported_and_left():
    p = _problem(7, [4, 2, 3], 2, 2, 64, 16, BF)
    p["lens"][0, 1] = 3                       # fewer tokens than the row brings
    p["lens"][2, 0] = 16 * p["table"].shape[2] + 1
    p["lens"][2, 1] = -2 ** 31
    p["lens"][1, 0] = 2 ** 31 - 1
    p["lens"][1, 1] = -1
    res = _run(p, 2, 2, 64, "half")
    assert res[3] == mkv.MKV_DEV_BAD_SEQ_LEN
    # the tokens that do have a place in the short list are written: compare the other lists alone
    t = p["table"][0, 1, 0]
    for pool, old in ((res[1], p["k"]), (res[2], p["v"])):
        pu.raw(pool)[t] = pu.raw(old)[t]
    _check(p, res, 2, 2, 64, "half", 1.0, (1.0, 1.0), skip_rows={(0, 1), (2, 0), (2, 1), (1, 0), (1, 1)})
    p = _problem(8, [4, 2], 2, 2, 64, 16, BF)
    last = pu.pages_of(int(p["lens"][1, 1]), 16) - 1
    p["lens"][1, 1] = last * 16 + 10  # both new tokens inside the last page
    p["table"][1, 1, last] = p["k"].shape[0]
    res = _run(p, 2, 2, 64, "half")
    assert res[3] == mkv.MKV_DEV_BAD_PAGE
    _check(p, res, 2, 2, 64, "half", 1.0, (1.0, 1.0), skip_rows={(1, 1)})


@pytest.mark.parametrize("start", [[0, 5, 3, 9], [-2, 1, 3, 9], [0, 3, 6, 1000], [9, 6, 3, 0]])
def test_bad_row_starts_write_inside_the_buffers_only(start):
    p = _problem(9, [3, 3, 3], 1, 2, 64, 16, BF)
    p["start"] = torch.tensor(start, dtype=torch.int32)
    p["lens"].clamp_(min=9)
    res = _run(p, 1, 2, 64, "half")
    # no token stands in a decreasing or outside range without a report, unless no token is in any range
    assert res[3] in (0, mkv.MKV_DEV_BAD_TOKENS, mkv.MKV_DEV_BAD_SEQ_LEN | mkv.MKV_DEV_BAD_TOKENS,
                      mkv.MKV_DEV_BAD_SEQ_LEN, mkv.MKV_DEV_BAD_PAGE, mkv.MKV_DEV_BAD_PAGE | mkv.MKV_DEV_BAD_TOKENS)
