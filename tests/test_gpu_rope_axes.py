"""Rotary positions with several axes, and new tokens rounded into 4-bit pages: queries within their rounding of the
rotation in 64 bits, 4-bit pages byte for byte the definition's, E4M3 and bf16 pages as mkv_rope_append writes them."""
import math
import random

import pytest
import torch

import e2m1_util as eu
import geometric_kv_cache_gb300 as mkv
import paged_util as pu
from test_gpu_paged_rope import _close

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


class Step:
    """New tokens, lists and a pool; positions [n_axes, n]."""

    def __init__(self, seed, counts, H, G, d, page, dtype, n_axes=1, pad_front=0, pad_back=0, pos_max=200000):
        rng = random.Random(seed)
        start = [pad_front]
        for n in counts:
            start.append(start[-1] + n)
        self.n, self.H, self.G, self.d, self.page, self.dtype = start[-1] + pad_back, H, G, d, page, dtype
        lens = [[c + rng.choice([0, 1, page - 1, page, 3 * page + 5]) for _ in range(H)] for c in counts]
        need = sum(pu.pages_of(x, page) for r in lens for x in r)
        self.table, self.lens, _ = pu.random_lists(rng, lens, page, need + 3, pu.pages_of(max(max(r) for r in lens), page) + 1)
        self.start = torch.tensor(start, dtype=torch.int32)
        if dtype is U8:
            self.k, self.v = eu.random_pages(seed, need + 3, page, d)
        else:
            self.k, self.v = pu.random_pool(seed, need + 3, page, d, dtype)
        g = torch.Generator().manual_seed(seed)
        self.qkv = (torch.randn((self.n, H * (G + 2), d), generator=g) * 2).to(BF)
        self.positions = torch.randint(0, pos_max, (n_axes, self.n), generator=g).to(torch.int32)

    def run(self, inv_freq, axes, layout, factor, scales):
        """axes None: mkv_rope_append with the first axis."""
        hq = self.H * self.G
        raw = lambda x: x.view(U8) if x.dtype is F8 else x  # noqa: E731
        qkv, k, v = self.qkv.to(DEV), raw(self.k).to(DEV).view(self.k.dtype), raw(self.v).to(DEV).view(self.v.dtype)
        Q_out = torch.full((self.n, hq, self.d), 7.0, dtype=BF, device=DEV)
        table, lens, start, pos = (x.to(DEV) for x in (self.table, self.lens, self.start, self.positions))
        ws = mkv.page_workspace_for(k, table)
        part = (qkv[:, :hq], qkv[:, hq:hq + self.H], qkv[:, hq + self.H:])
        more = dict(layout=layout, factor=factor, k_scale=scales[0], v_scale=scales[1])
        if axes is None:
            mkv.mkv_rope_append(*part, pos[0], inv_freq.to(DEV), k, v, table, lens, start, Q_out, ws, **more)
        else:
            mkv.mkv_rope_append_axes(*part, pos, axes.to(DEV), inv_freq.to(DEV), k, v, table, lens, start, Q_out, ws, **more)
        self.status = mkv.mkv_device_status(ws)
        return Q_out.cpu(), raw(k).cpu().view(k.dtype), raw(v).cpu().view(v.dtype)

    def rotated(self, inv_freq, axes, layout, factor):
        """All heads in 64 bits, and |factor| (|x| + |y|) of each element's pair."""
        rot = 2 * inv_freq.numel()
        place = self.positions[0][:, None].expand(-1, rot // 2) if axes is None else self.positions[axes.long()].T
        a = (place.double() * inv_freq.double())[:, None]
        factor = float(torch.tensor(factor))
        i = torch.arange(rot // 2)
        lo, hi = (i, i + rot // 2) if layout == "half" else (2 * i, 2 * i + 1)
        x = self.qkv.double()
        y, size = x.clone(), torch.zeros_like(x)
        c, s = a.cos() * factor, a.sin() * factor
        y[..., lo], y[..., hi] = x[..., lo] * c - x[..., hi] * s, x[..., lo] * s + x[..., hi] * c
        size[..., lo] = size[..., hi] = abs(factor) * (x[..., lo].abs() + x[..., hi].abs())
        return y, size

    def check(self, res, inv_freq, axes, layout, factor, scales):
        Q, k, v = res
        y, size = self.rotated(inv_freq, axes, layout, factor)
        hq, H = self.H * self.G, self.H
        at = []  # (page, row, token, head) of every new token
        for b in range(len(self.start) - 1):
            t0, t1 = int(self.start[b]), int(self.start[b + 1])
            _close(Q[t0:t1], y[t0:t1, :hq], size[t0:t1, :hq], BF, "Q")
            for j in range(H):
                for t in range(t0, t1):
                    s = int(self.lens[b, j]) - (t1 - t)
                    at.append((int(self.table[b, j, s // self.page]), s % self.page, t, j))
        outside = torch.ones(self.n, dtype=torch.bool)
        outside[int(self.start[0]):int(self.start[-1])] = False
        assert (Q[outside] == 7.0).all()
        page, row, t, j = (torch.tensor(x) for x in zip(*at))
        for got, old, x, sz, scale in ((k, self.k, y[t, hq + j], size[t, hq + j], scales[0]),
                                       (v, self.v, self.qkv.double()[t, hq + H + j], 0 * size[t, hq + j], scales[1])):
            if self.dtype is U8:
                want = eu.rows_of(old).view(U8).clone()
                want[page, row] = torch.cat(eu.encode(x.float(), scale), -1)
                got = eu.rows_of(got).view(U8)
                assert torch.equal(got, want), (int((got != want).any(-1).sum()), got.shape)
                continue
            ref = x / scale
            _close(pu.raw(got)[page, row].view(got.dtype), ref.clamp(-448, 448) if self.dtype is F8 else ref, sz / scale, self.dtype, "pages")
            got, want = pu.raw(got).clone(), pu.raw(old).clone()
            got[page, row] = want[page, row] = 0
            assert torch.equal(got, want)


def _scales(dtype):
    return {BF: (1.0, 1.0), F8: (0.02, 0.3), U8: (0.013, 0.3)}[dtype]


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("d,rot,H,G,page", [(64, 64, 1, 1, 16), (64, 16, 3, 5, 16), (128, 128, 8, 4, 16), (128, 64, 2, 7, 64),
                                            (128, 48, 10, 4, 32), (128, 112, 3, 1, 16), (256, 256, 2, 3, 128), (256, 96, 1, 16, 64)])
def test_4_bit_append(layout, d, rot, H, G, page):
    inv_freq = mkv.mkv_rope_frequencies(rot, 10000.0)
    for seed, counts in enumerate([[1], [0, 3, 1, 0, 37], [1, 1, 1, 1, 1], [page + 1, 0], [300]]):
        p = Step(seed, counts, H, G, d, page, U8, pad_front=seed % 2, pad_back=2 * (seed % 2))
        res = p.run(inv_freq, None, layout, 1.25, (0.013, 0.3))
        assert p.status == 0
        p.check(res, inv_freq, None, layout, 1.25, (0.013, 0.3))


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_4_bit_append_where_values_stand_on_borders(layout):
    # position 0 turns nothing: bf16 keys stand exactly on borders of codes; so do they where a turn is nearly whole
    inv_freq = mkv.mkv_rope_frequencies(128, 10000.0)
    p = Step(1, [70, 2], 4, 2, 128, 16, U8)
    p.positions[0, :50] = 0
    grid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 0.0, -0.0, -0.25, -2.5, -5.0])
    g = torch.Generator().manual_seed(0)
    p.qkv[:, 8:] = (grid[torch.randint(0, len(grid), p.qkv[:, 8:].shape, generator=g)]
                    * torch.tensor([1.0, 1.125, 0.25])[torch.randint(0, 3, (*p.qkv[:, 8:].shape[:2], 1), generator=g)]).to(BF)
    p.qkv[3] = 0
    p.qkv[4, :, ::2] = 0
    p.qkv[5] = (p.qkv[5].double() * 2.0 ** -120).to(BF)
    p.qkv[6] = (p.qkv[6].double() * 2.0 ** 100).to(BF)
    for scales in ((1.0, 1.0), (0.3, 3.0)):
        res = p.run(inv_freq, None, layout, 1.0, scales)
        assert p.status == 0
        p.check(res, inv_freq, None, layout, 1.0, scales)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_4_bit_append_far_positions_and_fast_pairs(layout):
    p = Step(5, [64, 64], 2, 2, 128, 16, U8, pos_max=2 ** 31 - 1)
    p.positions[0, :4] = torch.tensor([0, 1, 2 ** 31 - 1, 2 ** 24 + 1], dtype=torch.int32)
    freqs = torch.exp2(torch.linspace(3, -45, 64))
    res = p.run(freqs, None, layout, 1.0, (0.013, 0.3))
    assert p.status == 0
    p.check(res, freqs, None, layout, 1.0, (0.013, 0.3))


@pytest.mark.parametrize("dtype", [BF, F8, U8])
@pytest.mark.parametrize("layout,dealt", [("half", False), ("half", True), ("interleaved", False), ("interleaved", True)])
@pytest.mark.parametrize("d,sections,H,G,page", [(64, [8], 1, 1, 16), (64, [16, 16], 3, 5, 16), (128, [16, 24, 24], 8, 4, 16),
                                                 (128, [32, 16, 16], 10, 2, 64), (128, [0, 5, 0, 19], 2, 3, 32),
                                                 (256, [1, 2, 3, 4, 5, 6, 7, 20], 2, 3, 128), (256, [44, 42, 42], 1, 16, 32)])
def test_axes(dtype, layout, dealt, d, sections, H, G, page):
    axes, scales = mkv.mkv_rope_axes(sections, dealt), _scales(dtype)
    inv_freq = mkv.mkv_rope_frequencies(2 * sum(sections), 500000.0)
    for seed, counts in enumerate([[1, 1, 1], [0, 3, 40]]):
        p = Step(seed, counts, H, G, d, page, dtype, len(sections), pad_front=seed, pad_back=seed)
        res = p.run(inv_freq, axes, layout, 1.5, scales)
        assert p.status == 0
        p.check(res, inv_freq, axes, layout, 1.5, scales)


@pytest.mark.parametrize("dtype", [BF, F8, U8])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_axes_that_agree_give_the_bits_of_one(dtype, layout):
    p = Step(2, [17, 1, 300], 4, 3, 128, 16, dtype, 3)
    p.positions[1:] = p.positions[0]
    inv_freq, scales = mkv.mkv_rope_frequencies(128, 10000.0), _scales(dtype)
    one = p.run(inv_freq, None, layout, 1.1, scales)
    for axes in (mkv.mkv_rope_axes([22, 21, 21], True), torch.zeros(64, dtype=torch.int32)):
        three = p.run(inv_freq, axes, layout, 1.1, scales)
        assert p.status == 0
        for x, y in zip(one, three):
            assert torch.equal(x.view(U8), y.view(U8))


@pytest.mark.parametrize("dtype", [BF, U8])
def test_axes_outside_are_reported_and_count_as_the_first(dtype):
    p = Step(3, [5, 2], 2, 2, 128, 16, dtype, 3)
    inv_freq, scales = mkv.mkv_rope_frequencies(64, 10000.0), _scales(dtype)
    axes = mkv.mkv_rope_axes([12, 10, 10])
    axes[5], axes[20], axes[31] = 3, -1, 2 ** 31 - 1
    res = p.run(inv_freq, axes, "half", 1.0, scales)
    assert p.status == mkv.MKV_DEV_BAD_AXIS
    axes[[5, 20, 31]] = 0
    p.check(res, inv_freq, axes, "half", 1.0, scales)


def test_invalid_lists_of_4_bit_pages_are_reported_and_left():
    p = Step(7, [4, 2, 3], 2, 2, 64, 16, U8)
    p.lens[2, 0] = 16 * p.table.shape[2] + 1
    p.lens[1, 1] = -1
    p.table[0, 0, :] = p.k.shape[0]
    inv_freq = mkv.mkv_rope_frequencies(64, 10000.0)
    Q, k, v = p.run(inv_freq, None, "half", 1.0, (0.013, 0.3))
    assert p.status == mkv.MKV_DEV_BAD_SEQ_LEN | mkv.MKV_DEV_BAD_PAGE
    y, size = p.rotated(inv_freq, None, "half", 1.0)
    _close(Q, y[:, :4], size[:, :4], BF, "Q")
    k, want = eu.rows_of(k).view(U8), eu.rows_of(p.k).view(U8).clone()
    for b, j in ((0, 1), (1, 0), (2, 1)):
        t0, t1 = int(p.start[b]), int(p.start[b + 1])
        for t in range(t0, t1):
            s = int(p.lens[b, j]) - (t1 - t)
            want[int(p.table[b, j, s // 16]), s % 16] = torch.cat(eu.encode(y[t, 4 + j].float(), 0.013), -1)
    assert torch.equal(k, want)


def test_captured_append_replays_on_new_tokens():
    p = Step(11, [1] * 6, 4, 4, 128, 16, U8, 3)
    inv_freq, axes = mkv.mkv_rope_frequencies(128, 10000.0), mkv.mkv_rope_axes([24, 20, 20], True)
    k, v, qkv, pos = (x.to(DEV) for x in (p.k, p.v, p.qkv, p.positions))
    table, lens, start, f, ax = (x.to(DEV) for x in (p.table, p.lens, p.start, inv_freq, axes))
    Q_out, ws = torch.full((6, 16, 128), 7.0, dtype=BF, device=DEV), mkv.page_workspace_for(k, table)
    call = lambda: mkv.mkv_rope_append_axes(qkv[:, :16], qkv[:, 16:20], qkv[:, 20:], pos, ax, f, k, v, table, lens,  # noqa: E731
                                            start, Q_out, ws, k_scale=0.013, v_scale=0.3)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    p.qkv = (p.qkv.double() * 1.5).to(BF)
    p.positions = p.positions.flip(1).contiguous()
    qkv.copy_(p.qkv)
    pos.copy_(p.positions)
    k.copy_(p.k)
    v.copy_(p.v)
    graph.replay()
    torch.cuda.synchronize()
    assert mkv.mkv_device_status(ws) == 0
    p.check((Q_out.cpu(), k.cpu(), v.cpu()), inv_freq, axes, "half", 1.0, (0.013, 0.3))
