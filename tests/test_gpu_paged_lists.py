"""Page lists on the GPU against Python integers: fork, copy, free and extend (mkv_page_update) and compaction in pages
(mkv_page_compact). Everything is compared bit for bit."""
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


class State:
    """One problem on the CPU, and its copy on the GPU with output buffers of a marker value."""

    def __init__(self, seed, B, H, page, d, dtype, t_max, spare, max_pages=None, lens=None):
        rng = random.Random(seed)
        lens = lens or [[rng.choice([0, 1, page - 1, page, page + 1, rng.randint(0, t_max)]) for _ in range(H)]
                        for _ in range(B)]
        lens = [[min(x, t_max) for x in r] for r in lens]
        self.page, self.rng = page, rng
        need = sum(pu.pages_of(x, page) for r in lens for x in r)
        self.table, self.lens, self.refs = pu.random_lists(rng, lens, page, need + spare,
                                                           max_pages or pu.pages_of(t_max, page) + 4)
        self.k, self.v = pu.random_pool(seed, need + spare, page, d, dtype)

    def gpu(self):
        self.g = {n: getattr(self, n).to(DEV) for n in ("table", "lens", "refs")}
        self.g["k"], self.g["v"] = pu.raw(self.k).to(DEV).view(self.k.dtype), pu.raw(self.v).to(DEV).view(self.v.dtype)
        self.g["ws"] = mkv.page_workspace_for(self.g["k"], self.g["table"])
        self.g["out"] = [self.g["table"].clone(), torch.full_like(self.g["lens"], -5), torch.full_like(self.g["refs"], -5)]
        return self.g

    def update(self, parent=None, n_new=None, out=None):
        g = self.g
        out = out or g["out"]
        mkv.mkv_page_update(g["k"], g["v"], g["table"], g["lens"], g["refs"], *out, g["ws"],
                            parent=None if parent is None else torch.tensor(parent, dtype=torch.int32, device=DEV),
                            n_new=None if n_new is None else torch.tensor(n_new, dtype=torch.int32, device=DEV))
        return out

    def compact(self, idx, kept, K=None, V=None, seq_lens=None, out=None):
        g = self.g
        out = out or g["out"]
        dev = lambda x: None if x is None else x.to(DEV)  # noqa: E731
        mkv.mkv_page_compact(g["k"], g["v"], g["table"], g["lens"], g["refs"], dev(idx), dev(kept), *out, g["ws"],
                             K=K, V=V, seq_lens=dev(seq_lens))
        return out

    def same(self, out, want):
        assert mkv.mkv_device_status(self.g["ws"]) == 0
        for name, a, b in zip(("table", "lens", "refs"), out, want):
            assert torch.equal(a.cpu(), b), name
        for name, a, b in (("k", self.g["k"], want[3]), ("v", self.g["v"], want[4])):
            assert torch.equal(pu.raw(a).cpu(), pu.raw(b)), name


def _parents(rng, B, kind):
    if kind == "none":
        return None
    if kind == "beams":  # everything from a few rows
        some = [rng.randrange(B) for _ in range(2)]
        return [rng.choice(some) for _ in range(B)]
    if kind == "free":
        return [-1] * B
    if kind == "shift":
        return [(b + 1) % B for b in range(B)]
    return [rng.choice([b, b, -1, rng.randrange(B)]) for b in range(B)]


@pytest.mark.parametrize("d,dtype,page", [(64, F8, 16), (128, BF, 16), (128, BF, 128), (256, BF, 32), (256, F8, 64)])
@pytest.mark.parametrize("kind", ["none", "mixed", "beams", "free", "shift"])
def test_update_equals_the_plain_lists(d, dtype, page, kind):
    for seed, (B, H) in enumerate([(1, 1), (3, 2), (9, 5), (17, 40), (40, 3)]):
        s = State(100 * seed + page, B, H, page, d, dtype, 5 * page + 3, B * H * 8)
        parent = _parents(s.rng, B, kind)
        n_new = [s.rng.choice([0, 1, 1, page, 2 * page + 3]) for _ in range(B)] if seed % 2 == 0 else None
        want = pu.page_update(s.k, s.v, s.table, s.lens, s.refs, parent, n_new, page)
        s.gpu()
        s.same(s.update(parent, n_new), want)


def test_update_over_many_pages_and_rows():
    # several chunks of the pool and of the rows, few free pages among many held ones
    s = State(7, 300, 8, 16, 64, BF, 200, 9000)
    parent = _parents(s.rng, 300, "mixed")
    n_new = [s.rng.choice([0, 1, 17]) for _ in range(300)]
    want = pu.page_update(s.k, s.v, s.table, s.lens, s.refs, parent, n_new, 16)
    s.gpu()
    s.same(s.update(parent, n_new), want)


def test_update_in_place_and_step_by_step():
    # extension in place, then forks between two buffers, over several steps
    s = State(11, 6, 3, 16, 128, BF, 60, 400, max_pages=12)
    g = s.gpu()
    cpu = (s.table, s.lens, s.refs, s.k, s.v)
    two = [[g["table"], g["lens"], g["refs"]], [x.clone() for x in g["out"]]]
    for step in range(12):
        a, b = two
        if step % 3 == 2:
            parent = [s.rng.choice([i, s.rng.randrange(6)]) for i in range(6)]
        else:
            parent = None
        n_new = [s.rng.choice([1, 1, 7]) for _ in range(6)]
        n_new = [0 if max(cpu[1][parent[i] if parent else i].tolist()) + n_new[i] > 12 * 16 else n_new[i] for i in range(6)]
        cpu = pu.page_update(cpu[3], cpu[4], cpu[0], cpu[1], cpu[2], parent, n_new, 16)
        g["table"], g["lens"], g["refs"] = a
        if parent is None:
            s.update(None, n_new, out=a)  # all three in place
        else:
            s.update(parent, n_new, out=b)
            two = [b, a]
        cur = two[0]
        assert mkv.mkv_device_status(g["ws"]) == 0
        assert torch.equal(cur[1].cpu(), cpu[1]) and torch.equal(cur[2].cpu(), cpu[2])
        live = torch.arange(12)[None, None] < (-(-cpu[1] // 16))[..., None]
        assert torch.equal(cur[0].cpu()[live], cpu[0][live])
        assert torch.equal(pu.raw(g["k"]).cpu(), pu.raw(cpu[3])) and torch.equal(pu.raw(g["v"]).cpu(), pu.raw(cpu[4]))


def _unchanged(s, out, bit):
    assert mkv.mkv_device_status(s.g["ws"]) == bit
    assert torch.equal(out[1].cpu(), s.lens) and torch.equal(out[2].cpu(), s.refs)
    ok = (s.lens >= 0) & (s.lens <= s.table.shape[2] * s.page)
    live = torch.arange(s.table.shape[2])[None, None] < (-(-s.lens // s.page) * ok)[..., None]
    assert torch.equal(out[0].cpu()[live], s.table[live])
    assert torch.equal(pu.raw(s.g["k"]).cpu(), pu.raw(s.k)) and torch.equal(pu.raw(s.g["v"]).cpu(), pu.raw(s.v))


def test_invalid_device_arguments_change_nothing():
    mk = lambda spare=3: State(13, 5, 4, 16, 64, BF, 70, spare, lens=[[33, 20, 0, 70]] * 5)  # noqa: E731
    s = mk()
    s.gpu()
    s.g["out"][0].fill_(-1)
    _unchanged(s, s.update([0, 0, 0, 3, 4]), mkv.MKV_DEV_NO_PAGES)  # 2 forks need 6 pages of the 3
    for parent, n_new in (([0, 1, 5, 3, 4], None), ([0, -2, 2, 3, 4], None), (None, [0, -1, 0, 0, 0]),
                          (None, [0, 0, 0, 0, 500]), (None, [2 ** 31 - 1, 0, 0, 0, 0])):
        s = mk(100)
        s.gpu()
        s.g["out"][0].fill_(-1)
        _unchanged(s, s.update(parent, n_new), mkv.MKV_DEV_BAD_PARENT)
    for bad in (-1, 2 ** 31 - 1, 16 * mk().table.shape[2] + 1):
        s = mk(100)
        s.lens[2, 1] = bad
        s.gpu()
        s.g["out"][0].fill_(-1)
        _unchanged(s, s.update([0, 0, 2, 2, 4], [1] * 5), mkv.MKV_DEV_BAD_SEQ_LEN)
    kept = torch.tensor([[10, 3, 0, 7]] * 5, dtype=torch.int32)
    idx = torch.zeros((5, 4, 10), dtype=torch.int32)
    for bad in (-1, 11, 2 ** 31 - 1):
        s = mk(100)
        s.gpu()
        s.g["out"][0].fill_(-1)
        k2 = kept.clone()
        k2[3, 3] = bad
        _unchanged(s, s.compact(idx, k2), mkv.MKV_DEV_BAD_N_KEEP)
    s = mk(100)  # without indices: more tokens than the list has
    s.gpu()
    k2 = torch.zeros((5, 4), dtype=torch.int32)
    k2[1, 0] = 34
    _unchanged(s, s.compact(None, k2), mkv.MKV_DEV_BAD_N_KEEP)


def test_failed_update_in_place_leaves_the_lists():
    s = State(17, 4, 2, 16, 64, BF, 40, 0, lens=[[16, 5]] * 4)
    g = s.gpu()
    s.update(None, [1, 1, 1, 1], out=[g["table"], g["lens"], g["refs"]])
    assert mkv.mkv_device_status(g["ws"]) == mkv.MKV_DEV_NO_PAGES
    for n in ("table", "lens", "refs"):
        assert torch.equal(g[n].cpu(), getattr(s, n))


def test_pages_outside_the_pool_are_reported_and_skipped():
    s = State(19, 3, 2, 16, 64, BF, 60, 60, lens=[[33, 20]] * 3)
    good = s.table.clone()
    s.table[1, 0, 0] = s.refs.numel()
    s.table[1, 0, 2] = -3
    g = s.gpu()
    out = s.update([0, 1, 1], [0, 0, 0])
    assert mkv.mkv_device_status(g["ws"]) == mkv.MKV_DEV_BAD_PAGE
    assert out[1].cpu().tolist() == [[33, 20]] * 3
    s.table = good
    assert torch.equal(out[0][0].cpu(), good[0])
    s.table[1, 0, 0] = 2 ** 30
    g = s.gpu()
    s.compact(torch.arange(20, dtype=torch.int32).expand(3, 2, 20).contiguous(), torch.full((3, 2), 20, dtype=torch.int32))
    assert mkv.mkv_device_status(g["ws"]) == mkv.MKV_DEV_BAD_PAGE


@pytest.mark.parametrize("d,dtype,page", [(64, F8, 16), (128, BF, 16), (128, F8, 64), (256, BF, 128)])
@pytest.mark.parametrize("source", ["pages", "cache"])
def test_compaction_equals_the_plain_lists(d, dtype, page, source):
    for seed, (B, H) in enumerate([(1, 1), (2, 3), (5, 33)]):
        t_max = 4 * page + 7
        s = State(31 * seed + d, B, H, page, d, dtype, t_max, B * H * 6)
        if source == "cache":
            lens = [s.rng.randint(0, t_max) for _ in range(B)]
            T = torch.tensor(lens)[:, None].expand(B, H)
        else:
            T = s.lens
        kept = torch.tensor([[s.rng.choice([0, min(1, int(T[b, j])), s.rng.randint(0, int(T[b, j])), int(T[b, j])])
                              for j in range(H)] for b in range(B)], dtype=torch.int32)
        idx = torch.full((B, H, t_max), 2 ** 30, dtype=torch.int32)
        for b in range(B):
            for j in range(H):
                if kept[b, j]:
                    idx[b, j, :kept[b, j]] = torch.tensor(sorted(s.rng.sample(range(int(T[b, j])), int(kept[b, j]))))
        K = V = None
        if source == "cache":
            K, V = pu.random_pool(seed + 1, B * H, t_max, d, dtype)
            K, V = K.view(B, H, t_max, d), V.view(B, H, t_max, d)
        want = pu.page_compact(s.k, s.v, s.table, s.lens, s.refs, idx, kept, page, K, V)
        s.gpu()
        dev = lambda x: None if x is None else pu.raw(x).to(DEV).view(x.dtype)  # noqa: E731
        s.same(s.compact(idx, kept, dev(K), dev(V), torch.tensor(lens, dtype=torch.int32) if source == "cache" else None),
               want)


def test_compaction_without_indices_any_order_and_repeats():
    s = State(41, 2, 2, 16, 128, BF, 50, 30, lens=[[50, 17], [16, 1]])
    kept = torch.tensor([[33, 17], [0, 1]], dtype=torch.int32)
    want = pu.page_compact(s.k, s.v, s.table, s.lens, s.refs, None, kept, 16)
    s.gpu()
    s.same(s.compact(None, kept), want)
    s = State(43, 1, 2, 16, 128, BF, 50, 30, lens=[[50, 17]])
    idx = torch.tensor([[[49, 0, 0, 3] + [7] * 60, [16, 2, 2, 1] + [0] * 60]], dtype=torch.int32)
    kept = torch.tensor([[64, 3]], dtype=torch.int32)
    want = pu.page_compact(s.k, s.v, s.table, s.lens, s.refs, idx, kept, 16)
    s.gpu()
    s.same(s.compact(idx, kept), want)


@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_compaction_of_many_lists_mostly_empty(page):
    # runs of empty lists longer than a warp, single tokens, one long list: the copying warps' runs begin and end anywhere
    for seed in range(3):
        rng = random.Random(seed)
        lens = [[0 if rng.random() < 0.8 else rng.choice([1, page, 2 * page + 1]) for _ in range(7)] for _ in range(90)]
        lens[rng.randrange(90)][3] = 40 * page + 5
        s = State(seed, 90, 7, page, 64, F8, 41 * page, sum(pu.pages_of(x, page) for r in lens for x in r) + 2, lens=lens)
        kept = torch.where(torch.rand((90, 7), generator=torch.Generator().manual_seed(seed)) < 0.3, 0, s.lens)
        want = pu.page_compact(s.k, s.v, s.table, s.lens, s.refs, None, kept, page)
        s.gpu()
        s.same(s.compact(None, kept), want)


def test_compaction_reports_indices_outside_and_copies_the_others():
    s = State(47, 1, 2, 16, 64, BF, 50, 30, lens=[[50, 17]])
    idx = torch.tensor([[[1, 50, 3], [-1, 16, 2 ** 30]]], dtype=torch.int32)
    kept = torch.full((1, 2), 3, dtype=torch.int32)
    fixed = torch.tensor([[[1, 1, 3], [16, 16, 16]]], dtype=torch.int32)
    want = pu.page_compact(s.k, s.v, s.table, s.lens, s.refs, fixed, kept, 16)
    g = s.gpu()
    before = pu.raw(g["k"]).cpu()
    out = s.compact(idx, kept)
    assert mkv.mkv_device_status(g["ws"]) == mkv.MKV_DEV_BAD_INDEX
    for a, b in zip(out, want):
        assert torch.equal(a.cpu(), b)
    for x, w in ((g["k"], want[3]), (g["v"], want[4])):
        for j, rows in ((0, [0, 2]), (1, [1])):
            p = int(out[0][0, j, 0])
            assert torch.equal(pu.raw(x)[p].cpu()[rows], pu.raw(w)[p][rows])
    p = int(out[0][0, 0, 0])
    assert torch.equal(pu.raw(g["k"])[p, 1].cpu(), before[p, 1])  # the refused token's row as it was


def test_two_lists_may_share_pages_and_a_held_back_page_is_not_taken():
    s = State(53, 2, 1, 16, 64, BF, 40, 8, lens=[[32], [0]])
    s.table[1, 0, :2] = s.table[0, 0, :2]
    s.lens[1, 0] = 32
    s.refs[s.table[0, 0, :2].long()] = 2
    free = [p for p in range(s.refs.numel()) if s.refs[p] == 0]
    s.refs[free[0]] = 1  # the program's own
    want = pu.page_compact(s.k, s.v, s.table, s.lens, s.refs, None, torch.tensor([[20], [32]], dtype=torch.int32), 16)
    assert int(want[2][s.table[0, 0, 0]]) == 0 and int(want[2][free[0]]) == 1
    s.gpu()
    s.same(s.compact(None, torch.tensor([[20], [32]], dtype=torch.int32)), want)


def test_captured_update_replays_on_new_lists_beside_another_stream():
    s = State(59, 8, 4, 16, 128, BF, 100, 300, max_pages=16)
    g = s.gpu()
    n_new = torch.ones(8, dtype=torch.int32, device=DEV)
    parent = torch.arange(8, dtype=torch.int32, device=DEV)
    side = torch.cuda.Stream()

    def call(stream=None):
        mkv.mkv_page_update(g["k"], g["v"], g["table"], g["lens"], g["refs"], *g["out"], g["ws"], parent=parent,
                            n_new=n_new, stream=stream)

    with torch.cuda.stream(side):
        call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for step in range(3):
        pick = [s.rng.choice([b, s.rng.randrange(8), -1]) for b in range(8)]
        parent.copy_(torch.tensor(pick, dtype=torch.int32))
        k, v = (pu.raw(g[x]).cpu().view(BF) for x in ("k", "v"))
        want = pu.page_update(k, v, s.table, s.lens, s.refs, pick, [1] * 8, 16)
        graph.replay()
        torch.cuda.synchronize()
        assert mkv.mkv_device_status(g["ws"]) == 0
        live = torch.arange(16)[None, None] < (-(-want[1] // 16))[..., None]
        assert torch.equal(g["out"][0].cpu()[live], want[0][live])
        assert torch.equal(g["out"][1].cpu(), want[1]) and torch.equal(g["out"][2].cpu(), want[2])
        assert torch.equal(pu.raw(g["k"]).cpu(), pu.raw(want[3]))


def test_no_lists_and_no_pages():
    ws = torch.zeros(1 << 16, dtype=torch.uint8, device=DEV)
    k = torch.zeros((4, 16, 64), dtype=BF, device=DEV)
    i32 = lambda *shape: torch.zeros(shape, dtype=torch.int32, device=DEV)  # noqa: E731
    refs, out = i32(4) + 3, i32(4)
    mkv.mkv_page_update(k, k.clone(), i32(0, 2, 3), i32(0, 2), refs, i32(0, 2, 3), i32(0, 2), out, ws)
    assert out.tolist() == [3] * 4
    e = torch.zeros((0, 16, 64), dtype=BF, device=DEV)
    lens = i32(2, 2) + 9
    mkv.mkv_page_update(e, e.clone(), i32(2, 2, 3), i32(2, 2), i32(0), i32(2, 2, 3), lens, i32(0), ws)
    assert lens.sum() == 0 and mkv.mkv_device_status(ws) == 0
    mkv.mkv_page_update(e, e.clone(), i32(2, 2, 0), i32(2, 2), i32(0), i32(2, 2, 0), lens, i32(0), ws,
                        n_new=i32(2) + 1)
    assert mkv.mkv_device_status(ws) == mkv.MKV_DEV_BAD_PARENT
