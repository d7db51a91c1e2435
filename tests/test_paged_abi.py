"""Host-side checks of the paged-cache calls (no GPU needed): bad arguments are refused before anything is enqueued,
workspace sizes and the rotary frequencies are those of their definitions."""
import ctypes
import math

import pytest
import torch

import geometric_kv_cache_gb300 as mkv

vp = ctypes.c_void_p
A = 1 << 20  # a fake, aligned device address: no call below may touch it
BIG = 1 << 40
OK, ARG, UNS, WS = mkv.MKV_OK, mkv.MKV_ERR_INVALID_ARG, mkv.MKV_ERR_UNSUPPORTED, mkv.MKV_ERR_WORKSPACE


def _pool(n_pages=100, page_size=16, head_dim=128, dtype=0, k=A, v=2 * A):
    return mkv.MkvPagePool(n_pages, page_size, head_dim, dtype, k, v)


def _lists(batch=4, heads=8, max_pages=10, table=3 * A, lens=4 * A):
    return mkv.MkvPageLists(batch, heads, max_pages, table, lens)


def _out(**k):
    return _lists(**dict(dict(table=5 * A, lens=6 * A), **k))


SIZES = [
    (dict(pool=_pool(n_pages=-1)), ARG), (dict(pool=_pool(page_size=0)), ARG), (dict(pool=_pool(head_dim=0)), ARG),
    (dict(pool=_pool(page_size=8)), UNS), (dict(pool=_pool(page_size=24)), UNS), (dict(pool=_pool(page_size=256)), UNS),
    (dict(pool=_pool(head_dim=96)), UNS), (dict(pool=_pool(dtype=2)), UNS),
    (dict(pool=_pool(n_pages=(1 << 26) + 1)), UNS), (dict(lists=_lists(max_pages=(1 << 26) + 1)), UNS),
    (dict(lists=_lists(batch=65537)), UNS), (dict(lists=_lists(batch=65536, heads=257)), UNS),
    (dict(lists=_lists(batch=-1)), ARG), (dict(lists=_lists(heads=-1)), ARG), (dict(lists=_lists(max_pages=-1)), ARG),
]
POINTERS = [
    (dict(pool=_pool(k=A + 8)), ARG), (dict(pool=_pool(v=0)), ARG), (dict(pool=_pool(v=A)), ARG),
    (dict(lists=_lists(table=0)), ARG), (dict(lists=_lists(lens=0)), ARG), (dict(lists=_lists(table=3 * A + 2)), ARG),
    (dict(ws=0), WS), (dict(ws=A + 16), WS), (dict(ws_bytes=200), WS),
]


def _update(pool=_pool(), lists=_lists(), out=None, refs=7 * A, parent=8 * A, n_new=9 * A, refs_out=10 * A, ws=11 * A,
            ws_bytes=BIG):
    out = out or _out(batch=lists.batch, heads=lists.heads, max_pages=lists.max_pages)
    return mkv.load().mkv_page_update(pool, lists, vp(refs), vp(parent), vp(n_new), out, vp(refs_out), vp(ws), ws_bytes,
                                      None)


@pytest.mark.parametrize("kwargs,status", SIZES + POINTERS + [
    (dict(refs=0), ARG), (dict(refs_out=0), ARG), (dict(refs=7 * A + 1), ARG), (dict(parent=8 * A + 2), ARG),
    (dict(n_new=9 * A + 2), ARG), (dict(out=_out(batch=3)), ARG), (dict(out=_out(max_pages=11)), ARG),
    (dict(out=_lists()), ARG),                       # in place with a parent
    (dict(out=_lists(lens=6 * A), parent=0), ARG),   # half in place
    (dict(out=_lists(table=5 * A), parent=0), ARG),
    (dict(out=_out(table=0)), ARG),
])
def test_update_refusals(kwargs, status):
    assert _update(**kwargs) == status


def _compact(pool=_pool(), lists=_lists(), out=None, refs=7 * A, idx=8 * A, idx_stride=100, kept=9 * A, K=0, V=0,
             t_max=0, seq_lens=0, refs_out=10 * A, ws=11 * A, ws_bytes=BIG):
    out = out or _out(batch=lists.batch, heads=lists.heads, max_pages=lists.max_pages)
    return mkv.load().mkv_page_compact(pool, lists, vp(refs), vp(idx), idx_stride, vp(kept), vp(K), vp(V), t_max,
                                       vp(seq_lens), out, vp(refs_out), vp(ws), ws_bytes, None)


@pytest.mark.parametrize("kwargs,status", SIZES + POINTERS + [
    (dict(kept=0), ARG), (dict(idx=8 * A + 1), ARG), (dict(idx_stride=-1), ARG), (dict(K=A), ARG), (dict(V=A), ARG),
    (dict(K=A + 8, V=A, t_max=4), ARG), (dict(K=A, V=A, t_max=-1), ARG), (dict(K=A, V=A, t_max=(1 << 30) + 1), UNS),
    (dict(out=_lists()), ARG), (dict(seq_lens=A + 1), ARG),
])
def test_compact_refusals(kwargs, status):
    assert _compact(**kwargs) == status


def _tokens(n=50, q_heads=32, q_start=12 * A):
    return mkv.MkvNewTokens(n, q_heads, q_start)


def _rope(Q=A, qs=4096, K=2 * A, ks=1024, V=3 * A, vs=1024, tokens=_tokens(), pos=4 * A, freq=5 * A, rot=128, layout=0,
          factor=1.0, Q_out=6 * A, pool=_pool(k=7 * A, v=8 * A), lists=_lists(), k_scale=1.0, v_scale=1.0, ws=11 * A,
          ws_bytes=BIG):
    return mkv.load().mkv_rope_append(vp(Q), qs, vp(K), ks, vp(V), vs, tokens, vp(pos), vp(freq), rot, layout, factor,
                                      vp(Q_out), pool, lists, k_scale, v_scale, vp(ws), ws_bytes, None)


@pytest.mark.parametrize("kwargs,status", SIZES + POINTERS + [
    (dict(Q=0), ARG), (dict(Q=A + 8), ARG), (dict(qs=4095), ARG), (dict(qs=4088), ARG), (dict(ks=1023), ARG),
    (dict(vs=8), ARG), (dict(K=0), ARG), (dict(V=0), ARG), (dict(Q_out=0), ARG), (dict(Q_out=A, qs=6144), ARG),
    (dict(tokens=_tokens(n=-1)), ARG), (dict(tokens=_tokens(q_heads=20)), ARG), (dict(tokens=_tokens(q_heads=0)), ARG),
    (dict(tokens=_tokens(q_heads=1032)), UNS), (dict(tokens=_tokens(q_start=0)), ARG), (dict(pos=0), ARG),
    (dict(freq=0), ARG), (dict(freq=5 * A + 2), ARG), (dict(rot=0), ARG), (dict(rot=8), ARG), (dict(rot=72), ARG),
    (dict(rot=144), ARG), (dict(layout=2), ARG), (dict(factor=float("nan")), ARG), (dict(k_scale=0.5), ARG),
    (dict(pool=_pool(dtype=1), k_scale=0.0), ARG), (dict(pool=_pool(dtype=1), v_scale=-1.0), ARG),
    (dict(pool=_pool(dtype=1), v_scale=float("inf")), ARG),
    (dict(tokens=_tokens(n=0), Q=0, K=0, V=0, Q_out=0), OK), (dict(lists=_lists(batch=0)), OK),
])
def test_rope_refusals(kwargs, status):
    assert _rope(**kwargs) == status


def _attend(Q=A, qs=4096, tokens=_tokens(), max_q=8, pool=_pool(k=7 * A, v=8 * A), lists=_lists(), max_len=160,
            scale=0.1, k_scale=1.0, v_scale=1.0, window=0, sinks=0, O=2 * A, os_=4096, lse=3 * A, ws=11 * A, ws_bytes=BIG):
    return mkv.load().mkv_paged_attention(vp(Q), qs, tokens, max_q, pool, lists, max_len, scale, k_scale, v_scale,
                                          window, sinks, vp(O), os_, vp(lse), vp(ws), ws_bytes, None)


@pytest.mark.parametrize("kwargs,status", [(dict(max_len=0) | k if "lists" in k else k, s) for k, s in SIZES] + POINTERS + [
    (dict(Q=0), ARG), (dict(O=0), ARG), (dict(O=A), ARG), (dict(Q=A + 2), ARG), (dict(qs=4092), ARG), (dict(os_=4088), ARG),
    (dict(pool=_pool(n_pages=0)), ARG),
    (dict(lse=3 * A + 2), ARG), (dict(max_q=-1), ARG), (dict(max_q=(1 << 20) + 1), UNS), (dict(max_len=161), ARG),
    (dict(max_len=-1), ARG), (dict(window=-1), ARG), (dict(sinks=-1), ARG), (dict(scale=float("inf")), ARG),
    (dict(k_scale=2.0), ARG), (dict(pool=_pool(dtype=1), k_scale=0.0), ARG), (dict(tokens=_tokens(q_heads=20)), ARG),
    (dict(tokens=_tokens(q_start=0)), ARG), (dict(tokens=_tokens(n=0), Q=0, O=0), OK), (dict(max_q=0), OK),
    (dict(lists=_lists(heads=0)), OK),
    (dict(lists=_lists(batch=65536, heads=256), tokens=_tokens(q_heads=256), max_q=1 << 20, max_len=0), UNS),
])
def test_attention_refusals(kwargs, status):
    assert _attend(**kwargs) == status


def test_workspace_sizes():
    size = lambda **k: mkv.load().mkv_page_workspace_size(k.get("pool", _pool()), k.get("lists", _lists()))  # noqa: E731
    for kwargs, _ in SIZES:
        assert size(**kwargs) == 0
        assert mkv.load().mkv_attention_workspace_size(kwargs.get("pool", _pool()), kwargs.get("lists", _lists()),
                                                       _tokens(), 1, 0) == 0
    assert 0 < size() < size(pool=_pool(n_pages=10 ** 6), lists=_lists(max_pages=1000))
    att = lambda max_q, max_len: mkv.load().mkv_attention_workspace_size(  # noqa: E731
        _pool(), _lists(max_pages=1000), _tokens(), max_q, max_len)
    assert att(1, 16001) == 0 and att(0, 16000) == 256
    assert 0 < att(1, 1) <= att(1, 16000)
    need = att(1, 16000)
    shape = dict(lists=_lists(max_pages=1000), max_q=1, max_len=16000)
    assert _attend(**shape, ws_bytes=need - 1) == WS


def test_binding_refuses_what_the_library_cannot_see():
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    k = torch.zeros((4, 16, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):  # CPU tensors
        mkv.mkv_page_update(k, k.clone(), i32(1, 1, 2), i32(1, 1), i32(4), i32(1, 1, 2), i32(1, 1), i32(4),
                            torch.zeros(4096, dtype=torch.uint8))
    with pytest.raises(ValueError):
        mkv.pool_of(k, torch.zeros((4, 16, 128), dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        mkv.pool_of(k.float(), k.float())
    with pytest.raises(ValueError):
        mkv.lists_of(i32(1, 1, 2), i32(1, 2))
    with pytest.raises(ValueError):
        mkv.lists_of(torch.zeros((1, 1, 2), dtype=torch.int64))
    with pytest.raises(ValueError):
        mkv._token_rows(torch.zeros((3, 64, 4), dtype=torch.bfloat16).transpose(1, 2), 4, 64, 3, "Q")
    assert mkv._token_rows(torch.zeros((3, 6, 64), dtype=torch.bfloat16)[:, 1:5], 4, 64, 3, "Q") == 384
    assert mkv._token_rows(torch.zeros((1, 6, 64), dtype=torch.bfloat16)[:, 1:5], 4, 64, 1, "Q") == 256


def test_rope_frequencies():
    for rot, theta in ((16, 10000.0), (64, 500000.0), (128, 1e6), (256, 1.5)):
        f = [theta ** (-2.0 * i / rot) for i in range(rot // 2)]
        half = 2.0 ** -24 * 1.001
        for got, want in ((mkv.mkv_rope_frequencies(rot, theta), f),
                          (mkv.mkv_rope_frequencies(rot, theta, "linear", 8.0), [x / 8 for x in f])):
            assert all(abs(float(g) - w) <= half * w for g, w in zip(got, want)) and len(got) == rot // 2
        got = mkv.mkv_rope_frequencies(rot, theta, "by_parts", 8.0, 8192, 1.0, 4.0)
        for g, w in zip(got, f):
            turns = 8192 * w / (2 * math.pi)
            share = min(max((turns - 1) / 3, 0), 1)
            assert abs(float(g) - w * (share + (1 - share) / 8)) <= half * w
    bad = [(0, 1e4), (24, 1e4), (-16, 1e4), (64, 1.0), (64, float("nan")), (64, 1e4, "linear", 0.5),
           (64, 1e4, "by_parts", 2.0, 0, 1, 4), (64, 1e4, "by_parts", 2.0, 100, 0, 4), (64, 1e4, "by_parts", 2.0, 100, 4, 4)]
    for args in bad:
        with pytest.raises(mkv.MKVError):
            mkv.mkv_rope_frequencies(*args)
    assert mkv.load().mkv_rope_frequencies(64, 1e4, 7, 1.0, 0, 0.0, 0.0, vp(A)) == -1
    assert mkv.load().mkv_rope_frequencies(64, 1e4, 0, 1.0, 0, 0.0, 0.0, None) == -1
