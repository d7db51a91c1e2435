"""Host-side checks of 4-bit pages, mkv_page_quantize and positions on several axes (no GPU needed: every call here is
refused, or has nothing to do), and the references that their tests use."""
import ctypes

import numpy as np
import pytest
import torch

import geometric_kv_cache_gb300 as mkv
from test_paged_abi import (A, ARG, BIG, OK, POINTERS, SIZES, UNS, WS, _attend, _compact, _lists, _out, _pool, _rope, _tokens,
                            _update, vp)

FOUR = _pool(k=7 * A, v=8 * A, dtype=4)


def test_contiguous_calls_refuse_4_bit_caches():
    shape = mkv.MkvShape(1, 1, 64, 128, 4, None)
    lib = mkv.load()
    assert lib.mkv_workspace_size(shape, 0) == 0
    assert lib.mkv_centroid(vp(A), shape, 0, vp(A), vp(A), BIG, None) == UNS
    assert lib.mkv_compress(vp(A), vp(2 * A), shape, 0.5, None, 0, 0, 32, vp(3 * A), vp(4 * A), vp(5 * A), vp(6 * A), vp(7 * A),
                            BIG, None) == UNS


@pytest.mark.parametrize("dtype", [-1, 2, 3, 5])
def test_types_that_are_none(dtype):
    pool = _pool(k=7 * A, v=8 * A, dtype=dtype)
    assert _update(pool=pool) == UNS and _compact(pool=pool) == UNS and _attend(pool=pool) == UNS
    assert _rope(pool=pool) == UNS and _quantize(pool=pool) == UNS


def test_4_bit_pools_are_sized_and_checked_as_others():
    lib = mkv.load()
    assert lib.mkv_page_workspace_size(FOUR, _lists()) == lib.mkv_page_workspace_size(_pool(), _lists())
    assert lib.mkv_attention_workspace_size(FOUR, _lists(max_pages=1000), _tokens(), 1, 16000) > 256
    for kwargs, status in ((dict(pool=_pool(head_dim=96, dtype=4)), UNS), (dict(pool=_pool(k=A + 8, dtype=4)), ARG),
                           (dict(pool=_pool(page_size=8, dtype=4)), UNS)):
        assert _update(**kwargs) == status and _attend(**kwargs) == status and _quantize(**kwargs) == status
    assert _compact(pool=FOUR, K=A, V=A, t_max=4) == UNS  # no contiguous cache has this type
    assert _attend(pool=FOUR, tokens=_tokens(n=0), Q=0, O=0, k_scale=0.5, v_scale=3.0) == OK
    assert _attend(pool=FOUR, k_scale=0.0) == ARG and _attend(pool=FOUR, scale=3e38, k_scale=2.0) == ARG
    none = dict(pool=FOUR, tokens=_tokens(n=0), Q=0, K=0, V=0, Q_out=0)
    assert _rope(**none, k_scale=0.5) == OK
    # 512 times the reciprocals is to be finite
    assert _rope(**none, k_scale=2.0 ** -118) == OK and _rope(**none, k_scale=2.0 ** -119) == ARG
    assert _rope(**none, v_scale=2.0 ** -120) == ARG and _rope(**none, v_scale=-1.0) == ARG


def _quantize(pool=FOUR, lists=_lists(), out=None, refs=7 * A, idx=8 * A, idx_stride=100, kept=9 * A, K=A, V=2 * A, t_max=50,
              seq_lens=0, k_scale=1.0, v_scale=1.0, refs_out=10 * A, ws=11 * A, ws_bytes=BIG):
    out = out or _out(batch=lists.batch, heads=lists.heads, max_pages=lists.max_pages)
    return mkv.load().mkv_page_quantize(pool, lists, vp(refs), vp(idx), idx_stride, vp(kept), vp(K), vp(V), t_max,
                                        vp(seq_lens), k_scale, v_scale, out, vp(refs_out), vp(ws), ws_bytes, None)


def _as_four(kwargs):
    """The shared cases with 4-bit pools (they are refused for other reasons)."""
    if "pool" in kwargs and kwargs["pool"].dtype == 0:
        p = kwargs["pool"]
        kwargs = dict(kwargs, pool=mkv.MkvPagePool(p.n_pages, p.page_size, p.head_dim, 4, p.k_pages, p.v_pages))
    return kwargs


@pytest.mark.parametrize("kwargs,status", [(_as_four(k), s) for k, s in SIZES + POINTERS] + [
    (dict(pool=_pool()), UNS),  # bf16 pages are copied, not rounded
    (dict(K=0), ARG), (dict(V=0), ARG), (dict(K=A + 8), ARG), (dict(t_max=-1), ARG), (dict(t_max=(1 << 30) + 1), UNS),
    (dict(kept=0), ARG), (dict(idx=8 * A + 1), ARG), (dict(idx_stride=-1), ARG), (dict(seq_lens=A + 1), ARG),
    (dict(out=_lists()), ARG), (dict(k_scale=0.0), ARG), (dict(v_scale=-1.0), ARG), (dict(k_scale=float("nan")), ARG),
    (dict(v_scale=float("inf")), ARG), (dict(k_scale=2.0 ** -119), ARG), (dict(pool=_pool(dtype=1), k_scale=2.0 ** -130), ARG),
    (dict(lists=_lists(batch=0), refs_out=7 * A), OK),
])
def test_quantize_refusals(kwargs, status):
    assert _quantize(**kwargs) == status


def _axes(n_axes=3, axes=13 * A, tokens=_tokens(), pos=4 * A, rot=128, pool=FOUR, lists=_lists(), ws=11 * A, ws_bytes=BIG, Q=A):
    return mkv.load().mkv_rope_append_axes(vp(Q), 4096, vp(2 * A), 1024, vp(3 * A), 1024, tokens, vp(pos), n_axes, vp(axes),
                                           vp(5 * A), rot, 0, 1.0, vp(6 * A), pool, lists, 1.0, 1.0, vp(ws), ws_bytes, None)


@pytest.mark.parametrize("kwargs,status", [(_as_four(k), s) for k, s in SIZES + POINTERS] + [
    (dict(n_axes=0), ARG), (dict(n_axes=9), ARG), (dict(n_axes=-1), ARG), (dict(axes=0), ARG), (dict(axes=13 * A + 2), ARG),
    (dict(pos=0), ARG), (dict(rot=8), ARG), (dict(Q=0), ARG), (dict(tokens=_tokens(n=0), axes=0), OK),
])
def test_rope_axes_refusals(kwargs, status):
    assert _axes(**kwargs) == status


def test_axes_of_pairs():
    assert mkv.mkv_rope_axes([4, 2, 2]).tolist() == [0, 0, 0, 0, 1, 1, 2, 2]
    assert mkv.mkv_rope_axes([4, 2, 2], dealt=True).tolist() == [0, 1, 2, 0, 1, 2, 0, 0]
    assert mkv.mkv_rope_axes([0, 3, 5], dealt=True).tolist() == [1, 2, 1, 2, 1, 2, 2, 2]
    assert mkv.mkv_rope_axes([8], dealt=True).tolist() == [0] * 8
    assert mkv.mkv_rope_axes([1] * 8, dealt=True).tolist() == list(range(8))
    assert mkv.mkv_rope_axes([0, 0, 8]).tolist() == [2] * 8
    for sections in ([], [3, 3], [-1, 9], [1] * 9, [0, 0], [2 ** 31 - 1, 9]):
        with pytest.raises(mkv.MKVError):
            mkv.mkv_rope_axes(sections)
    three = (ctypes.c_int32 * 3)(4, 2, 2)
    out = (ctypes.c_int32 * 8)()
    lib = mkv.load()
    assert lib.mkv_rope_axes(16, 3, three, 0, out) == 0
    assert lib.mkv_rope_axes(32, 3, three, 0, out) == -1 and lib.mkv_rope_axes(16, 0, three, 0, out) == -1
    assert lib.mkv_rope_axes(16, 3, None, 0, out) == -1 and lib.mkv_rope_axes(16, 3, three, 0, None) == -1


def test_binding_of_4_bit_pages():
    pages = mkv.e2m1_pages(4, 16, 128, device="cpu")
    pool = mkv.pool_of(pages, pages.clone())
    assert (pool.n_pages, pool.page_size, pool.head_dim, pool.dtype) == (4, 16, 128, mkv.E2M1)
    for bad in (torch.zeros((4, 16, 64), dtype=torch.uint8), torch.zeros((4, 16, 72), dtype=torch.int8),
                torch.zeros((4, 72), dtype=torch.uint8)):
        with pytest.raises(ValueError):
            mkv.pool_of(bad, bad.clone())
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    x = torch.zeros((1, 1, 8, 128), dtype=torch.bfloat16)
    ws = torch.zeros(4096, dtype=torch.uint8)
    with pytest.raises(ValueError, match="mkv_page_quantize"):
        mkv.mkv_page_compact(pages, pages.clone(), i32(1, 1, 2), i32(1, 1), i32(4), None, i32(1, 1), i32(1, 1, 2), i32(1, 1),
                             i32(4), ws, K=x, V=x)
    with pytest.raises(ValueError):  # no cache
        mkv.mkv_page_quantize(pages, pages.clone(), i32(1, 1, 2), i32(1, 1), i32(4), None, i32(1, 1), None, x, i32(1, 1, 2),
                              i32(1, 1), i32(4), ws)


def test_reference_codes_against_torch_and_by_hand():
    import e2m1_util as eu
    x = torch.randn(4000).abs().float() * torch.exp2(torch.randint(-12, 8, (4000,)).float())
    mine = torch.from_numpy(eu.nearest(x.numpy(), eu.E4M3))
    assert torch.equal(mine, x.clamp(max=448).to(torch.float8_e4m3fn).view(torch.uint8))
    ties = np.float32([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.0001, 100.0, 0.2500001, 0.0])
    assert eu.nearest(ties, eu.E2M1).tolist() == [0, 2, 2, 4, 4, 6, 6, 7, 7, 1, 0]
    codes, scales = eu.encode(torch.tensor([[6.0, -3.0, 0.0, -0.1] + [0.5] * 12]), 1.0)
    assert scales.tolist() == [[0x38]] and codes[0, :3].tolist() == [0x7 | 0xD << 4, 0x0, 0x11]
    assert eu.decode(codes, scales)[0, :5].tolist() == [6.0, -3.0, 0.0, 0.0, 0.5]
    pages = torch.arange(2 * 16 * 36, dtype=torch.int64).to(torch.uint8).view(2, 16, 36)
    assert torch.equal(eu.rows_to_pages(eu.rows_of(pages)), pages)
    assert torch.equal(eu.to_pages(*eu.from_pages(pages)), pages)
