"""Host-side refusals of the paged-cache calls that a user could run into with values in range by themselves (no GPU
needed: every call here is refused, or has nothing to do)."""
import pytest

from test_paged_abi import A, ARG, OK, UNS, _attend, _lists, _pool, _tokens

CODES = _pool(k=7 * A, v=8 * A, dtype=1)  # E4M3


@pytest.mark.parametrize("scale,k_scale", [(3e38, 2.0), (-3e38, 2.0), (1e20, 1e20), (3e38, 1.0), (-2.4e38, 1.0)])
def test_attention_refuses_scales_whose_product_is_infinite(scale, k_scale):
    assert _attend(pool=CODES, scale=scale, k_scale=k_scale) == ARG
    nothing = dict(tokens=_tokens(n=0), Q=0, O=0, pool=CODES)
    assert _attend(**nothing, scale=scale, k_scale=k_scale) == ARG


@pytest.mark.parametrize("scale,k_scale", [(3e38, 0.5), (-3e38, 0.78), (1e30, 1e8), (2.3e38, 1.0), (1e-38, 1e-38), (0.0, 3e38)])
def test_attention_takes_scales_whose_product_is_finite(scale, k_scale):
    assert _attend(tokens=_tokens(n=0), Q=0, O=0, pool=CODES, scale=scale, k_scale=k_scale) == OK


@pytest.mark.parametrize("batch,q_heads,max_len,status", [(32768, 32, 2 ** 17, UNS), (32768, 32, 2 ** 17 - 256, OK),
                                                          (32768, 512, 2 ** 17, UNS), (16384, 512, 2 ** 17, OK),
                                                          (16384, 1024, 2 ** 17, UNS)])
def test_attention_refuses_more_blocks_of_keys_than_32_bits(batch, q_heads, max_len, status):
    # 32 KV heads, one token per row: a tile per 16 query heads of a group, whether they are there or not
    lists = _lists(batch=batch, heads=32, max_pages=2 ** 13)
    assert _attend(tokens=_tokens(n=0, q_heads=q_heads), Q=0, O=0, lists=lists, max_q=1, max_len=max_len) == status
    assert _attend(tokens=_tokens(n=0, q_heads=q_heads), lists=lists, max_q=0, max_len=max_len) == OK
