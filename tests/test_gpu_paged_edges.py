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
