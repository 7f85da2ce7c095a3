"""attention_paged over scaled caches at the ends of the range."""
import numpy as np
import pytest
import torch

import fp8_mqa_logits_02_gb300 as fm
from test_paged import gpu
from test_paged4 import F4, cache

pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _lib():
    fm.build()
    fm.lib()


def caches(rng, kind, pages=6, page=32, heads=2, dim=128):
    """(k, v, keyword arguments) of attention_paged."""
    if kind == "4 bits":
        k, v = cache(rng, pages, page, heads, dim), cache(rng, pages, page, heads, dim)
        return k[0].view(F4), v[0].view(F4), dict(k_scale=k[2], v_scale=v[2], k_groups=k[1], v_groups=v[1])
    k, v = (torch.from_numpy(rng.standard_normal((pages, page, heads, dim))).float().cuda().to(F8) for _ in range(2))
    return k, v, dict(k_scale=torch.ones(pages, page, heads, device="cuda"), v_scale=torch.ones(pages, page, heads, device="cuda"))


@pytest.mark.parametrize("q_heads", [8, 32])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("kind", ["4 bits", "e4m3"])
def test_a_scale_that_is_nan(kind, dtype, q_heads):
    rng = np.random.default_rng(1)
    k, v, more = caches(rng, kind)
    table, lens = gpu(np.array([[0, 1], [2, 3], [4, 5], [-1, 6]])).int(), gpu(np.array([33, 0, 64, 40])).int()
    q = torch.from_numpy(rng.standard_normal((4, q_heads, 128))).to(dtype).cuda()
    out, lse = fm.attention_paged(q, k, v, table, lens, sm_scale=float("nan"), return_lse=True, **more)
    assert out[[0, 2]].isnan().all() and lse[[0, 2]].isnan().all()
    assert (out[[1, 3]] == 0).all() and (lse[[1, 3]] == -float("inf")).all()      # no position, none that is there


@pytest.mark.parametrize("q_heads", [8, 32])
@pytest.mark.parametrize("kind", ["4 bits", "e4m3"])
@pytest.mark.parametrize("e", [-80, 60, 112, 120])
def test_large_and_small_bfloat16_queries(kind, e, q_heads):
    # scores are sm_scale q . k: a power of two that goes from one to the other leaves every bit of the result
    rng = np.random.default_rng(2)
    k, v, more = caches(rng, kind)
    table, lens = gpu(np.array([[0, 1], [2, 3], [4, 5]])).int(), gpu(np.array([33, 1, 64])).int()
    q = torch.from_numpy(rng.standard_normal((3, q_heads, 128))).to(torch.bfloat16).cuda()
    want = fm.attention_paged(q, k, v, table, lens, sm_scale=0.0625, return_lse=True, **more)
    got = fm.attention_paged(q * 2.0 ** e, k, v, table, lens, sm_scale=0.0625 * 2.0 ** -e, return_lse=True, **more)
    assert torch.isfinite(want[0]).all()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
