"""Norms with rotation at the ends of the range.  Tolerances as in test_norm_rotate.py but where stated."""
import numpy as np
import pytest
import torch

import fp8_mqa_logits_02_gb300 as fm
from test_norm_rotate import F8, TYPES, check, freq, rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    fm.build()
    fm.lib()


def back(out):
    return out[0].float() * out[1].unsqueeze(-1)


@pytest.mark.parametrize("eps", [1e-12, 1e-20])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", TYPES)
def test_zero_and_tiny_rows_to_e4m3(dtype, interleaved, eps):
    # The norm's factor is eps^-1/2 for these, and 448 over the row's maximum up to 4.48e32: their product is past fp32
    # for rows of zeros (padding) and of 1e-37, though every value is finite.  (A subnormal term of such a row is off by
    # 2^-150, in the result by that times the factor: 7e-40 for 1e-12 and 7e-36 for 1e-20, where 2^-10 of the row's scale
    # is 2e-36 and 2e-33.)
    rng = np.random.default_rng(1)
    x = rows(rng, 8, 3, 128, dtype)
    x[0] = 0
    x[1, 1] = 0
    x[2] = 1e-37
    x[3] = -1e-25
    x[4, 0] = 1e-10
    x[5, 2, 1:] = 0
    pos = torch.arange(8, dtype=torch.int32, device="cuda") * 1000
    w = torch.from_numpy(1 + 0.5 * rng.random(128)).float().cuda()
    got, k = fm.norm_rotate(x, x[:, :1], pos, freq(128), w, w, eps=eps, interleaved=interleaved, dtype=F8)
    check(x, got, w, pos, freq(128), eps, interleaved, F8)
    check(x[:, :1], k, w, pos, freq(128), eps, interleaved, F8)
    assert (back(got)[0] == 0).all() and (back(got)[1, 1] == 0).all()
    assert torch.isfinite(got[1]).all() and (got[1] > 0).all()


@pytest.mark.parametrize("eps", [0.0, 1e-20, 1e-6])
def test_rows_without_weight_to_e4m3(eps):
    # small rows whose weights are all zero: zeros, with the least scale
    x = torch.full((3, 2, 64), 1e-7, device="cuda")
    x[1] = 1.0
    pos = torch.arange(3, dtype=torch.int64, device="cuda")
    w = torch.zeros(64, device="cuda")
    got, _ = fm.norm_rotate(x, None, pos, freq(64), w, eps=eps, dtype=F8)
    check(x, got, w, pos, freq(64), eps, False, F8)
    assert (back(got) == 0).all() and torch.isfinite(got[1]).all()


@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("at", [0, 5, 31])
def test_a_frequency_that_is_not_finite_is_nan(at, interleaved, bad):
    rng = np.random.default_rng(2)
    x = rows(rng, 4, 2, 128, torch.float32)
    pos = torch.tensor([0, 1, -7, 99], dtype=torch.int32, device="cuda")
    f = freq(64)
    want, _ = fm.norm_rotate(x, None, pos, f, interleaved=interleaved)
    f[at] = bad
    got, _ = fm.norm_rotate(x, None, pos, f, interleaved=interleaved)
    pair = [2 * at, 2 * at + 1] if interleaved else [at, at + 32]
    rest = [d for d in range(128) if d not in pair]
    assert got[..., pair].isnan().all()
    assert torch.equal(got[..., rest], want[..., rest])
    v, s = fm.norm_rotate(x, None, pos, f, interleaved=interleaved, dtype=F8)[0]
    assert s.isnan().all() and v.float().isnan().all()
