"""NaN in what the paged logits read is NaN in what they give, as in the definition (relu(NaN) is NaN): a
key's for its position, a query's or a weight's for its token, and no other entry."""
import numpy as np
import pytest
import torch

import fp8_mqa_logits_02_gb300 as fm
from oracle import paged as plain
from test_paged import F8, U, cache, f64, gpu, tables

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    fm.build()
    fm.lib()


@pytest.mark.parametrize("page", [64, 16])   # TMA, and copies of 16 bytes
@pytest.mark.parametrize("T", [1, 2, 3])
def test_logits_of_nan(T, page):
    rng = np.random.default_rng(10 * T + page)
    lens = np.array([300, 140, 200, 77], np.int32)
    table, pages = tables(rng, lens, page)
    data, scale = cache(rng, pages, page, 1, 128)
    q = torch.from_numpy(rng.standard_normal((4, T, 32, 128))).float().to(F8).cuda()
    w = torch.from_numpy(rng.standard_normal((4, T, 32)).astype(np.float32) / 64).cuda()
    q.view(torch.uint8)[0, T - 1, 5, 17] = 0x7F          # one value of one head of the newest token
    w[1, 0, 31] = float("nan")
    bytes_ = data.view(torch.uint8)
    bytes_[int(table[2, 0]), 3, 0, 100] = 0xFF           # one value of position 3
    bytes_[int(table[2, 199 // page]), 199 % page] = 0x7F    # all of the last position
    scale[int(table[3, 1 if page == 16 else 0]), 2, 0] = float("nan")
    got = fm.logits_paged(q, data, scale, w, gpu(table), gpu(lens)).cpu().double().numpy()
    with np.errstate(invalid="ignore"):
        want, size = plain.logits(f64(q), f64(w), f64(data)[:, :, 0], f64(scale)[:, :, 0], table, lens, got.shape[1])
    assert np.isnan(want).sum() >= 300
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(np.isneginf(got), np.isneginf(want))
    seen = np.isfinite(want)
    assert np.all(np.abs(got[seen] - want[seen]) <= (128 + 32 + 2) * U * size[seen])
