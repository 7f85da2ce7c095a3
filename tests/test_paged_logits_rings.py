"""The paged logits' rings, gone round more than twice: stages, items and the slots of a row's queries.

A CTA takes an equal share of all tiles (128 keys of a row), two CTAs an SM.  Its rings have at most 4 stages,
7 items and 4 slots, so 15 tiles use every place three times and 9 rows every slot.  Compared with the
plain form, tolerances of tests/test_paged.py.
"""
import numpy as np
import pytest
import torch

import fp8_mqa_logits_02_gb300 as fm
from test_paged import F8, cache, check_logits, gpu

pytestmark = pytest.mark.gpu

ITEMS, SLOTS = 7, 4


@pytest.fixture(scope="module", autouse=True)
def _lib():
    fm.build()
    fm.lib()


def ctas():
    return 2 * torch.cuda.get_device_properties(0).multi_processor_count


@pytest.mark.parametrize("page", [64, 16])     # TMA, and copies of 16 bytes
@pytest.mark.parametrize("T", [1, 2, 4])
def test_many_short_rows_go_round_the_slots(T, page):
    rng = np.random.default_rng(T + page)
    lens = rng.integers(1, 257, (2 * SLOTS + 2) * ctas()).astype(np.int32)
    lens[rng.random(len(lens)) < 0.1] = 0
    assert np.count_nonzero(lens) > (2 * SLOTS + 1) * ctas() * 0.95
    check_logits(rng, lens, T, page)


@pytest.mark.parametrize("page", [64, 33])
@pytest.mark.parametrize("T", [1, 2, 3, 4])
def test_long_ragged_rows_go_round_the_stages(T, page):
    rng = np.random.default_rng(10 * T + page)
    lens = rng.integers(2, 2 * 21 * 128 * ctas() // 24, 24).astype(np.int32)
    lens = (lens * (20 * 128 * ctas() / lens.sum())).astype(np.int32)
    assert (-(-lens // 128)).sum() >= (2 * ITEMS + 1) * ctas()
    check_logits(rng, lens, T, page)


@pytest.mark.parametrize("page", [32, 96, 128, 160, 256])     # pieces of 32 rows, 64, 128 and one a tile; tiles across pages
@pytest.mark.parametrize("T", [1, 2, 4])
def test_page_sizes_that_tma_fetches(T, page):
    rng = np.random.default_rng(T * page)
    check_logits(rng, [1, 31, 32, 33, 127, 128, 129, 500, 1003], T, page)
    check_logits(rng, [700, 300, 129], T, page, holes=True)
    check_logits(rng, [700, 300, 129], T, page, holes=True, clean=False, layout="joint")


def test_logits_see_the_rows_written_just_before_through_tma():
    # pages of 64: the keys come by the asynchronous proxy, behind the kernel that wrote them
    rng = np.random.default_rng(5)
    B, page, cols, steps = 5, 64, 4, 150
    data, scale = cache(rng, B * cols, page, 1, 128)
    table = torch.arange(B * cols, dtype=torch.int32, device="cuda").view(B, cols)
    x = torch.from_numpy(rng.standard_normal((steps, B, 1, 128))).to(torch.bfloat16).cuda()
    q = torch.from_numpy(rng.standard_normal((steps, B, 1, 32, 128))).float().to(F8).cuda()
    w = torch.from_numpy(rng.standard_normal((steps, B, 1, 32)).astype(np.float32)).cuda()

    def run(pause):
        d, s = data.clone(), scale.clone()
        lens = torch.zeros(B, dtype=torch.int32, device="cuda")
        first = torch.arange(B, dtype=torch.int32, device="cuda") * cols * page
        out = []
        for t in range(steps):
            slots = first + lens
            lens = lens + 1
            pause()
            fm.cache_write(slots, x[t], d, s)
            pause()
            out.append(fm.logits_paged(q[t], d, s, w[t], table, lens))
            pause()
        torch.cuda.synchronize()
        return out

    want = run(torch.cuda.synchronize)
    assert all(torch.isfinite(o[:, :t + 1]).all() for t, o in enumerate(want))
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(run(lambda: None), want))
