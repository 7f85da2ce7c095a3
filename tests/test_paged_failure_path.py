"""The paged logits' failure path, made to run without planting anything.

Every wait of the kernel is bounded by the limit that fp8_mqa_logits_set_wait_limit_ns sets; a limit far
below a stage's latency makes the waits of a normal call run out.  The call returns, check_error reports
FP8MQA_ERR_TIMEOUT and clears it, and later calls are right again: tensor memory and shared memory were
given back with nothing under way.
"""
import numpy as np
import pytest
import torch

import fp8_mqa_logits_02_gb300 as fm
from oracle import paged as plain
from test_paged import U, cache, f64, gpu, tables

pytestmark = pytest.mark.gpu

TIMEOUT = -6


@pytest.fixture(scope="module", autouse=True)
def _lib():
    fm.build()
    fm.lib()
    yield
    fm.set_wait_limit_ns(0)


@pytest.mark.parametrize("page", [64, 16])   # TMA, and copies of 16 bytes
@pytest.mark.parametrize("T", [1, 2, 4])
def test_short_wait_limit_times_out_then_recovers(T, page):
    rng = np.random.default_rng(T * 100 + page)
    lens = rng.integers(20000, 30000, 24).astype(np.int32)    # 4000 tiles or more: 13 for each of 304 CTAs
    table, pages = tables(rng, lens, page)
    data, scale = cache(rng, pages, page, 1, 128)
    q = torch.from_numpy(rng.standard_normal((24, T, 32, 128))).float().to(torch.float8_e4m3fn).cuda()
    w = torch.from_numpy(rng.standard_normal((24, T, 32)).astype(np.float32) / 64).cuda()
    table_g, lens_g = gpu(table), gpu(lens)
    N = int(lens.max())
    out = torch.empty((24 * T, N), device="cuda")

    def call():
        fm.logits_paged(q, data, scale, w, table_g, lens_g, max_len=N, out=out)
        return fm.check_error()

    assert call() == 0
    want = out.clone()
    for _ in range(3):
        prev = fm.set_wait_limit_ns(200)
        try:
            assert call() == TIMEOUT
        finally:
            fm.set_wait_limit_ns(prev)
        assert fm.check_error() == 0            # cleared by the read
        out.fill_(float("nan"))
        assert call() == 0
        assert torch.equal(out, want)           # the same kernel on the same inputs, in the same order
    rows = [0, 11, 23]
    pick = [b * T + t for b in rows for t in range(T)]
    ref, size = plain.logits(f64(q)[rows], f64(w)[rows], f64(data)[:, :, 0], f64(scale)[:, :, 0], table[rows], lens[rows], N)
    got = out[pick].cpu().double().numpy()
    seen = np.isfinite(ref)
    assert np.array_equal(np.isfinite(got), seen)
    # the sums' bound of tests/test_paged.py
    assert np.all(np.abs(got[seen] - ref[seen]) <= (128 + 32 + 2) * U * size[seen])


@pytest.mark.parametrize("page", [64, 16])
def test_a_short_limit_is_kept_in_time(page):
    # every wait of these calls takes some microseconds at most: a suspension longer than the limit would
    # let them all end before the limit is looked at
    rng = np.random.default_rng(page)
    lens = np.array([4096], np.int32)
    table, pages = tables(rng, lens, page)
    data, scale = cache(rng, pages, page, 1, 128)
    q = torch.from_numpy(rng.standard_normal((1, 1, 32, 128))).float().to(torch.float8_e4m3fn).cuda()
    w = torch.from_numpy(rng.standard_normal((1, 1, 32)).astype(np.float32) / 64).cuda()
    want = fm.logits_paged(q, data, scale, w, gpu(table), gpu(lens))
    assert fm.check_error() == 0
    prev = fm.set_wait_limit_ns(100)
    try:
        for _ in range(5):
            fm.logits_paged(q, data, scale, w, gpu(table), gpu(lens))
            assert fm.check_error() == TIMEOUT
    finally:
        fm.set_wait_limit_ns(prev)
    assert torch.equal(fm.logits_paged(q, data, scale, w, gpu(table), gpu(lens)), want)
    assert fm.check_error() == 0
