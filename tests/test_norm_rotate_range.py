"""Norms with rotation at the ends of the range.  Tolerances as in test_norm_rotate.py but where stated."""
from fractions import Fraction

import numpy as np
import pytest
import torch

import fp8_mqa_logits_02_gb300 as fm
from test_norm_rotate import F8, TYPES, check, freq, rows

pytestmark = pytest.mark.gpu

TWO_PI = 2 * Fraction("3.14159265358979323846264338327950288419716939937510582097494459")


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


def test_angles_of_positions_up_to_2_39():
    # With f the frequency in turns, its 64-bit fraction is off by (1 + |f|) 2^-64 at most (what is cut off, and the
    # rounding of 1 / 2 pi), so the angle by that times |position|: 2^-25 turns at 2^39 for a slow pair.  Cut to 2^-32
    # of a turn and rounded to 24 bits of half a turn it is off by 2^-32 + 2^-26 more.  Sine and cosine are within
    # 2 U (U = 2^-24), and the products and their difference take 3 U.  Nothing of it grows with the angle, which is up
    # to 4e12 radians here.
    rng = np.random.default_rng(3)
    pos = [2 ** 39, -2 ** 39, 2 ** 39 - 1, 2 ** 38 + 12345, -(2 ** 36) - 7, 2 ** 33 + 1, 2 ** 31 - 1, -1]
    x = rows(rng, len(pos), 2, 128, torch.float32)
    f = freq(128)
    f[3], f[5], f[9] = 7.5, -0.25, 1e-30
    got, _ = fm.norm_rotate(x, None, torch.tensor(pos, dtype=torch.int64, device="cuda"), f)
    freqs = [Fraction(v) for v in f.cpu().double().tolist()]
    t = np.array([[float(p * v / TWO_PI % 1 * TWO_PI) for v in freqs] for p in pos])[:, None]
    off = np.array([[float((1 + abs(v / TWO_PI)) * abs(p) / 2 ** 64) for v in freqs] for p in pos])[:, None]
    err = 2 * np.pi * (off + 2.0 ** -26 + 2.0 ** -32) + 5 * 2.0 ** -24
    assert err.max() < 20 * 2.0 ** -24
    a, b = np.split(x.cpu().double().numpy(), 2, -1)
    want = np.concatenate([a * np.cos(t) - b * np.sin(t), b * np.cos(t) + a * np.sin(t)], -1)
    tol = np.concatenate([err * (np.abs(a) + np.abs(b))] * 2, -1)
    assert np.all(np.abs(got.cpu().double().numpy() - want) <= tol), (np.abs(got.cpu().double().numpy() - want) / tol).max()
