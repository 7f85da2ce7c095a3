"""Norms with rotation against a plain form in 64 bits.

Tolerance, with u = 2^-24: the sum of squares has 8 + 4 roundings of positive terms, of which the root takes half,
with rsqrt's 2 ulp (4 u) and eps: 11 u.  Sine and cosine are off by 1 ulp (2 u) and by their angle's rounding, at
most pi 2^-25 (1.6 u) + |t| 2^-52.  Their product with the weight, the two products, their difference and the
factor take 5 u more: |err| <= (20 u + |t| 2^-52) (|y_a| + |y_b|), then half a step of the type.  E4M3: a value is off
by 2^-4 of itself or 2^-10 of its scale (half its least step) from the row's y, and 3 u of the quantising products.
"""
import numpy as np
import pytest
import torch

import fp8_mqa_logits_02_gb300 as fm
from oracle import paged
from oracle import step as plain

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
F8 = torch.float8_e4m3fn
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
LEAST = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}  # half the least step
TYPES = list(HALF)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    fm.build()
    fm.lib()


def freq(R, base=10000.0):
    return torch.tensor([base ** (-2 * i / max(R, 1)) for i in range(R // 2)], dtype=torch.float32, device="cuda")


def f64(t):
    return t.cpu().float().double().numpy() if t.dtype != torch.float64 else t.cpu().numpy()


def check(x, out, weight, positions, inv_freq, eps=1e-6, interleaved=False, dtype=None):
    pos, f = positions.cpu().numpy(), inv_freq.cpu().double().numpy()
    want, size = plain.norm_rotate(f64(x), None if weight is None else f64(weight), pos, f, eps, interleaved)
    # per token, its fastest pair's angle
    far = np.abs(pos.astype(np.float64)) * (f.max() if len(f) else 0.0)
    err = (20 * U + far * 2.0 ** -52)[:, None, None] * size
    if dtype != F8:
        tol = err * (1 + HALF[x.dtype]) + HALF[x.dtype] * np.abs(want) + LEAST[x.dtype]
        assert np.all(np.abs(f64(out) - want) <= tol), (np.abs(f64(out) - want) / tol).max()
        return
    values, scale = paged.e4m3_values()[out[0].cpu().view(torch.uint8).numpy()], f64(out[1])
    a = np.maximum(np.abs(want).max(-1), 1e-30)
    assert np.all(np.abs(scale - a / 448) <= (err.max(-1) + 3 * U * a) / 448)
    got, s = values * scale[..., None], scale[..., None]
    tol = (2.0 ** -4 + 6 * U) * (np.abs(want) + err) + 2.0 ** -10 * s + err
    assert np.all(np.abs(got - want) <= tol), (np.abs(got - want) / tol).max()


def rows(rng, T, H, D, dtype):
    return torch.from_numpy(rng.standard_normal((T, H, D)) * np.exp(rng.standard_normal((T, H, 1)))).to(dtype).cuda()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,hq,hk,dim,R", [(1, 1, 1, 128, 128), (1, 32, 8, 128, 64), (3, 5, 2, 64, 64), (7, 8, 1, 64, 48),
                                           (130, 3, 0, 128, 16), (257, 12, 4, 128, 112), (33, 0, 2, 64, 32)])
def test_sizes(T, hq, hk, dim, R, interleaved, dtype):
    rng = np.random.default_rng(T + R)
    # slices of a fused projection, two heads of something else between them
    x = rows(rng, T, hq + hk + 2, dim, dtype)
    q, k = x[:, :hq], x[:, hq + 2:]
    pos = torch.from_numpy(rng.integers(0, 200000, T).astype(np.int32)).cuda()
    wq, wk = (torch.from_numpy(rng.standard_normal(dim)).to(t).cuda() for t in (dtype, torch.float32))
    got = fm.norm_rotate(q, k, pos, freq(R), wq, wk, interleaved=interleaved)
    check(q, got[0], wq, pos, freq(R), interleaved=interleaved)
    check(k, got[1], wk, pos, freq(R), interleaved=interleaved)
    got = fm.norm_rotate(q, k, pos, freq(R), None, wk, eps=0.25, interleaved=interleaved, dtype=F8)
    check(q, got[0], None, pos, freq(R), interleaved=interleaved, dtype=F8)
    check(k, got[1], wk, pos, freq(R), 0.25, interleaved, F8)


@pytest.mark.parametrize("dtype", TYPES)
def test_many_heads_a_group(dtype):
    # enough tokens that a group of lanes takes several heads, and the last group of a tensor's fewer
    rng = np.random.default_rng(0)
    T = 3001
    x = rows(rng, T, 21, 64, dtype)
    pos = torch.arange(T, device="cuda") + 100000
    w = torch.from_numpy(rng.standard_normal(64)).to(dtype).cuda()
    for out in (None, F8):
        got = fm.norm_rotate(x[:, :18], x[:, 18:], pos, freq(64), w, None, dtype=out)
        check(x[:, :18], got[0], w, pos, freq(64), dtype=out)
        check(x[:, 18:], got[1], None, pos, freq(64), dtype=out)


@pytest.mark.parametrize("out", [None, F8])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,hq,hk,dim", [(1, 1, 1, 64), (1, 1, 1, 128), (5, 3, 2, 64), (5, 2, 1, 128), (1500, 17, 3, 64)])
def test_a_norm_of_one_tensor(T, hq, hk, dim, dtype, out):
    # groups of lanes of one warp, of which some norm their heads and others do not
    rng = np.random.default_rng(T + dim)
    q, k = rows(rng, T, hq, dim, dtype), rows(rng, T, hk, dim, dtype)
    pos = torch.from_numpy(rng.integers(0, 200000, T).astype(np.int32)).cuda()
    w = torch.from_numpy(rng.standard_normal(dim)).to(dtype).cuda()
    for wq, wk in ((w, None), (None, w)):
        got = fm.norm_rotate(q, k, pos, freq(dim), wq, wk, dtype=out)
        check(q, got[0], wq, pos, freq(dim), dtype=out)
        check(k, got[1], wk, pos, freq(dim), dtype=out)


@pytest.mark.parametrize("wide", [torch.int32, torch.int64])
def test_far_positions(wide):
    rng = np.random.default_rng(1)
    pos = [0, 1, -1, 131071, 1 << 20, (1 << 24) + 1, (1 << 30) + 7, 2 ** 31 - 1, -2 ** 31]
    if wide == torch.int64:
        pos += [2 ** 31, 2 ** 36 + 12345, -2 ** 40]
    pos = torch.tensor(pos, dtype=wide, device="cuda")
    x = rows(rng, len(pos), 2, 128, torch.float32)
    f = freq(128)
    f[3], f[5], f[7], f[9] = 0.0, -0.25, 7.5, 1e-30      # still, backwards, over a turn a position, hardly
    got = fm.norm_rotate(x, None, pos, f)
    assert got[1] is None
    check(x, got[0], None, pos, f)


def test_no_tokens_and_no_heads():
    x, pos = torch.empty(0, 3, 64, device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda")
    q, k = fm.norm_rotate(x, x[:, :1], pos, freq(64))
    assert q.shape == (0, 3, 64) and k.shape == (0, 1, 64)
    (q, by), _ = fm.norm_rotate(x, None, pos, freq(64), dtype=F8)
    assert q.shape == (0, 3, 64) and by.shape == (0, 3)
    one = torch.ones(2, 1, 64, device="cuda")
    q, k = fm.norm_rotate(one[:, :0], one, torch.zeros(2, dtype=torch.int32, device="cuda"), freq(64))
    assert q.shape == (2, 0, 64) and torch.equal(k, one)


def test_norm_without_rotation_and_rotation_without_norm():
    rng = np.random.default_rng(2)
    x = rows(rng, 9, 3, 128, torch.bfloat16)
    pos = torch.zeros(9, dtype=torch.int32, device="cuda")
    w = torch.from_numpy(rng.standard_normal(128)).float().cuda()
    got, _ = fm.norm_rotate(x, None, pos, freq(0), w)
    check(x, got, w, pos, freq(0))
    got, _ = fm.norm_rotate(x, None, pos, freq(0))
    assert torch.equal(got, x)
    got, _ = fm.norm_rotate(x, None, pos, freq(64))      # position 0 turns nothing
    assert torch.equal(got, x)


def test_in_place_and_into_strided_results():
    rng = np.random.default_rng(3)
    for dtype in TYPES:
        x = rows(rng, 40, 6, 128, dtype)
        pos = torch.arange(40, dtype=torch.int32, device="cuda")
        w = torch.from_numpy(rng.standard_normal(128)).to(dtype).cuda()
        want = fm.norm_rotate(x[:, :4], x[:, 5:], pos, freq(128), w, w)
        to = torch.full((40, 9, 130), 3.0, dtype=dtype, device="cuda")
        got = fm.norm_rotate(x[:, :4], x[:, 5:], pos, freq(128), w, w, q_out=to[:, 1:5, 1:129], k_out=to[:, 7:8, :128])
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        to[:, 1:5, 1:129] = to[:, 7:8, :128] = 3.0
        assert (to == 3.0).all()
        other = x[:, 4].clone()
        got = fm.norm_rotate(x[:, :4], x[:, 5:], pos, freq(128), w, w, q_out=x[:, :4], k_out=x[:, 5:])
        assert torch.equal(x[:, :4], want[0]) and torch.equal(x[:, 5:], want[1]) and torch.equal(x[:, 4], other)


@pytest.mark.parametrize("dtype", TYPES)
def test_unaligned_rows(dtype):
    rng = np.random.default_rng(4)
    flat = torch.from_numpy(rng.standard_normal(3 + 40 * 131)).to(dtype).cuda()
    x = flat.as_strided((20, 2, 64), (262, 131, 1), 3)
    pos = torch.arange(20, dtype=torch.int32, device="cuda")
    w = torch.from_numpy(rng.standard_normal(65)).to(dtype).cuda()[1:]
    for interleaved in (False, True):
        got, _ = fm.norm_rotate(x, None, pos, freq(48), w, interleaved=interleaved)
        check(x, got, w, pos, freq(48), interleaved=interleaved)


def test_special_values():
    x = torch.zeros(6, 1, 128, device="cuda")
    x[1, 0, 3] = float("inf")
    x[2, 0, 100] = float("-inf")     # a value that does not turn
    x[3, 0, 5] = float("nan")
    x[4] = 1e-30
    pos = torch.full((6,), 9, dtype=torch.int32, device="cuda")
    got, _ = fm.norm_rotate(x, None, pos, freq(64))
    assert (got[0] == 0).all() and torch.isfinite(got[4]).all()
    assert got[2, 0, 100] == float("-inf") and (got[2].isinf().sum() == 1) and not got[2].isnan().any()
    assert got[1].isfinite().sum() == 126 and got[3].isnan().sum() == 2
    w = torch.ones(128, device="cuda")
    got, _ = fm.norm_rotate(x, None, pos, freq(64), w, eps=0.0)
    assert got[0].isnan().all()      # 0 / 0, as the formula has it
    assert got[3].isnan().all()
    got, _ = fm.norm_rotate(x, None, pos, freq(64), w)
    assert (got[0] == 0).all()
    v, s = fm.norm_rotate(x, None, pos, freq(64), dtype=F8)[0]
    back = v.float() * s.unsqueeze(-1)
    assert back[1].isnan().all() and back[3].isnan().all() and (back[0] == 0).all()


def test_feeds_the_indexer():
    # the indexer's queries: E4M3 with scales, which go into the weights
    rng = np.random.default_rng(5)
    T, N = 65, 300
    x = rows(rng, T, 32, 128, torch.bfloat16)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    (q, by), _ = fm.norm_rotate(x, None, pos, freq(64), interleaved=True, dtype=F8)
    k = torch.randn(N, 128, device="cuda").to(F8)
    w = torch.randn(T, 32, device="cuda") / 64
    ks, ke = torch.zeros(T, dtype=torch.int32, device="cuda"), torch.full((T,), N, dtype=torch.int32, device="cuda")
    got = fm.fp8_mqa_logits(q, k, torch.ones(N, device="cuda"), w * by, ks, ke)
    assert fm.check_error() == 0
    heads = torch.einsum("thd,nd->thn", q.double() * by.double().unsqueeze(-1), k.double())
    want = (heads.relu() * w.double().unsqueeze(-1)).sum(1)
    assert torch.allclose(got.double(), want, rtol=1e-3, atol=1e-3)


def test_captured_and_replayed():
    rng = np.random.default_rng(6)
    x = rows(rng, 4, 6, 128, torch.bfloat16)
    pos, w = torch.zeros(4, dtype=torch.int64, device="cuda"), torch.ones(128, device="cuda")
    f = freq(128)
    fm.norm_rotate(x[:, :4], x[:, 4:], pos, f, w, w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = fm.norm_rotate(x[:, :4], x[:, 4:], pos, f, w, w)
    for at in (0, 77, 123456):
        pos.fill_(at)
        x.copy_(rows(rng, 4, 6, 128, torch.bfloat16))
        graph.replay()
        check(x[:, :4], got[0], w, pos, freq(128))
        check(x[:, 4:], got[1], w, pos, freq(128))
