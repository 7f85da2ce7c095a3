"""GPU parity of the paged-cache operators against their plain 64-bit forms.

Tolerances, with u = 2^-24 the unit of fp32 rounding:
  cache_write, cache_read   exact: every step is defined in fp32.
  logits_paged   a sum of 128 products, then of 32 weighted terms, then one product:
                 |err| <= (128 + 32 + 2) u * sum_h |w_h| sum_d |q_d k_d| * |scale|.
  attention_paged   the score's error dx <= (dim + 8) u * max_n sum_d |q_d k_d| * sm_scale, of which a
                 weight takes twice (its own and the sum's) and the exponential 2^-20; a weight is
                 rounded to 11 bits (8 for bfloat16 caches), half a unit of the last place; the largest
                 rounded weight scales the subnormal ones (2^-14 of the largest channel's sum); the
                 result is rounded to q's type:
                 |err| <= (2 dx + 2^-20 + 2^-11 | 2^-8) sum p |v| + 2^-14 max_d sum p |v| + 2^-11 | 2^-8 |out|
                 lse: |err| <= dx + 2^-20 (1 + |lse|).
"""
import numpy as np
import pytest
import torch

import fp8_mqa_logits_02_gb300 as fm
from oracle import paged as plain

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
F8 = torch.float8_e4m3fn
VALUES = plain.e4m3_values()


@pytest.fixture(scope="module", autouse=True)
def _lib():
    fm.build()
    fm.lib()


def f64(t):
    return VALUES[t.cpu().view(torch.uint8).numpy()] if t.dtype == F8 else t.cpu().double().numpy()


def same(a, b):
    return np.array_equal(a, b, equal_nan=True)


def cache(rng, pages, page, heads, dim, dtype=F8, layout="plain"):
    """(data, scale) on the GPU, filled; "joint" is one half of [pages, 2, ...], "heads" puts heads before rows."""
    n = {"plain": (pages, page, heads, dim), "joint": (pages, 2, page, heads, dim),
         "heads": (pages, heads, page, dim)}[layout]
    x = rng.standard_normal(n) * np.exp(0.5 * rng.standard_normal(n[:-1]))[..., None]
    if dtype == F8:
        data = torch.from_numpy(np.clip(x * 60, -448, 448)).float().to(F8).cuda()
        scale = torch.from_numpy((0.01 * np.exp(rng.standard_normal(n[:-1]))).astype(np.float32)).cuda()
    else:
        data, scale = torch.from_numpy(x).to(dtype).cuda(), None
    pick = {"plain": lambda t: t, "joint": lambda t: t[:, 1],
            "heads": lambda t: t.transpose(1, 2)}[layout]
    return pick(data), None if scale is None else pick(scale)


def as_rows(data, scale):
    x = f64(data)
    with np.errstate(invalid="ignore"):  # rows that stand for NaN
        return x if scale is None else x * f64(scale)[..., None]


def tables(rng, lens, page, spare=2, cols=None):
    need = [-(-max(0, int(n)) // page) for n in lens]
    cols = max(need + [1]) if cols is None else cols
    pages = sum(need) + spare
    pool = rng.permutation(pages)
    table = np.full((len(lens), cols), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = pool[at:at + n]
        at += n
    return table, pages


def gpu(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


# ------------------------------------------------------------------------------------ write

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("T,heads,dim,page", [(1, 1, 128, 64), (7, 8, 64, 1), (33, 3, 128, 16), (130, 2, 64, 100),
                                              (257, 1, 128, 33)])
def test_write_pair_is_exact(T, heads, dim, page, dtype):
    rng = np.random.default_rng(T * 7 + heads)
    pages = -(-T // page) + 2
    caches = [cache(rng, pages, page, heads, dim) for _ in range(2)]
    want = [[f64(t).copy() for t in c] for c in caches]
    # a slice of a fused projection: strided rows and heads
    qkv = torch.from_numpy(rng.standard_normal((T, 2 * heads + 3, dim)) * np.exp(rng.standard_normal((T, 1, 1)))).to(dtype).cuda()
    k, v = qkv[:, 1:1 + heads], qkv[:, 2 + heads:2 + 2 * heads]
    slots = rng.permutation(pages * page)[:T].astype(np.int32)
    slots[::5] = [-1, pages * page, -2 ** 31, 2 ** 31 - 1][T % 4]  # padding and slots out of range
    fm.cache_write(gpu(slots), k, *caches[0], v, *caches[1])
    for x, c, w in zip((k, v), caches, want):
        values, scale = plain.quantise32(x.float().cpu().numpy())
        ok = (slots >= 0) & (slots < pages * page)
        w[0].reshape(-1, heads, dim)[slots[ok]] = values[ok]
        w[1].reshape(-1, heads)[slots[ok]] = scale[ok]
        assert same(f64(c[0]), w[0]) and same(f64(c[1]), w[1])


@pytest.mark.parametrize("layout", ["joint", "heads"])
def test_write_one_into_strided_cache(layout):
    rng = np.random.default_rng(3)
    data, scale = cache(rng, 5, 24, 4, 128, layout=layout)
    before = (f64(data), f64(scale))
    x = torch.from_numpy(rng.standard_normal((50, 4, 128))).to(torch.bfloat16).cuda()
    slots = rng.permutation(120)[:50].astype(np.int32)
    fm.cache_write(gpu(slots), x, data, scale)
    values, by = plain.quantise32(x.float().cpu().numpy())
    page, row = slots // 24, slots % 24
    before[0][page, row], before[1][page, row] = values, by
    assert same(f64(data), before[0]) and same(f64(scale), before[1])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_write_unaligned_rows(dtype):
    # rows of 64 values 65 elements apart, from an odd element on
    rng = np.random.default_rng(4)
    flat = torch.from_numpy(rng.standard_normal(1 + 40 * 65)).to(dtype).cuda()
    x = flat.as_strided((20, 2, 64), (130, 65, 1), 1)
    data, scale = cache(rng, 2, 16, 2, 64)
    fm.cache_write(torch.arange(20, dtype=torch.int32, device="cuda"), x, data, scale)
    values, by = plain.quantise32(x.float().cpu().numpy())
    assert same(f64(data).reshape(32, 2, 64)[:20], values) and same(f64(scale).reshape(32, 2)[:20], by)


def test_write_special_rows():
    x = torch.zeros(8, 1, 64)
    x[1] = 3e38                       # the largest magnitudes
    x[2] = 1e-38                      # under the least maximum: still finite
    x[3, 0, 5] = float("nan")
    x[4, 0, 6] = float("inf")
    x[5, 0, 7] = -float("inf")
    x[6] = torch.linspace(-1, 1, 64)
    x[7, 0, 0] = -1e-45
    rng = np.random.default_rng(0)
    data, scale = cache(rng, 1, 8, 1, 64)
    fm.cache_write(torch.arange(8, dtype=torch.int32, device="cuda"), x.cuda(), data, scale)
    got = as_rows(data, scale).reshape(8, 64)
    assert np.isnan(got[3]).any() and np.isnan(got[4]).any() and np.isnan(got[5]).any()
    assert np.isnan(got[3:6]).all() and np.isfinite(got[[0, 1, 2, 6, 7]]).all()
    for r in (0, 1, 2, 6, 7):
        values, by = plain.quantise32(x[r].numpy())
        assert same(f64(data)[0, r], values) and same(f64(scale)[0, r], by.astype(np.float64))
    # against the definition in 64 bits: within half a step of e4m3 of the row's own scale
    assert np.all(np.abs(got[6] - x[6, 0].double().numpy()) <= 2.0 ** -4 * np.abs(x[6, 0].double().numpy()) + 2.0 ** -10 / 448)


# ------------------------------------------------------------------------------------ read

@pytest.mark.parametrize("dtype", [F8, torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("lens,heads,dim,page,layout", [
    ([5], 1, 128, 64, "plain"), ([0, 3, 0, 0, 70, 1, 0], 2, 64, 16, "plain"), ([129, 64, 1], 8, 128, 33, "heads"),
    ([40, 41], 4, 64, 1, "joint"), ([1] * 50 + [0] * 20 + [300], 1, 128, 100, "plain")])
def test_read_is_exact(lens, heads, dim, page, layout, dtype):
    rng = np.random.default_rng(sum(lens))
    table, pages = tables(rng, lens, page)
    data, scale = cache(rng, pages, page, heads, dim, layout=layout)
    if len(lens) > 2:
        table[-1, 0] = pages          # a page that is not there reads as zeros
    starts = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    total = int(starts[-1]) + 3       # rows past the last sequence are zeroed
    got = fm.cache_read(data, scale, gpu(table), gpu(starts), total, dtype=dtype)
    want, by = np.zeros((total, heads, dim), np.float32), np.zeros((total, heads), np.float32)
    d, s = f64(data).astype(np.float32), scale.cpu().numpy()
    for b, n in enumerate(lens):
        there, ids, row = plain.rows(d, table[b], np.arange(n), pages, page)
        want[starts[b]:starts[b] + n] = np.where(there[:, None, None], d[ids, row], 0)
        by[starts[b]:starts[b] + n] = np.where(there[:, None], s[ids, row], 0)
    if dtype == F8:
        assert same(f64(got[0]), want.astype(np.float64)) and same(got[1].cpu().numpy(), by)
    else:
        assert torch.equal(got.cpu(), torch.from_numpy(want * by[..., None]).to(dtype))


def test_read_feeds_the_prefill_logits():
    rng = np.random.default_rng(8)
    lens, page = [130, 61], 32
    table, pages = tables(rng, lens, page)
    data, scale = cache(rng, pages, page, 1, 128)
    starts = np.array([0, 130, 191], np.int32)
    k, kv = fm.cache_read(data, scale, gpu(table), gpu(starts), 191)
    q = torch.randn(2, 1, 32, 128, device="cuda").to(F8)
    w = torch.randn(2, 1, 32, device="cuda") / 64
    prefill = fm.fp8_mqa_logits(q.view(2, 32, 128), k.squeeze(1), kv.squeeze(1), w.view(2, 32), gpu(starts[:2]), gpu(starts[1:]))
    assert fm.check_error() == 0
    paged = fm.logits_paged(q, data, scale, w, gpu(table), gpu(np.array(lens, np.int32)), max_len=130)
    for b, n in enumerate(lens):
        assert torch.allclose(prefill[b, starts[b]:starts[b] + n], paged[b, :n], rtol=1e-4, atol=1e-5)


# ------------------------------------------------------------------------------------ logits

def check_logits(rng, lens, T, page, N=None, clean=True, layout="plain", holes=False, ld=None):
    lens = np.asarray(lens, np.int32)
    table, pages = tables(rng, lens, page)
    if holes:
        table[0, -1] = -5
        table[-1, 0] = pages
    data, scale = cache(rng, pages, page, 1, 128, layout=layout)
    B = len(lens)
    q = torch.from_numpy(rng.standard_normal((B, T, 32, 128))).float().to(F8).cuda()
    w = torch.from_numpy(rng.standard_normal((B, T, 32)).astype(np.float32) / 64).cuda()
    N = table.shape[1] * page if N is None else N
    out = None
    poison = 12345.0
    if ld is not None or not clean:
        out = torch.full((B * T, ld or N), poison, device="cuda")[:, :N]
    got = fm.logits_paged(q, data, scale, w, gpu(table), gpu(lens), max_len=N, out=out, clean_logits=clean)
    got = got.cpu().double().numpy()
    want, size = plain.logits(f64(q), f64(w), f64(data)[:, :, 0], f64(scale)[:, :, 0], table, lens, N)
    if not clean:   # past the row's end nothing is written; a page that is not there is still -inf
        end = np.repeat(lens, T) - (T - 1 - np.tile(np.arange(T), B))
        want[np.arange(N)[None] >= np.minimum(end, table.shape[1] * page)[:, None]] = poison
    seen = np.isfinite(want)
    assert same(np.isfinite(got), seen) and np.all(got[~seen] == -np.inf)
    err = np.abs(got - np.where(seen, want, 0))[seen]
    assert np.all(err <= (128 + 32 + 2) * U * size[seen]), err.max()
    if ld is not None:
        base = out.as_strided((B * T, ld), (ld, 1))
        assert (base[:, N:] == poison).all()


@pytest.mark.parametrize("T", [1, 2, 3, 5, 9])
@pytest.mark.parametrize("lens,page", [([1], 64), ([300], 64), ([0, 2, 127, 128, 129, 1000], 16),
                                       ([513, 0, 64], 100), ([77, 78], 1), ([260, 2000], 33)])
def test_logits_sizes(lens, page, T):
    check_logits(np.random.default_rng(T + sum(lens)), lens, T, page)


@pytest.mark.parametrize("clean", [True, False])
def test_logits_windows(clean):
    rng = np.random.default_rng(11)
    check_logits(rng, [200, -3, 0, 1, 333], 2, 64, clean=clean)
    check_logits(rng, [200, 100], 2, 64, N=129, clean=clean)              # lengths past N
    check_logits(rng, [200, 100], 1, 64, N=1001, clean=clean)             # N past the table
    check_logits(rng, [200, 100], 4, 32, N=201, clean=clean, ld=207, layout="joint")
    check_logits(rng, [200, 300], 2, 48, clean=clean, holes=True, layout="heads")


def test_logits_many_rows():
    rng = np.random.default_rng(12)
    check_logits(rng, rng.integers(0, 90, 700), 1, 16)
    check_logits(rng, rng.integers(1000, 3000, 20), 4, 64)


def test_logits_feed_topk():
    rng = np.random.default_rng(13)
    lens = np.array([700, 30, 0], np.int32)
    table, pages = tables(rng, lens, 64)
    data, scale = cache(rng, pages, 64, 1, 128)
    q, w = torch.randn(3, 1, 32, 128, device="cuda").to(F8), torch.randn(3, 1, 32, device="cuda")
    out = fm.logits_paged(q, data, scale, w, gpu(table), gpu(lens))
    idx, _ = fm.topk(out, 64)
    idx = idx.cpu().numpy()
    for b, n in enumerate(lens):
        k = min(64, int(n))
        order = np.argsort(-out[b].cpu().numpy()[:n], kind="stable")[:k]
        assert np.array_equal(idx[b, :k], order) and (idx[b, k:] == -1).all()


# ------------------------------------------------------------------------------------ attention

def check_attention(rng, lens, q_heads, heads, dim, page, dtype=torch.bfloat16, kind=F8, layout="plain", select=None,
                    holes=False, fused=False, shared=False, sharp=1.0, spread=None, indices=None, cols=None):
    lens = np.asarray(lens, np.int32)
    B = len(lens)
    kind = dtype if kind is None else kind
    table, pages = tables(rng, lens[:1] if shared else lens, page, cols=cols)
    if holes:
        table[0, -1] = -7
        table[-1, 0] = pages
    (kd, ks), (vd, vs) = (cache(rng, pages, page, heads, dim, kind, layout) for _ in range(2))
    if spread is not None and vs is not None:
        vs *= torch.from_numpy(np.exp(spread * rng.standard_normal(tuple(vs.shape))).astype(np.float32)).cuda()
    width = q_heads + (2 if fused else 0)
    q = torch.from_numpy(sharp * rng.standard_normal((B, width, dim))).to(dtype).cuda()[:, width - q_heads:]
    if select:
        indices = np.full((B, select + 3), -1, np.int32)
        for b in range(B):
            n = rng.permutation(max(0, int(lens[b])))[:select]
            at = rng.permutation(select)[:len(n)]
            indices[b, at] = n
            indices[b, select:] = [lens[b], -2 ** 31, 2 ** 31 - 1]  # out of range: ignored
    sm = dim ** -0.5
    tab = gpu(table).expand(B, -1) if shared else gpu(table)
    got, lse = fm.attention_paged(q, kd, vd, tab, gpu(lens), sm, k_scale=ks, v_scale=vs,
                                  indices=None if indices is None else gpu(indices), return_lse=True)
    want, wlse, size, dots = plain.attention(f64(q), as_rows(kd, ks), as_rows(vd, vs),
                                             np.broadcast_to(table, (B, table.shape[1])), lens, sm, indices)
    got, lse = got.cpu().double().numpy(), lse.cpu().double().numpy()
    dx = (dim + 8) * U * dots
    bits = 2.0 ** -8 if kind == torch.bfloat16 else 2.0 ** -11
    last = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -11
    tol = (2 * dx[..., None] + 2.0 ** -20 + bits) * size + 2.0 ** -14 * size.max(-1, keepdims=True) + last * np.abs(want) + 1e-7
    assert np.all(np.isfinite(got))
    assert np.all(np.abs(got - want) <= tol), (np.abs(got - want) / tol).max()
    empty = np.isneginf(wlse)
    assert same(np.isneginf(lse), empty) and (got[empty] == 0).all()
    lse, wlse, dx = lse[~empty], wlse[~empty], dx[~empty]
    assert np.all(np.abs(lse - wlse) <= dx + 2.0 ** -20 * (1 + np.abs(wlse)))


TYPES = [(torch.bfloat16, F8), (torch.float16, F8), (torch.bfloat16, None), (torch.float16, None)]


@pytest.mark.parametrize("dtype,kind", TYPES)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("lens,page", [([1], 64), ([0, 2, 31, 32, 33, 500], 16), ([1021], 64), ([77, 300, 0], 33)])
def test_attention_types_and_lengths(lens, page, dim, dtype, kind):
    check_attention(np.random.default_rng(sum(lens) + dim), lens, 8, 2, dim, page, dtype, kind)


@pytest.mark.parametrize("kind", [F8, None])
@pytest.mark.parametrize("q_heads,heads", [(1, 1), (3, 3), (6, 2), (7, 1), (8, 1), (9, 1), (16, 1), (17, 1), (32, 1), (40, 5),
                                           (128, 2), (64, 8)])
def test_attention_head_layouts(q_heads, heads, kind):
    check_attention(np.random.default_rng(q_heads), [65, 200], q_heads, heads, 128, 48, kind=kind)


@pytest.mark.parametrize("dtype,kind", TYPES)
@pytest.mark.parametrize("q_heads,heads,dim", [(2, 2, 128), (8, 2, 64), (12, 4, 128), (32, 2, 128), (64, 4, 64), (48, 6, 128)])
def test_attention_key_heads_side_by_side(q_heads, heads, dim, dtype, kind):
    # two key heads share a CTA where the shares may be long: room for 16 tiles of 64 positions a CTA
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    cols = 16 * 64 * 3 * sms // (2 * heads // 2 * 64)
    rng = np.random.default_rng(q_heads + heads)
    check_attention(rng, [300, 33], q_heads, heads, dim, 64, dtype, kind, cols=cols)
    check_attention(rng, [4000, 0], q_heads, heads, dim, 64, dtype, kind, cols=cols, layout="heads")


@pytest.mark.parametrize("dtype,kind", TYPES)
@pytest.mark.parametrize("q_heads,heads,dim", [(17, 1, 128), (32, 1, 64), (64, 2, 128), (33, 1, 128), (64, 1, 64), (100, 1, 128),
                                               (256, 2, 128)])
def test_attention_groups_that_share_a_ring(q_heads, heads, dim, dtype, kind):
    # wide groups share a ring where the shares may be long: the table has room for that, the sequences
    # are short (64 steps a warp of 3 CTAs an SM, of 32 positions)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    cols = 64 * 32 * 4 * 3 * sms // (2 * heads * 64)
    rng = np.random.default_rng(q_heads)
    check_attention(rng, [300, 33], q_heads, heads, dim, 64, dtype, kind, cols=cols)
    check_attention(rng, [4000, 0], q_heads, heads, dim, 64, dtype, kind, cols=cols)


@pytest.mark.parametrize("kind", [F8, None])
@pytest.mark.parametrize("layout", ["joint", "heads"])
def test_attention_strides_and_missing_pages(layout, kind):
    rng = np.random.default_rng(21)
    check_attention(rng, [300, 129], 8, 4, 128, 32, kind=kind, layout=layout, fused=True)
    check_attention(rng, [300, 129, 10], 8, 4, 64, 32, kind=kind, layout=layout, holes=True)


@pytest.mark.parametrize("kind", [F8, None])
@pytest.mark.parametrize("select", [1, 17, 64, 513])
def test_attention_selected(select, kind):
    rng = np.random.default_rng(select)
    check_attention(rng, [700, 40, 0, 1], 16, 2, 128, 64, kind=kind, select=select)
    check_attention(rng, [900] * 5, 8, 2, 64, 48, kind=kind, select=select, shared=True)


def test_attention_selected_nothing_and_twice():
    rng = np.random.default_rng(31)
    check_attention(rng, [100, 100], 4, 1, 128, 64, indices=np.full((2, 9), -1, np.int32))
    check_attention(rng, [100, 100], 4, 1, 128, 64, indices=np.zeros((2, 0), np.int32))
    check_attention(rng, [100], 4, 1, 128, 64, indices=np.array([[3, 3, 99, 3]], np.int32))


@pytest.mark.parametrize("kind", [F8, None])
def test_attention_long_caches(kind):
    # split over the length and joined: one row, few rows of unequal length, many heads
    rng = np.random.default_rng(41)
    check_attention(rng, [30011], 8, 1, 128, 64, kind=kind)
    check_attention(rng, [9001, 3, 0, 5000], 16, 4, 128, 100, kind=kind)
    check_attention(rng, rng.integers(0, 400, 60), 8, 2, 64, 16, kind=kind)


def test_attention_many_rows():
    rng = np.random.default_rng(42)
    check_attention(rng, rng.integers(0, 70, 1500), 2, 1, 64, 16)


@pytest.mark.parametrize("sharp", [0.0, 30.0])
def test_attention_flat_and_sharp_softmax(sharp):
    check_attention(np.random.default_rng(43), [2000, 100], 8, 2, 128, 64, sharp=sharp)


def test_attention_unequal_value_scales():
    # rows' value scales over many powers of two: the weights keep their bits relative to the largest
    check_attention(np.random.default_rng(44), [700, 90], 8, 2, 128, 64, spread=2.0)


def test_attention_huge_value_scale_of_a_row_that_the_softmax_rules_out():
    # key 0 has value scales 2^60 times the others', and a score 200 or more below them: its weight is 0
    # in 32 bits, and the other rows keep their bits
    rng = np.random.default_rng(47)
    kd, ks = cache(rng, 4, 64, 1, 128)
    vd, vs = cache(rng, 4, 64, 1, 128)
    q = torch.ones(1, 4, 128, device="cuda").to(torch.bfloat16)
    kd.view(torch.uint8)[0, 0] = 0xF8                       # -256 in all columns
    kd.view(torch.uint8)[0, 1:] &= 0x7F                     # the others: positive
    kd.view(torch.uint8)[1:] &= 0x7F
    ks.fill_(2.0 ** -4)
    vs[0, 0] *= 2.0 ** 60
    table, lens = gpu(np.array([[0, 1, 2, 3]], np.int32)), gpu(np.array([256], np.int32))
    got = fm.attention_paged(q, kd, vd, table, lens, k_scale=ks, v_scale=vs).double().cpu().numpy()
    want, _, size, dots = plain.attention(f64(q), as_rows(kd, ks), as_rows(vd, vs) * (np.arange(256).reshape(4, 64, 1, 1) > 0),
                                          table.cpu().numpy(), [256], 128 ** -0.5)
    dx = (128 + 8) * U * dots
    tol = (2 * dx[..., None] + 2.0 ** -20 + 2.0 ** -11) * size + 2.0 ** -14 * size.max(-1, keepdims=True) + 2.0 ** -8 * np.abs(want)
    assert np.all(np.abs(got - want) <= tol)


def test_attention_zero_and_negative_value_scales():
    rng = np.random.default_rng(48)
    kd, ks = cache(rng, 2, 64, 2, 128)
    vd, vs = cache(rng, 2, 64, 2, 128)
    vs[0, ::3] *= -1.0
    vs[1, ::2] = 0.0
    q = torch.from_numpy(rng.standard_normal((2, 8, 128))).to(torch.bfloat16).cuda()
    table, lens = np.array([[1, 0], [1, 0]], np.int32), np.array([128, 1], np.int32)
    got = fm.attention_paged(q, kd, vd, gpu(table), gpu(lens), k_scale=ks, v_scale=vs).double().cpu().numpy()
    want, _, size, dots = plain.attention(f64(q), as_rows(kd, ks), as_rows(vd, vs), table, lens, 128 ** -0.5)
    tol = (2 * (128 + 8) * U * dots[..., None] + 2.0 ** -20 + 2.0 ** -11) * size + 2.0 ** -14 * size.max(-1, keepdims=True) \
        + 2.0 ** -8 * np.abs(want)
    assert np.all(np.abs(got - want) <= tol) and (got[1] == 0).all()


def test_no_pages_at_all():
    kd = torch.empty(0, 64, 2, 128, dtype=F8, device="cuda")
    ks = torch.empty(0, 64, 2, device="cuda")
    table, lens = torch.zeros(2, 3, dtype=torch.int32, device="cuda"), gpu(np.array([100, 0], np.int32))
    out, lse = fm.attention_paged(torch.ones(2, 8, 128, device="cuda").to(torch.bfloat16), kd, kd, table, lens, k_scale=ks,
                                  v_scale=ks, return_lse=True)
    assert (out == 0).all() and torch.isneginf(lse).all()
    logits = fm.logits_paged(torch.ones(2, 1, 32, 128, device="cuda").to(F8), kd[:, :, :1], ks[:, :, :1],
                             torch.ones(2, 1, 32, device="cuda"), table, lens)
    assert torch.isneginf(logits).all()
    rows, by = fm.cache_read(kd, ks, table, gpu(np.array([0, 100, 100], np.int32)), 100)
    assert (rows.view(torch.uint8) == 0).all() and (by == 0).all()
    fm.cache_write(gpu(np.array([0, 5], np.int32)), torch.ones(2, 2, 128, device="cuda"), kd, ks)


def test_attention_beyond_the_length_is_not_read():
    # NaN in the rows past the length, in pages of other sequences and in padding changes nothing
    rng = np.random.default_rng(45)
    kd, ks = cache(rng, 4, 64, 2, 128)
    vd, vs = cache(rng, 4, 64, 2, 128)
    table, lens = gpu(np.array([[2, 0, 1]], np.int32)), gpu(np.array([70], np.int32))
    q = torch.randn(1, 8, 128, device="cuda").to(torch.bfloat16)
    want = fm.attention_paged(q, kd, vd, table, lens, k_scale=ks, v_scale=vs)
    for d, s in ((kd, ks), (vd, vs)):
        d.view(torch.uint8)[0, 6:] = 0x7F
        d.view(torch.uint8)[[1, 3]] = 0x7F
        s[0, 6:] = float("nan")
        s[[1, 3]] = float("inf")
    assert torch.equal(fm.attention_paged(q, kd, vd, table, lens, k_scale=ks, v_scale=vs), want)


def test_attention_offsets_past_32_bits():
    # page strides that put the last page of each cache past 2^32 bytes
    free, _ = torch.cuda.mem_get_info()
    if free < 24 << 30:
        pytest.skip("needs 24 GB of device memory")
    pages, page = 9, 64
    step = (1 << 29) + 16 * 128
    base = torch.empty(pages * step, dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(46)
    small, scale = cache(rng, pages, page, 1, 128)
    data = base.view(F8).as_strided((pages, page, 1, 128), (step, 128, 128, 1))
    data.view(torch.uint8).copy_(small.view(torch.uint8))
    q = torch.randn(1, 4, 128, device="cuda").to(torch.bfloat16)
    table = torch.arange(pages - 1, -1, -1, dtype=torch.int32, device="cuda").view(1, -1)
    lens = torch.tensor([pages * page - 5], dtype=torch.int32, device="cuda")
    a = fm.attention_paged(q, data, data, table, lens, k_scale=scale, v_scale=scale)
    b = fm.attention_paged(q, small, small, table, lens, k_scale=scale, v_scale=scale)
    assert torch.equal(a, b)
    w = torch.randn(1, 1, 32, device="cuda")
    q8 = torch.randn(1, 1, 32, 128, device="cuda").to(F8)
    assert torch.equal(fm.logits_paged(q8, data, scale, w, table, lens), fm.logits_paged(q8, small, scale, w, table, lens))
    starts = torch.tensor([0, pages * page - 5], dtype=torch.int32, device="cuda")
    got = fm.cache_read(data, scale, table, starts, pages * page - 5)
    want = fm.cache_read(small, scale, table, starts, pages * page - 5)
    assert torch.equal(got[0].view(torch.uint8), want[0].view(torch.uint8))
    x = torch.randn(pages * page, 1, 128, device="cuda").to(torch.bfloat16)
    slots = torch.arange(pages * page, dtype=torch.int32, device="cuda")
    fm.cache_write(slots, x, data, scale)
    fm.cache_write(slots, x, small, scale)
    assert torch.equal(data.view(torch.uint8), small.view(torch.uint8).as_strided(small.shape, small.stride()))


# ------------------------------------------------------------------------------------ streams, graphs, repeats

def _attention_inputs(seed, lens=(5000, 17, 0, 900)):
    rng = np.random.default_rng(seed)
    lens = np.array(lens, np.int32)
    table, pages = tables(rng, lens, 64)
    kd, ks = cache(rng, pages, 64, 2, 128)
    vd, vs = cache(rng, pages, 64, 2, 128)
    q = torch.from_numpy(rng.standard_normal((len(lens), 16, 128))).to(torch.bfloat16).cuda()
    return (q, kd, vd, gpu(table), gpu(lens), None, ks, vs)


def test_attention_is_the_same_every_time_and_on_any_stream():
    sets = [_attention_inputs(s) for s in (51, 52)]
    want = [fm.attention_paged(*a, return_lse=True) for a in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    got = []
    for i in range(40):  # calls that overlap, on streams that are not the current one
        got.append((i % 2, fm.attention_paged(*sets[i % 2], return_lse=True, stream=streams[i % 4])))
    torch.cuda.synchronize()
    for i, (out, lse) in got:
        assert torch.equal(out, want[i][0]) and torch.equal(lse, want[i][1])


def test_calls_see_what_the_kernel_before_them_wrote():
    # steps whose kernels follow one another closely (each is set up while the one before ends) give what
    # the same steps give with the device idle between any two
    rng = np.random.default_rng(56)
    B, page, cols, steps = 3, 16, 8, 60
    first = {}
    for name, heads in (("k", 2), ("v", 2), ("i", 1)):
        first[name] = cache(rng, B * cols, page, heads, 128)
    table = torch.arange(B * cols, dtype=torch.int32, device="cuda").view(B, cols)
    x = torch.from_numpy(rng.standard_normal((steps, B, 5, 128))).to(torch.bfloat16).cuda()
    q = torch.from_numpy(rng.standard_normal((steps, B, 8, 128))).to(torch.bfloat16).cuda()
    q8 = torch.from_numpy(rng.standard_normal((steps, B, 1, 32, 128))).float().to(F8).cuda()
    w = torch.from_numpy(rng.standard_normal((steps, B, 1, 32)).astype(np.float32)).cuda()

    def run(pause):
        c = {n: (d.clone(), s.clone()) for n, (d, s) in first.items()}
        lens = torch.zeros(B, dtype=torch.int32, device="cuda")
        starts = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
        slots = torch.empty(B, dtype=torch.int32, device="cuda")
        out = []
        for t in range(steps):
            torch.add(torch.arange(B, dtype=torch.int32, device="cuda") * cols * page, lens, out=slots)
            pause()
            fm.cache_write(slots, x[t, :, :2], *c["k"], x[t, :, 2:4], *c["v"])
            pause()
            fm.cache_write(slots, x[t, :, 4:], *c["i"])
            pause()
            lens.add_(1)
            starts[1:] = lens.cumsum(0)
            pause()
            logits = fm.logits_paged(q8[t], *c["i"], w[t], table, lens)
            pause()
            idx, _ = fm.topk(logits, 8)
            pause()
            out += [logits, idx, fm.attention_paged(q[t], c["k"][0], c["v"][0], table, lens, k_scale=c["k"][1],
                                                    v_scale=c["v"][1], indices=idx)]
            pause()
            out.append(fm.attention_paged(q[t], c["k"][0], c["v"][0], table, lens, k_scale=c["k"][1], v_scale=c["v"][1]))
            pause()
            out.append(fm.cache_read(*c["k"], table, starts, B * (t + 1), dtype=torch.float32))
            pause()
        torch.cuda.synchronize()
        return out

    want = run(torch.cuda.synchronize)
    for _ in range(3):
        for a, b in zip(run(lambda: None), want):
            assert torch.equal(a, b)


def test_operators_in_a_graph():
    rng = np.random.default_rng(53)
    a = _attention_inputs(54)
    q8 = torch.from_numpy(rng.standard_normal((4, 1, 32, 128))).float().to(F8).cuda()
    w = torch.from_numpy(rng.standard_normal((4, 1, 32)).astype(np.float32)).cuda()
    data, scale = cache(rng, a[1].shape[0], 64, 1, 128)
    x = torch.from_numpy(rng.standard_normal((4, 1, 128))).to(torch.bfloat16).cuda()
    slots = torch.tensor([0, 65, -1, 130], dtype=torch.int32, device="cuda")

    def step():
        fm.cache_write(slots, x, data, scale)
        logits = fm.logits_paged(q8, data, scale, w, a[3], a[4])
        idx, _ = fm.topk(logits, 64, sorted=True)
        return logits, fm.attention_paged(*a, indices=idx), fm.attention_paged(*a)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        want = step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(3):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for g, e in zip(got, want):
            assert torch.equal(g, e)


def test_the_bounds_checking_library_has_the_operators_too():
    a = _attention_inputs(57)
    want = fm.attention_paged(*a)
    fm.use_debug_library(True)
    try:
        got = fm.attention_paged(*a)
        torch.cuda.synchronize()
        assert fm.check_error() == 0
    finally:
        fm.use_debug_library(False)
    assert torch.equal(got, want)


def test_refusals_on_the_gpu():
    q, kd, vd, table, lens, _, ks, vs = _attention_inputs(55)
    call = fm.attention_paged
    for bad in (dict(k_scale=None), dict(v_scale=ks[:1])):
        with pytest.raises((TypeError, ValueError)):
            call(q, kd, vd, table, lens, **{**dict(k_scale=ks, v_scale=vs), **bad})
    with pytest.raises(ValueError, match="does not go with"):
        call(q[:, :15], kd, vd, table, lens, k_scale=ks, v_scale=vs)
    with pytest.raises(TypeError):
        call(q.float(), kd, vd, table, lens, k_scale=ks, v_scale=vs)
    with pytest.raises(TypeError):
        call(q, kd.to(torch.float16), vd.to(torch.float16), table, lens)
    with pytest.raises(TypeError):
        call(q, kd, vd, table.long(), lens, k_scale=ks, v_scale=vs)
    with pytest.raises(ValueError):
        call(q, kd, vd, table[:2], lens, k_scale=ks, v_scale=vs)
    with pytest.raises(fm.Fp8MqaError):  # a width that no kernel has
        call(q[..., :32], kd[..., :32], vd[..., :32], table, lens, k_scale=ks, v_scale=vs)
    with pytest.raises(fm.Fp8MqaError):  # rows that do not start on 16 bytes
        call(q[..., :64].contiguous(), kd[..., 8:72], vd[..., 8:72], table, lens, k_scale=ks, v_scale=vs)
    x = torch.zeros(4, 2, 128, dtype=torch.bfloat16, device="cuda")
    slots = torch.arange(4, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        fm.cache_write(slots, x, kd, ks, x)
    with pytest.raises(ValueError):
        fm.cache_write(slots[:3], x, kd, ks)
    with pytest.raises(TypeError):
        fm.cache_write(slots, x, kd, ks, x.float(), vd, vs)
    with pytest.raises(TypeError):
        fm.cache_read(kd, ks, table, torch.zeros(5, dtype=torch.int32, device="cuda"), 3, dtype=torch.float64)
    with pytest.raises(ValueError):
        fm.logits_paged(torch.zeros(4, 1, 32, 128, device="cuda").to(F8), kd, ks, torch.zeros(4, 1, 32, device="cuda"), table, lens)
    # no rows: nothing to do
    assert call(q[:0], kd, vd, table[:0], lens[:0], k_scale=ks, v_scale=vs).shape == (0, 16, 128)
    fm.cache_write(slots[:0], x[:0], kd, ks)
