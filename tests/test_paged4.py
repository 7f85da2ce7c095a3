"""Paged caches in 4 bits: writing, reading and attention against their plain forms.

cache_write and cache_read are exact: every step is defined in fp32.  attention_paged has the tolerance of E4M3
caches (test_paged.py): a value's data * group is exact in the 16 bits that are multiplied, so it is the
scores' fp32 sums, the weights' 11 bits and the result's rounding again.
"""
import struct

import numpy as np
import pytest
import torch

import fp8_mqa_logits_02_gb300 as fm
from oracle import paged as plain
from oracle import step
from test_paged import U, f64, gpu, same, tables

pytestmark = pytest.mark.gpu

F4, F8 = torch.float4_e2m1fn_x2, torch.float8_e4m3fn
TYPES = [torch.bfloat16, torch.float16]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    fm.build()
    fm.lib()


def cache(rng, pages, page, heads, dim, layout="plain", spread=0.5):
    """(codes, groups, scale) on the GPU, filled; "joint" is one half of [pages, 2, ...], "heads" puts heads before rows."""
    n = {"plain": (pages, page, heads), "joint": (pages, 2, page, heads), "heads": (pages, heads, page)}[layout]
    codes = torch.from_numpy(rng.integers(0, 256, n + (dim // 2,), np.uint8)).cuda()
    groups = np.exp(spread * rng.standard_normal(n + (dim // 16,))) * 60
    groups = torch.from_numpy(np.clip(groups, 0, 448)).float().to(F8).cuda()
    scale = torch.from_numpy((0.004 * np.exp(rng.standard_normal(n))).astype(np.float32)).cuda()
    pick = {"plain": lambda t: t, "joint": lambda t: t[:, 1], "heads": lambda t: t.transpose(1, 2)}[layout]
    return pick(codes), pick(groups), pick(scale)


def values(c):
    """The data's values times the groups' scales, exact."""
    return step.unpack(c[0].cpu().numpy()) * np.repeat(f64(c[1]), 16, -1)


def as_rows(c):
    with np.errstate(invalid="ignore"):
        return values(c) * f64(c[2])[..., None]


# ------------------------------------------------------------------------------------ write

def check_write(x, slots, caches, pairs):
    """Writes rows into one cache or two, and looks at every byte of them afterwards."""
    want = [[step.unpack(c[0].cpu().numpy()), f64(c[1]), f64(c[2])] for c in caches]
    more = () if pairs is None else (pairs, caches[1][0].view(F4), caches[1][2])
    fm.cache_write(gpu(slots), x, caches[0][0].view(F4), caches[0][2], *more, k_groups=caches[0][1],
                   v_groups=None if pairs is None else caches[1][1])
    pages, page = caches[0][2].shape[:2]
    ok = (slots >= 0) & (slots < pages * page)
    at = (slots[ok] // page, slots[ok] % page)
    for rows, c, w in zip((x, pairs), caches, want):
        for to, new in zip(w, step.quantise4(rows.float().cpu().numpy())):
            to[at] = new[ok]
        assert same(step.unpack(c[0].cpu().numpy()), w[0])
        assert same(f64(c[1]), w[1]) and same(f64(c[2]), w[2])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("T,heads,dim,page", [(1, 1, 128, 64), (7, 8, 64, 1), (33, 3, 128, 16), (130, 2, 64, 100),
                                              (257, 1, 128, 33)])
def test_write_pair_is_exact(T, heads, dim, page, dtype):
    rng = np.random.default_rng(T * 7 + heads)
    pages = -(-T // page) + 2
    caches = [cache(rng, pages, page, heads, dim) for _ in range(2)]
    qkv = torch.from_numpy(rng.standard_normal((T, 2 * heads + 3, dim)) * np.exp(rng.standard_normal((T, 1, 1)))).to(dtype).cuda()
    slots = rng.permutation(pages * page)[:T].astype(np.int32)
    slots[::5] = [-1, pages * page, -2 ** 31, 2 ** 31 - 1][T % 4]  # padding and slots out of range
    check_write(qkv[:, 1:1 + heads], slots, caches, qkv[:, 2 + heads:2 + 2 * heads])


def test_write_pair_into_caches_of_two_layouts():
    rng = np.random.default_rng(21)
    x = torch.from_numpy(rng.standard_normal((50, 8, 128))).to(torch.float16).cuda()
    caches = [cache(rng, 5, 24, 4, 128, layout="heads"), cache(rng, 5, 24, 4, 128, layout="joint")]
    check_write(x[:, :4], rng.permutation(120)[:50].astype(np.int32), caches, x[:, 4:])


@pytest.mark.parametrize("layout", ["joint", "heads"])
def test_write_one_into_strided_cache(layout):
    rng = np.random.default_rng(3)
    x = torch.from_numpy(rng.standard_normal((50, 4, 128))).to(torch.bfloat16).cuda()
    check_write(x, rng.permutation(120)[:50].astype(np.int32), [cache(rng, 5, 24, 4, 128, layout=layout)], None)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_write_unaligned_rows(dtype):
    # rows of 64 values 65 elements apart, from an odd element on
    rng = np.random.default_rng(4)
    flat = torch.from_numpy(rng.standard_normal(1 + 40 * 65)).to(dtype).cuda()
    check_write(flat.as_strided((20, 2, 64), (130, 65, 1), 1), np.arange(20, dtype=np.int32), [cache(rng, 2, 16, 2, 64)], None)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_ties_of_16_bit_rows_fall_as_in_real_numbers(dtype):
    # small whole numbers over small whole numbers hit the midpoints of both roundings again and again
    rng = np.random.default_rng(5)
    x = rng.integers(-28, 29, (4000, 1, 128)) * np.exp2(rng.integers(-12, 12, (4000, 1, 1)))
    rows = torch.from_numpy(x).to(dtype)
    assert torch.equal(rows.double(), torch.from_numpy(x))
    c = cache(rng, 4000, 1, 1, 128)
    fm.cache_write(torch.arange(4000, dtype=torch.int32, device="cuda"), rows.cuda(), c[0].view(F4), c[2], k_groups=c[1])
    a = np.abs(x).max(-1, keepdims=True)
    m = np.abs(x.reshape(4000, 1, 8, 16)).max(-1)
    groups = plain.round_e4m3(448 * m / a)               # quotients correct to 53 bits: a tie is exact
    by = groups[..., None] * a[..., None]
    v = np.where(by > 0, step.round_e2m1(2688 * x.reshape(4000, 1, 8, 16) / np.where(by > 0, by, 1)), 0)
    assert same(f64(c[1])[:, 0], groups) and same(step.unpack(c[0].cpu().numpy())[:, 0], v.reshape(4000, 1, 128))


def test_write_special_rows():
    x = torch.zeros(12, 1, 64)
    x[1] = 3e38                       # the largest magnitudes
    x[2] = 1e-38                      # under the least maximum: still finite
    x[3, 0, 5] = float("nan")
    x[4, 0, 6] = float("inf")
    x[5, 0, 7] = -float("inf")
    x[6] = torch.linspace(-1, 1, 64)
    x[7, 0, 0] = -1e-45
    x[8] = torch.linspace(-1, 1, 64) * 2.5e-30
    x[9, 0, 0], x[9, 0, 20] = 1e5, 1e-3      # a group of so small values that its scale is 0
    x[10, 0] = float("inf")
    x[11] = torch.linspace(-1, 1, 64) * 3.3e38
    rng = np.random.default_rng(0)
    c = cache(rng, 1, 12, 1, 64)
    fm.cache_write(torch.arange(12, dtype=torch.int32, device="cuda"), x.cuda(), c[0].view(F4), c[2], k_groups=c[1])
    got = as_rows(c).reshape(12, 64)
    assert np.isnan(got[[3, 4, 5, 10]]).all()
    fine = [0, 1, 2, 6, 7, 8, 9, 11]
    assert np.isfinite(got[fine]).all()
    v, groups, scale = step.quantise4(x.numpy()[fine])
    assert same(step.unpack(c[0].cpu().numpy())[0, fine], v)
    assert same(f64(c[1])[0, fine], groups) and same(f64(c[2])[0, fine], scale.astype(np.float64))
    # against the row itself: a group's scale is off by 2^-4 at most (so its largest value may be cut by as much),
    # and a value by half a step of its own, 1/4 up to 1 or 1/4 of it above, in units of at most m / 6 (1 + 2^-4)
    for r in (6, 8, 11):
        want = x[r, 0].double().numpy()
        m = np.repeat(np.abs(want.reshape(4, 16)).max(-1), 16)
        assert np.all(np.abs(got[r] - want) <= (1 + 2.0 ** -4) * np.maximum(m / 24, np.abs(want) / 4))


# ------------------------------------------------------------------------------------ read

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("lens,heads,dim,page,layout", [
    ([5], 1, 128, 64, "plain"), ([0, 3, 0, 0, 70, 1, 0], 2, 64, 16, "plain"), ([129, 64, 1], 8, 128, 33, "heads"),
    ([40, 41], 4, 64, 1, "joint"), ([1] * 50 + [0] * 20 + [300], 1, 128, 100, "plain"), ([2000, 1500], 8, 128, 64, "plain")])
def test_read_is_exact(lens, heads, dim, page, layout, dtype):
    rng = np.random.default_rng(sum(lens))
    table, pages = tables(rng, lens, page)
    c = cache(rng, pages, page, heads, dim, layout)
    if len(lens) > 2:
        table[-1, 0] = pages          # a page that is not there reads as zeros
    starts = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    total = int(starts[-1]) + 3       # rows past the last sequence are zeroed
    got = fm.cache_read(c[0].view(F4), c[2], gpu(table), gpu(starts), total, dtype=dtype, groups=c[1])
    want, by = np.zeros((total, heads, dim), np.float32), np.zeros((total, heads), np.float32)
    d, s = values(c).astype(np.float32), c[2].cpu().numpy()
    for b, n in enumerate(lens):
        there, ids, row = plain.rows(d, table[b], np.arange(n), pages, page)
        want[starts[b]:starts[b] + n] = np.where(there[:, None, None], d[ids, row], 0)
        by[starts[b]:starts[b] + n] = np.where(there[:, None], s[ids, row], 0)
    assert torch.equal(got.cpu(), torch.from_numpy(want * by[..., None]).to(dtype))


@pytest.mark.parametrize("kind,dtype", [(1, torch.bfloat16), (2, torch.float16), (3, torch.float32)])
def test_read_to_16_bytes(kind, dtype):
    # through the C entry, whose results lie on 16 bytes and need not on 32
    rng = np.random.default_rng(22)
    table, pages = tables(rng, [70, 9], 16)
    c = cache(rng, pages, 16, 2, 64)
    starts = gpu(np.array([0, 70, 79], np.int32))
    want = fm.cache_read(c[0].view(F4), c[2], gpu(table), starts, 79, dtype=dtype, groups=c[1])
    to = torch.full((79 * 128 + 64,), 5.0, dtype=dtype, device="cuda")
    at = 16 // to.element_size()
    st = [s for t in (c[0], c[2]) for s in t.stride()[:3]]
    struct_ = struct.pack("@PPqiiiiqqqqqqPqqq", c[0].data_ptr(), c[2].data_ptr(), pages, 16, 2, 64, 4, *st, c[1].data_ptr(),
                          *c[1].stride()[:3])
    t = gpu(table)
    assert fm.lib().fp8_mqa_cache_read(struct_, t.data_ptr(), t.stride(0), t.shape[1], starts.data_ptr(), 2, 79, kind,
                                       to.data_ptr() + 16, None, None) == 0
    torch.cuda.synchronize()
    assert torch.equal(to[at:at + 79 * 128].view(79, 2, 64), want)
    assert (to[:at] == 5).all() and (to[at + 79 * 128:] == 5).all()


# ------------------------------------------------------------------------------------ attention

def close(got, lse, want, wlse, size, dots, dtype):
    """The tolerance of test_paged.py."""
    got, lse, dim = f64(got), f64(lse), got.shape[-1]
    dx = (dim + 8) * U * dots
    last = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -11
    tol = (2 * dx[..., None] + 2.0 ** -20 + 2.0 ** -11) * size + 2.0 ** -14 * size.max(-1, keepdims=True) + last * np.abs(want) + 1e-7
    assert np.all(np.isfinite(got))
    assert np.all(np.abs(got - want) <= tol), (np.abs(got - want) / tol).max()
    empty = np.isneginf(wlse)
    assert same(np.isneginf(lse), empty) and (got[empty] == 0).all()
    lse, wlse, dx = lse[~empty], wlse[~empty], dx[~empty]
    assert np.all(np.abs(lse - wlse) <= dx + 2.0 ** -20 * (1 + np.abs(wlse)))


def check_attention(rng, lens, q_heads, heads, dim, page, dtype=torch.bfloat16, layout="plain", select=None, holes=False,
                    fused=False, shared=False, sharp=1.0, spread=None, cols=None, negative=False, sm=None, v_layout=None):
    lens = np.asarray(lens, np.int32)
    B = len(lens)
    table, pages = tables(rng, lens[:1] if shared else lens, page, cols=cols)
    if holes:
        table[0, -1] = -7
        table[-1, 0] = pages
    if holes == "many":
        at = rng.permutation(table.shape[1])[:table.shape[1] // 5]
        table[:, at] = rng.choice([-1, pages, 2 ** 31 - 1], len(at))
    k, v = cache(rng, pages, page, heads, dim, layout), cache(rng, pages, page, heads, dim, v_layout or layout)
    if spread is not None:
        v[2].mul_(torch.from_numpy(np.exp(spread * rng.standard_normal(tuple(v[2].shape))).astype(np.float32)).cuda())
    if negative:
        v[2].mul_(torch.from_numpy(rng.choice([-1.0, 1.0], tuple(v[2].shape)).astype(np.float32)).cuda())
    width = q_heads + (2 if fused else 0)
    q = torch.from_numpy(sharp * rng.standard_normal((B, width, dim))).to(dtype).cuda()[:, width - q_heads:]
    indices = None
    if select:
        indices = np.full((B, select + 3), -1, np.int32)
        for b in range(B):
            n = rng.permutation(max(0, int(lens[b])))[:select]
            indices[b, rng.permutation(select)[:len(n)]] = n
            indices[b, select:] = [lens[b], -2 ** 31, 2 ** 31 - 1]  # out of range: ignored
    sm = dim ** -0.5 if sm is None else sm
    tab = gpu(table).expand(B, -1) if shared else gpu(table)
    got, lse = fm.attention_paged(q, k[0].view(F4), v[0].view(F4), tab, gpu(lens), sm, k_scale=k[2], v_scale=v[2],
                                  indices=None if indices is None else gpu(indices), return_lse=True, k_groups=k[1],
                                  v_groups=v[1])
    want, wlse, size, dots = plain.attention(f64(q), as_rows(k), as_rows(v), np.broadcast_to(table, (B, table.shape[1])),
                                             lens, sm, indices)
    close(got, lse, want, wlse, size, dots, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("lens,page", [([1], 64), ([0, 2, 31, 32, 33, 500], 16), ([1021], 64), ([77, 300, 0], 33),
                                       ([63, 64, 65, 127, 128, 129], 1)])
def test_attention_types_and_lengths(lens, page, dim, dtype):
    check_attention(np.random.default_rng(sum(lens) + dim), lens, 8, 2, dim, page, dtype)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("q_heads,heads", [(1, 1), (3, 3), (6, 2), (7, 1), (8, 1), (9, 1), (16, 1), (17, 1), (32, 1), (40, 5),
                                           (128, 2), (64, 8)])
def test_attention_head_layouts(q_heads, heads, dim):
    check_attention(np.random.default_rng(q_heads), [65, 200], q_heads, heads, dim, 48)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("q_heads,heads,dim", [(2, 2, 128), (8, 2, 64), (12, 4, 128), (32, 2, 128), (64, 4, 64), (48, 6, 128)])
def test_attention_key_heads_side_by_side(q_heads, heads, dim, dtype):
    # a table wide enough that two key heads share a CTA
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    check_attention(np.random.default_rng(q_heads + dim), [700, 1, 64], q_heads, heads, dim, 64, dtype, cols=sms * 24 // heads)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("q_heads,heads", [(32, 1), (20, 1), (64, 1), (100, 2), (256, 2)])
def test_attention_groups_that_share_a_ring(q_heads, heads, dim):
    # a table so wide that the shares are long
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    check_attention(np.random.default_rng(q_heads + dim), [333, 40], q_heads, heads, dim, 64, cols=sms * 512 // heads)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [64, 128])
def test_attention_layouts_holes_and_selected(dim, dtype):
    rng = np.random.default_rng(dim)
    check_attention(rng, [300, 129, 10], 8, 4, dim, 32, dtype, layout="joint", holes=True, fused=True)
    check_attention(rng, [300, 129, 10], 8, 4, dim, 32, dtype, layout="heads", holes=True, select=64)
    check_attention(rng, [900] * 5, 8, 2, dim, 48, dtype, select=513, shared=True)
    check_attention(rng, [500, 0, 3], 4, 1, dim, 16, dtype, select=1)


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("dim", [64, 128])
def test_attention_keys_and_values_of_two_layouts(dim, page):
    rng = np.random.default_rng(23)
    check_attention(rng, [300, 129, 10], 8, 4, dim, page, layout="heads", v_layout="plain")
    check_attention(rng, [300, 129, 10], 8, 4, dim, page, layout="joint", v_layout="heads", select=64, holes=True)
    check_attention(rng, [3000], 32, 1, dim, page, layout="plain", v_layout="joint")


def test_attention_without_pages_or_columns():
    f = lambda *n: torch.zeros(n, dtype=torch.uint8, device="cuda")  # noqa: E731
    q = torch.ones(2, 4, 128, device="cuda").bfloat16()
    lens = gpu(np.array([5, 0], np.int32))
    for pages, cols in ((0, 3), (2, 0)):
        data, groups, scale = f(pages, 32, 2, 64).view(F4), f(pages, 32, 2, 8).view(F8), torch.ones(pages, 32, 2, device="cuda")
        for indices in (None, torch.zeros(2, 9, dtype=torch.int32, device="cuda")):
            out, lse = fm.attention_paged(q, data, data, torch.zeros(2, cols, dtype=torch.int32, device="cuda"), lens, k_scale=scale,
                                          v_scale=scale, k_groups=groups, v_groups=groups, indices=indices, return_lse=True)
            assert (out == 0).all() and lse.isneginf().all()
        rows = fm.cache_read(data, scale, torch.zeros(2, cols, dtype=torch.int32, device="cuda"),
                             torch.tensor([0, 5, 5], dtype=torch.int32, device="cuda"), 5, dtype=torch.float32, groups=groups)
        assert (rows == 0).all()
        fm.cache_write(torch.zeros(3, dtype=torch.int32, device="cuda") + 64, torch.ones(3, 2, 128, device="cuda"), data, scale,
                       k_groups=groups)


def test_attention_captured_and_replayed():
    rng = np.random.default_rng(24)
    table, pages = tables(rng, [500, 64, 1], 64)
    k, v = cache(rng, pages, 64, 2, 128), cache(rng, pages, 64, 2, 128)
    q, t, lens = torch.zeros(3, 8, 128, device="cuda").bfloat16(), gpu(table), gpu(np.array([1, 1, 1], np.int32))
    call = lambda: fm.attention_paged(q, k[0].view(F4), v[0].view(F4), t, lens, k_scale=k[2], v_scale=v[2],  # noqa: E731
                                      k_groups=k[1], v_groups=v[1], return_lse=True)
    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    for n in ([500, 64, 1], [0, 33, 1], [499, 0, 0]):
        lens.copy_(gpu(np.array(n, np.int32)))
        q.copy_(torch.from_numpy(rng.standard_normal((3, 8, 128))))
        graph.replay()
        close(*got, *plain.attention(f64(q), as_rows(k), as_rows(v), table, n, 128 ** -0.5), q.dtype)


def test_attention_split_and_joined():
    rng = np.random.default_rng(9)
    check_attention(rng, [30011], 8, 1, 128, 64)
    check_attention(rng, [40000, 1, 20001], 32, 2, 64, 128)
    check_attention(rng, [9001, 3, 0, 5000], 16, 4, 128, 100)
    check_attention(rng, list(rng.integers(0, 300, 500)), 4, 2, 128, 16)


@pytest.mark.parametrize("holes", [False, "many"])
@pytest.mark.parametrize("page", [32, 64, 160])
def test_attention_of_many_steps_a_warp(page, holes):
    # a warp looks up the pages of 32 steps at once: twice or more here (rows share their pages)
    lens = np.r_[np.full(60, 26000), 25999, 25001, 0, 33]
    check_attention(np.random.default_rng(page), lens, 2, 2, 64, page, shared=True, holes=holes)


def test_attention_sharp_scores_and_wide_scales():
    rng = np.random.default_rng(10)
    for dtype in TYPES:
        check_attention(rng, [400, 1000], 8, 2, 128, 64, dtype, sharp=30.0)
        check_attention(rng, [400, 1000], 8, 2, 128, 64, dtype, spread=4.0)
        check_attention(rng, [400, 1000], 8, 2, 64, 64, dtype, negative=True)


@pytest.mark.parametrize("dtype", TYPES)
def test_attention_scales_of_the_scores(dtype):
    rng = np.random.default_rng(14)
    for sm in (0.0, -0.05, -dim_root(64), 1e-30, 3.0):
        check_attention(rng, [200, 0, 65], 8, 2, 64, 32, dtype, sm=sm)
        check_attention(rng, [300], 4, 1, 128, 64, dtype, sm=sm, holes=True)


def dim_root(dim):
    return float(np.float32(dim ** -0.5))


def test_attention_scores_that_rise_and_fall():
    # keys grow from page to page and shrink again, so that the references move step after step, and stay far behind
    for dtype in TYPES:
        for power in (1.0, -1.0):
            rng = np.random.default_rng(15)
            table, pages = tables(rng, [900], 64)
            k, v = cache(rng, pages, 64, 2, 128), cache(rng, pages, 64, 2, 128)
            at = torch.arange(15, device="cuda", dtype=torch.float32)
            k[2][torch.from_numpy(table[0].astype(np.int64)).cuda()] = (0.0002 * 1.5 ** (power * (at - 7)))[:, None, None]
            q = torch.from_numpy(np.abs(rng.standard_normal((1, 8, 128)))).to(dtype).cuda()
            got, lse = fm.attention_paged(q, k[0].view(F4), v[0].view(F4), gpu(table), gpu(np.array([900], np.int32)),
                                          k_scale=k[2], v_scale=v[2], k_groups=k[1], v_groups=v[1], return_lse=True)
            close(got, lse, *plain.attention(f64(q), as_rows(k), as_rows(v), table, [900], 128 ** -0.5), dtype)


def test_attention_of_nan_and_zero_rows():
    rng = np.random.default_rng(11)
    k, v = cache(rng, 2, 64, 1, 128), cache(rng, 2, 64, 1, 128)
    v[2][0, 5] = 0.0                                # a row of zeros
    k[1][0, 6] = 0.0                                # groups of zero: a key of zeros
    q = torch.randn(1, 4, 128, device="cuda").bfloat16()
    table, lens = gpu(np.array([[0, 1]])), gpu(np.array([100]))
    call = lambda: fm.attention_paged(q, k[0].view(F4), v[0].view(F4), table.int(), lens.int(), k_scale=k[2],  # noqa: E731
                                      v_scale=v[2], k_groups=k[1], v_groups=v[1], return_lse=True)
    got, lse = call()
    close(got, lse, *plain.attention(f64(q), as_rows(k), as_rows(v), np.array([[0, 1]]), [100], 128 ** -0.5), q.dtype)
    k[2][1, 63] = v[2][1, 63] = float("nan")        # past the row's end: not looked at
    assert torch.equal(call()[0], got)
    v[2][0, 7] = float("nan")                       # a row that stands for NaN
    assert call()[0].isnan().all()


def test_attention_over_a_cache_past_32_bits():
    # keys and values further apart than 2^32 bytes, in one tensor
    pages, page, heads, dim = 9000, 128, 64, 128
    if torch.cuda.mem_get_info()[0] < 20 << 30:
        pytest.skip("needs 20 GB of device memory")
    rng = np.random.default_rng(12)
    codes = torch.randint(0, 256, (pages, page, heads, dim // 2), dtype=torch.uint8, device="cuda")
    assert codes.numel() > 2 ** 32
    groups = torch.ones(pages, page, heads, dim // 16, device="cuda").to(F8)
    scale = torch.full((pages, page, heads), 0.25, device="cuda")
    table = np.array([[8999, 0, 8998], [8500, 7, 3]], np.int32)
    lens = np.array([300, 257], np.int32)
    q = torch.from_numpy(rng.standard_normal((2, 64, dim))).to(torch.bfloat16).cuda()
    got, lse = fm.attention_paged(q, codes.view(F4), codes.view(F4), gpu(table), gpu(lens), k_scale=scale, v_scale=scale,
                                  k_groups=groups, v_groups=groups, return_lse=True)
    used = sorted(set(table.ravel().tolist()))
    small = step.unpack(codes[used].cpu().numpy()) * 0.25
    at = np.vectorize(used.index)(table)
    close(got, lse, *plain.attention(f64(q), small, small, at, lens, dim ** -0.5), q.dtype)


def test_write_then_attend_closely_following():
    # each step reads what the one before it wrote, on one stream with nothing in between
    rng = np.random.default_rng(13)
    k, v = cache(rng, 4, 64, 2, 128), cache(rng, 4, 64, 2, 128)
    table = gpu(np.array([[2, 0, 3, 1]], np.int32))
    x = torch.from_numpy(rng.standard_normal((200, 2, 2, 128))).to(torch.bfloat16).cuda()
    q = torch.from_numpy(rng.standard_normal((1, 8, 128))).to(torch.bfloat16).cuda()
    n = torch.arange(201, dtype=torch.int32, device="cuda")
    outs = []
    slots = (table[0, (n[:200] // 64).long()] * 64 + n[:200] % 64).to(torch.int32)
    for i in range(200):
        fm.cache_write(slots[i:i + 1], x[i:i + 1, 0], k[0].view(F4), k[2], x[i:i + 1, 1], v[0].view(F4), v[2],
                       k_groups=k[1], v_groups=v[1])
        outs.append(fm.attention_paged(q, k[0].view(F4), v[0].view(F4), table, n[i + 1:i + 2], k_scale=k[2], v_scale=v[2],
                                       k_groups=k[1], v_groups=v[1], return_lse=True))
    for i in (0, 1, 63, 64, 65, 199):
        want = plain.attention(f64(q), as_rows(k), as_rows(v), table.cpu().numpy(), [i + 1], 128 ** -0.5)
        close(*outs[i], *want, q.dtype)
