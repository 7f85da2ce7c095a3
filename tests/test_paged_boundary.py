"""The paged-cache entry points without a GPU: bad arguments are refused on the host before any
device work, and the 64-bit plain forms that the GPU tests compare with are pinned by hand."""
import ctypes
import struct

import numpy as np
import pytest
import torch

import fp8_mqa_logits_02_gb300 as fm
from oracle import paged as plain

OK, INVALID, UNSUPPORTED, MISALIGNED = 0, -1, -2, -3
E4M3, BF16, F16, F32 = 0, 1, 2, 3
P = 0x1000  # an aligned address that is never read


@pytest.fixture(scope="module")
def lib():
    fm.build()
    return fm.lib()


def cache(data=P, scale=P, pages=4, page=16, heads=1, dim=128, type=E4M3, strides=None):
    s = strides or (page * heads * dim, heads * dim, dim, page * heads, heads, 1)
    return struct.pack("@PPqiiiiqqqqqq", data or 0, scale or 0, pages, page, heads, dim, type, *s)


def test_header_struct_is_what_the_binding_packs():
    class Cache(ctypes.Structure):
        _fields_ = [("data", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("pages", ctypes.c_int64)] + \
            [(n, ctypes.c_int32) for n in ("page_size", "heads", "dim", "type")] + \
            [(n, ctypes.c_int64) for n in "abcdef"]
    assert ctypes.sizeof(Cache) == len(cache())
    c = Cache.from_buffer_copy(cache(type=2, pages=7))
    assert (c.pages, c.page_size, c.heads, c.dim, c.type) == (7, 16, 1, 128, 2)


@pytest.mark.parametrize("bad,status", [
    (dict(pages=-1), INVALID), (dict(page=0), INVALID), (dict(heads=0), INVALID), (dict(data=None), INVALID),
    (dict(scale=None), INVALID), (dict(type=7), INVALID), (dict(type=F32), INVALID), (dict(dim=96), UNSUPPORTED),
    (dict(pages=1 << 28), UNSUPPORTED), (dict(data=P + 8), MISALIGNED), (dict(scale=P + 2), MISALIGNED),
    (dict(strides=(2048 + 8, 128, 128, 16, 1, 1)), MISALIGNED), (dict(strides=(2048, 132, 128, 16, 1, 1)), MISALIGNED),
    (dict(heads=2, strides=(4096, 256, 100, 32, 2, 1)), MISALIGNED)])
def test_cache_refusals(lib, bad, status):
    c = cache(**bad)
    write = lib.fp8_mqa_cache_write
    assert write(P, 3, BF16, P, 128, 128, c, None, 0, 0, None, None) == status
    assert write(P, 3, BF16, P, 128, 128, cache(heads=bad.get("heads", 1)), P, 128, 128, c, None) == status
    assert lib.fp8_mqa_cache_read(c, P, 4, 4, P, 2, 9, E4M3, P, P, None) == status
    assert lib.fp8_mqa_logits_paged(P, P, 2, 1, 32, 128, c, P, 4, 4, P, P, 64, 64, 1, None) == status
    assert lib.fp8_mqa_attention_paged(P, BF16, 2, 8, 1024, 128, c, cache(), P, 4, 4, P, None, 0, -1, 1.0, P, P, P, 1 << 40,
                                       None) == status


def test_write_refusals(lib):
    f = lib.fp8_mqa_cache_write
    one = (None, 0, 0, None, None)
    assert f(P, 0, BF16, P, 128, 128, cache(), *one) == OK          # no rows: nothing to do
    assert f(None, 0, BF16, None, 128, 128, cache(), *one) == OK
    assert f(P, -1, BF16, P, 128, 128, cache(), *one) == INVALID
    assert f(None, 3, BF16, P, 128, 128, cache(), *one) == INVALID
    assert f(P, 3, BF16, None, 128, 128, cache(), *one) == INVALID
    assert f(P, 3, E4M3, P, 128, 128, cache(), *one) == INVALID     # rows are 16 or 32 bits
    assert f(P, 3, 9, P, 128, 128, cache(), *one) == INVALID
    assert f(P, 3, BF16, P, 128, 128, None, *one) == INVALID
    assert f(P, 3, BF16, P, 128, 128, cache(type=BF16, scale=None), *one) == INVALID
    assert f(P + 2, 3, BF16, P, 128, 128, cache(), *one) == MISALIGNED
    assert f(P, 3, BF16, P + 1, 128, 128, cache(), *one) == MISALIGNED
    assert f(P, 3, F32, P + 2, 128, 128, cache(), *one) == MISALIGNED
    assert f(P, 1 << 31, BF16, P, 128, 128, cache(), *one) == UNSUPPORTED
    assert f(P, 3, BF16, P, 128, 128, cache(), P, 128, 128, None, None) == INVALID      # rows without a cache
    assert f(P, 3, BF16, P, 128, 128, cache(), P, 128, 128, cache(heads=2), None) == INVALID
    assert f(P, 3, BF16, P, 128, 128, cache(), P, 128, 128, cache(page=32), None) == INVALID
    assert f(P, 3, BF16, P, 128, 128, cache(), P, 128, 128, cache(dim=64), None) == INVALID


def test_read_refusals(lib):
    f = lib.fp8_mqa_cache_read
    assert f(cache(), P, 4, 4, P, 2, 0, E4M3, None, None, None) == OK
    assert f(cache(), P, 4, 4, P, -1, 9, E4M3, P, P, None) == INVALID
    assert f(cache(), P, 4, 4, P, 2, -9, E4M3, P, P, None) == INVALID
    assert f(cache(), None, 4, 4, P, 2, 9, E4M3, P, P, None) == INVALID
    assert f(cache(), P, 4, 4, None, 2, 9, E4M3, P, P, None) == INVALID
    assert f(cache(), P, 4, 4, P, 2, 9, E4M3, None, P, None) == INVALID
    assert f(cache(), P, 4, 4, P, 2, 9, E4M3, P, None, None) == INVALID   # stored values go with their scales
    assert f(cache(), P, 4, 4, P, 2, 9, BF16, P, P, None) == INVALID
    assert f(cache(), P, 4, 4, P, 2, 9, 4, P, None, None) == INVALID
    assert f(cache(type=BF16, scale=None), P, 4, 4, P, 2, 9, BF16, P, None, None) == INVALID
    assert f(cache(), P, 4, 4, P, 2, 9, BF16, P + 8, None, None) == MISALIGNED
    assert f(cache(), P, 4, 4, P + 2, 2, 9, BF16, P, None, None) == MISALIGNED
    assert f(cache(), P, 4, 4, P, 2, 1 << 31, BF16, P, None, None) == UNSUPPORTED


def test_logits_refusals(lib):
    def f(q=P, w=P, B=2, T=1, H=32, D=128, c=None, table=P, cols=4, lens=P, out=P, ld=64, N=64, clean=1):
        return lib.fp8_mqa_logits_paged(q, w, B, T, H, D, c or cache(), table, 4, cols, lens, out, ld, N, clean, None)
    assert f(B=0) == f(T=0) == f(N=0) == OK
    assert f(B=-1) == f(T=-1) == f(N=-1) == f(cols=-1) == INVALID
    assert f(ld=63) == f(clean=2) == INVALID
    assert f(q=None) == f(w=None) == f(lens=None) == f(out=None) == f(table=None) == INVALID
    assert f(H=64) == f(D=64) == UNSUPPORTED
    assert f(c=cache(heads=2)) == f(c=cache(dim=64)) == f(c=cache(type=BF16, scale=None)) == UNSUPPORTED
    assert f(N=1 << 30, ld=1 << 30) == UNSUPPORTED
    assert f(q=P + 8) == f(w=P + 4) == f(lens=P + 2) == f(out=P + 1) == f(table=P + 2) == MISALIGNED


def test_attention_refusals(lib):
    def f(q=P, type=BF16, B=2, heads=8, qs=(1024, 128), k=None, v=None, table=P, cols=4, lens=P, indices=None, n=-1, out=P,
          lse=P, space=P):
        return lib.fp8_mqa_attention_paged(q, type, B, heads, *qs, k or cache(), v or cache(), table, 4, cols, lens, indices, 0,
                                           n, 1.0, out, lse, space, 1 << 40, None)
    plain16 = dict(type=BF16, scale=None)
    assert f(B=0) == OK
    assert f(B=-1) == f(heads=0) == f(cols=-1) == f(n=-2) == INVALID
    assert f(type=F32) == f(type=E4M3) == INVALID
    assert f(q=None) == f(lens=None) == f(out=None) == f(space=None) == f(table=None) == INVALID
    assert f(n=5) == INVALID                                                 # indices announced, not given
    assert f(heads=9, k=cache(heads=2), v=cache(heads=2)) == INVALID         # no whole group per head
    assert f(v=cache(heads=2)) == f(v=cache(page=32)) == f(v=cache(dim=64)) == f(v=cache(**plain16)) == INVALID
    assert f(type=F16, k=cache(**plain16), v=cache(**plain16)) == INVALID    # a 16-bit cache is of q's type
    assert f(q=P + 8) == f(qs=(1028, 128)) == f(qs=(1024, 129)) == f(out=P + 8) == MISALIGNED
    assert f(lens=P + 2) == f(lse=P + 2) == f(table=P + 1) == f(space=P + 16) == f(n=4, indices=P + 2) == MISALIGNED


def test_binding_refuses_cpu_tensors(lib):
    f8 = torch.float8_e4m3fn
    data, scale = torch.zeros(2, 16, 1, 128).to(f8), torch.ones(2, 16, 1)
    i = torch.zeros(1, dtype=torch.int32)
    for call in (lambda: fm.cache_write(i, torch.zeros(1, 1, 128), data, scale),
                 lambda: fm.cache_read(data, scale, i.view(1, 1), torch.zeros(2, dtype=torch.int32), 4),
                 lambda: fm.logits_paged(torch.zeros(1, 1, 32, 128).to(f8), data, scale, torch.ones(1, 1, 32), i.view(1, 1), i),
                 lambda: fm.attention_paged(torch.zeros(1, 8, 128).bfloat16(), data, data, i.view(1, 1), i, k_scale=scale,
                                            v_scale=scale)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


# ------------------------------------------------------------------------------------ the plain forms

def test_e4m3_table_and_rounding_by_hand():
    v = plain.e4m3_values()
    assert v[0x01] == 2.0 ** -9 and v[0x08] == 2.0 ** -6 and v[0x38] == 1.0 and v[0x7E] == 448.0 and np.isnan(v[0x7F])
    assert np.array_equal(v[128:255], -v[:127])
    assert np.array_equal(v[:127], torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy())
    y = np.array([1.0625, 1.1875, 17.0, 19.0, 2.0 ** -10, 3 * 2.0 ** -10, 460.0, -1.06, 0.0])
    assert np.array_equal(plain.round_e4m3(y), [1.0, 1.25, 16.0, 20.0, 0.0, 2.0 ** -8, 448.0, -1.0, 0.0])
    x = np.random.default_rng(0).standard_normal(4000) * 100
    assert np.array_equal(plain.round_e4m3(x), torch.from_numpy(x).float().to(torch.float8_e4m3fn).double().numpy())


def test_quantise_by_hand():
    values, scale = plain.quantise32(np.array([[0.5, -448.0, 1.0, 0.0], [0.0, 0.0, 0.0, 0.0]]))
    assert np.array_equal(values, [[0.5, -448.0, 1.0, 0.0], [0, 0, 0, 0]])
    assert np.allclose(scale, [1.0, 1e-30 / 448], rtol=1e-6)


def test_plain_attention_by_hand():
    # two positions on one page, weights 1/4 and 3/4; a missing page; selected positions; nothing
    k = np.zeros((2, 2, 1, 1))
    k[0, :, 0, 0] = [0.0, np.log(3.0)]
    v = np.array([[[[4.0]], [[8.0]]], [[[100.0]], [[100.0]]]])
    q = np.ones((4, 1, 1))
    table = np.array([[0, -1], [0, 1], [0, 1], [7, 7]])
    lens = np.array([4, 2, 4, 4])
    idx = np.array([[0, 1, -1], [0, 1, 9], [1, 1, 4], [0, 1, 2]])
    out, lse, _, _ = plain.attention(q, k, v, table, lens, 1.0, idx)
    assert np.allclose(out[:, 0, 0], [7.0, 7.0, 8.0, 0.0]) and np.allclose(lse[:3, 0], np.log([4, 4, 6]))
    assert np.isneginf(lse[3, 0])
    dense, _, _, _ = plain.attention(q, k, v, table, lens, 1.0)
    assert np.allclose(dense[0], out[0]) and np.allclose(dense[2, 0, 0], (4 + 24 + 200) / 6)


def test_plain_logits_by_hand():
    q = np.zeros((1, 2, 2, 1))
    q[0, :, :, 0] = [[1.0, -1.0], [2.0, 1.0]]
    w = np.array([[[3.0, 5.0], [1.0, -1.0]]])
    k = np.array([[[1.0], [-2.0]], [[4.0], [9.0]]])
    scale = np.array([[1.0, 0.5], [2.0, 1.0]])
    out, _ = plain.logits(q, w, k, scale, np.array([[0, 1]]), [3], 4)
    assert np.array_equal(out[0], [3.0, 5.0, -np.inf, -np.inf])      # the older token sees positions 0 and 1
    assert np.array_equal(out[1], [2.0 - 1.0, 0.0, 2 * (8.0 - 4.0), -np.inf])
