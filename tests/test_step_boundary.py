"""The entry points of 4-bit caches, page tables and norms with rotation without a GPU: bad arguments are refused on
the host before any device work, and the plain forms that the GPU tests compare with are pinned by hand."""
import ctypes
import struct

import numpy as np
import pytest
import torch

import fp8_mqa_logits_02_gb300 as fm
from oracle import step as plain

OK, INVALID, UNSUPPORTED, MISALIGNED = 0, -1, -2, -3
E4M3, BF16, F16, F32, E2M1 = 0, 1, 2, 3, 4
P = 0x1000  # an aligned address that is never read


@pytest.fixture(scope="module")
def lib():
    fm.build()
    return fm.lib()


def cache(data=P, scale=P, groups=P, pages=4, page=16, heads=1, dim=128, type=E2M1, strides=None, by=None):
    s = strides or (page * heads * dim // 2, heads * dim // 2, dim // 2, page * heads, heads, 1)
    g = by or (page * heads * dim // 16, heads * dim // 16, dim // 16)
    return struct.pack("@PPqiiiiqqqqqqPqqq", data or 0, scale or 0, pages, page, heads, dim, type, *s, groups or 0, *g)


def e4m3(**kw):
    return cache(type=E4M3, strides=(2048, 128, 128, 16, 1, 1), groups=None, **kw)


def calls(lib, c):
    return (lib.fp8_mqa_cache_write(P, 3, BF16, P, 128, 128, c, None, 0, 0, None, None),
            lib.fp8_mqa_cache_read(c, P, 4, 4, P, 2, 9, BF16, P, None, None),
            lib.fp8_mqa_attention_paged(P, BF16, 2, 8, 1024, 128, c, cache(), P, 4, 4, P, None, 0, -1, 1.0, P, P, P, 1 << 40, None),
            lib.fp8_mqa_attention_paged(P, BF16, 2, 8, 1024, 128, cache(), c, P, 4, 4, P, None, 0, -1, 1.0, P, P, P, 1 << 40, None))


@pytest.mark.parametrize("bad,status", [
    (dict(data=None), INVALID), (dict(scale=None), INVALID), (dict(groups=None), INVALID), (dict(pages=-1), INVALID),
    (dict(page=0), INVALID), (dict(type=5), INVALID), (dict(type=-1), INVALID), (dict(dim=96), UNSUPPORTED),
    (dict(pages=1 << 28), UNSUPPORTED), (dict(data=P + 8), MISALIGNED), (dict(scale=P + 2), MISALIGNED),
    (dict(groups=P + 4), MISALIGNED), (dict(dim=64, groups=P + 2), MISALIGNED),
    (dict(strides=(1024 + 8, 64, 64, 16, 1, 1)), MISALIGNED), (dict(strides=(1024, 72, 64, 16, 1, 1)), MISALIGNED),
    (dict(by=(128 + 4, 8, 8)), MISALIGNED), (dict(by=(128, 12, 8)), MISALIGNED)])
def test_cache_refusals(lib, bad, status):
    assert calls(lib, cache(**bad)) == (status,) * 4


def test_caches_in_4_bits_go_with_their_own(lib):
    write, read, attend = lib.fp8_mqa_cache_write, lib.fp8_mqa_cache_read, lib.fp8_mqa_attention_paged
    assert write(P, 0, BF16, P, 128, 128, cache(), None, 0, 0, None, None) == OK
    assert write(P, 3, BF16, P, 128, 128, cache(), P, 128, 128, e4m3(), None) == INVALID
    assert write(P, 3, BF16, P, 128, 128, e4m3(), P, 128, 128, cache(), None) == INVALID
    assert write(P, 3, BF16, P, 128, 128, cache(), P, 128, 128, cache(dim=64), None) == INVALID
    assert write(P, 3, E2M1, P, 128, 128, cache(), None, 0, 0, None, None) == INVALID
    assert read(cache(), P, 4, 4, P, 2, 0, BF16, P, None, None) == OK
    for to in (E4M3, E2M1, -1):      # rows come back in 16 or 32 bits
        assert read(cache(), P, 4, 4, P, 2, 9, to, P, P if to == E4M3 else None, None) == INVALID
    assert read(e4m3(), P, 4, 4, P, 2, 9, E2M1, P, None, None) == INVALID
    assert lib.fp8_mqa_logits_paged(P, P, 2, 1, 32, 128, cache(), P, 4, 4, P, P, 64, 64, 1, None) == UNSUPPORTED
    for k, v in ((cache(), e4m3()), (e4m3(), cache()), (cache(), cache(dim=64)), (cache(heads=2), cache())):
        assert attend(P, BF16, 2, 8, 1024, 128, k, v, P, 4, 4, P, None, 0, -1, 1.0, P, P, P, 1 << 40, None) == INVALID
    # a struct without the members of 4-bit caches is as good as ever for other types
    short = e4m3()[:struct.calcsize("@PPqiiiiqqqqqq")]
    assert write(P, 0, BF16, P, 128, 128, ctypes.create_string_buffer(short, len(short)), None, 0, 0, None, None) == OK


def test_no_rows_of_a_pair(lib):
    # empty tensors have no memory: there is nothing to do, in either type of cache
    for c in (cache(), e4m3()):
        assert lib.fp8_mqa_cache_write(None, 0, BF16, None, 128, 128, c, None, 128, 128, c, None) == OK
        assert lib.fp8_mqa_cache_write(P, 3, BF16, P, 128, 128, c, None, 128, 128, c, None) == INVALID
        assert lib.fp8_mqa_cache_write(None, 0, BF16, None, 128, 128, c, P, 128, 128, None, None) == INVALID


def test_pages_refusals(lib):
    def f(table=P, stride=4, cols=4, page=64, lens=P, change=P, B=2, free=P, cap=9, n=P, total=5, slots=P, pos=P, rows=P,
          starts=P, changed=P):
        return lib.fp8_mqa_pages_update(table, stride, cols, page, lens, change, B, free, cap, n, total, slots, pos, rows,
                                        starts, changed, None)
    assert f(B=-1) == f(cols=-1) == f(page=0) == f(cap=-1) == f(total=-1) == INVALID
    assert f(table=None) == f(lens=None) == f(change=None) == f(free=None) == f(n=None) == INVALID
    assert f(slots=None) == f(pos=None) == f(rows=None) == f(starts=None) == f(changed=None) == INVALID
    assert f(stride=3) == f(stride=0) == INVALID                          # rows are written
    assert f(B=8193) == f(cols=1 << 20, stride=1 << 20, page=1 << 11) == f(cap=1 << 31) == f(total=1 << 31) == UNSUPPORTED
    for name in ("table", "lens", "change", "free", "n", "slots", "pos", "rows", "starts", "changed"):
        assert f(**{name: P + 2}) == MISALIGNED


def heads(x=P, weight=P, out=P, scale=None, row=1024, head=128, out_row=1024, out_head=128, n=8, type=BF16):
    return struct.pack("@PPPPqqqqii", x or 0, weight or 0, out or 0, scale or 0, row, head, out_row, out_head, n, type)


def test_norm_rotate_refusals(lib):
    def f(q=None, k=None, x=BF16, to=BF16, T=3, dim=128, pos=P, wide=4, freq=P, rotated=64, inter=0, **kw):
        return lib.fp8_mqa_norm_rotate(q or heads(**kw), k, x, to, T, dim, pos, wide, freq, rotated, inter, 1e-6, None)
    assert f(T=0, q=heads(x=None, out=None), pos=None) == OK               # empty tensors have no memory
    assert f(T=0) == f(n=0) == f(n=0, x=F16, to=F16) == OK
    assert lib.fp8_mqa_norm_rotate(None, None, BF16, BF16, 3, 128, P, 4, P, 64, 0, 1e-6, None) == INVALID
    assert f(T=-1) == f(rotated=-16) == f(inter=2) == f(wide=2) == f(n=-1) == INVALID
    assert f(x=E4M3) == f(x=7) == f(to=F16) == f(to=E2M1) == INVALID
    assert f(**{"q": heads(x=None)}) == f(**{"q": heads(out=None)}) == f(scale=P) == f(to=E4M3) == INVALID
    assert f(type=F16) == f(type=E4M3) == INVALID                         # a weight of another type
    assert f(k=heads(type=F16)) == f(k=heads(n=-1)) == f(k=heads(out=None)) == INVALID
    assert f(pos=None) == f(freq=None) == INVALID
    assert f(dim=96) == f(rotated=24) == f(rotated=144) == f(dim=64, rotated=80) == f(T=1 << 28) == f(T=1 << 31) == UNSUPPORTED
    assert f(q=heads(x=P + 1)) == f(q=heads(out=P + 1)) == f(q=heads(weight=P + 1)) == f(q=heads(weight=P + 2, type=F32)) == MISALIGNED
    assert f(pos=P + 2) == f(pos=P + 4, wide=8) == f(freq=P + 2) == MISALIGNED
    assert f(to=E4M3, scale=P, q=heads(scale=P, out=P + 2)) == f(to=E4M3, q=heads(scale=P, out_head=130)) == MISALIGNED
    assert f(to=E4M3, q=heads(scale=P + 2)) == MISALIGNED


def test_binding_refuses_cpu_tensors(lib):
    i = torch.zeros(1, dtype=torch.int32)
    for call in (lambda: fm.pages_update(i.view(1, 1), i, i, i, i, 64, 1),
                 lambda: fm.norm_rotate(torch.zeros(1, 1, 128), None, i, torch.zeros(64))):
        with pytest.raises(ValueError, match="CUDA"):
            call()


# ------------------------------------------------------------------------------------ the plain forms

def test_e2m1_by_hand():
    assert np.array_equal(plain.unpack(np.array([0x10, 0x32, 0x54, 0x76, 0x98, 0xFE], np.uint8)),
                          [0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -4, -6])
    y = np.array([0.25, 0.26, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.1, 7.0, -0.75, -2.6, 0.1])
    assert np.array_equal(plain.round_e2m1(y), [0, 0.5, 1, 1, 2, 2, 4, 4, 6, 6, -1, -3, 0])


def test_quantise4_by_hand():
    x = np.zeros((2, 64))
    x[0, :4] = [6, -3, 0.26, 0.2]     # a group of its own scale 448 / 448
    x[0, 16:18] = [3, -1.25]          # half of it
    x[0, 32] = 6 / 1000               # 0.448 of a step of 0.0417: 224 / 512 = 7 * 2^-4
    values, groups, scale = plain.quantise4(x)
    assert np.array_equal(groups[0], [448, 224, 0.4375, 0]) and np.allclose(scale, [6 / 2688, 1e-30 / 2688], rtol=1e-6)
    assert np.array_equal(values[0, :4], [6, -3, 0.5, 0]) and np.array_equal(values[0, 16:18], [6, -2])
    assert values[0, 32] == 6 and (values[0, 48:] == 0).all() and (values[1] == 0).all()


def test_pages_by_hand():
    table = np.array([[5, -1, -1], [2, 7, -1], [-1, -1, -1]], np.int32)
    lens, free = np.array([3, 6, 0], np.int32), np.array([9, 8, 1, -1, -1, -1], np.int32)
    n, slots, positions, rows, starts, changed = plain.pages(table, lens, np.array([2, -4, 1]), free, 3, 4, 5)
    # request 1 gives back page 7, which request 0 then takes; request 2 takes page 1
    assert n == 2 and table.tolist() == [[5, 7, -1], [2, 7, -1], [1, -1, -1]] and lens.tolist() == [5, 2, 1]
    assert slots.tolist() == [5 * 4 + 3, 7 * 4, 1 * 4, -1, -1] and positions.tolist() == [3, 4, 0, 0, 0]
    assert rows.tolist() == [0, 0, 2, 0, 0] and starts.tolist() == [0, 2, 2, 3] and changed.tolist() == [2, -4, 1]
    assert free[:2].tolist() == [9, 8]


def test_norm_rotate_by_hand():
    x = np.array([[[3.0, 4.0, 0.0, 0.0]]])
    out, _ = plain.norm_rotate(x, np.full(4, 2.0), np.array([1]), np.array([float(plain.PI) / 2, 0.0]), 0.0, False)
    assert np.allclose(out, [[[0.0, 3.2, 2.4, 0.0]]])       # rms 2.5; (0, 2) a quarter turn, (1, 3) none
    out, _ = plain.norm_rotate(x, None, np.array([3]), np.array([float(plain.PI) / 2]), 0.0, True)
    assert np.allclose(out, [[[4.0, -3.0, 0.0, 0.0]]])
