"""The paged operators in the bounds-checking build (libfp8mqa_debug.so).

There every access to global memory, and every TMA box, is held against what the call's arguments span
before it is made; one outside is recorded (check_error then returns FP8MQA_ERR_BOUNDS) and skipped.  Small
parity cases record nothing.  That each kind of memory is checked at all is shown by taking it to be shorter
than it is: the accesses past that end are valid, and have to be recorded and not made.
"""
import ctypes

import numpy as np
import pytest
import torch

import fp8_mqa_logits_02_gb300 as fm
import test_paged as tp
from test_paged import F8, cache, gpu, tables

pytestmark = pytest.mark.gpu

BOUNDS = -8
KINDS = {"slots": 1, "rows": 2, "rows2": 3, "data": 4, "data2": 5, "scale": 6, "scale2": 7, "table": 8, "lens": 9,
         "indices": 10, "q": 11, "w": 12, "out": 13, "out_scale": 14, "splits": 15, "partial": 16}


@pytest.fixture(scope="module", autouse=True)
def _debug_lib():
    fm.build()
    fm.use_debug_library(True)
    lib = fm.lib()
    lib.fp8_mqa_debug_bounds_short.argtypes = [ctypes.c_int32, ctypes.c_uint64]
    lib.fp8_mqa_debug_bounds_short.restype = None
    yield
    fm.use_debug_library(False)


@pytest.fixture(autouse=True)
def _clean():
    assert fm.check_error() == 0
    yield
    assert fm.check_error() == 0


def test_the_library_itself_has_no_such_switch():
    assert not hasattr(fm.lib(debug=False), "fp8_mqa_debug_bounds_short")


# ------------------------------------------------------------------------------------ nothing is recorded

@pytest.mark.parametrize("T,heads,dim,page", [(1, 1, 128, 64), (7, 8, 64, 1), (130, 2, 64, 100)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_writes(T, heads, dim, page, dtype):
    tp.test_write_pair_is_exact(T, heads, dim, page, dtype)
    tp.test_write_unaligned_rows(dtype)


@pytest.mark.parametrize("layout", ["joint", "heads"])
def test_writes_into_strided_caches(layout):
    tp.test_write_one_into_strided_cache(layout)


@pytest.mark.parametrize("dtype", [F8, torch.bfloat16, torch.float32])
def test_reads(dtype):
    tp.test_read_is_exact([0, 3, 0, 0, 70, 1, 0], 2, 64, 16, "plain", dtype)
    tp.test_read_is_exact([129, 64, 1], 8, 128, 33, "heads", dtype)
    tp.test_read_is_exact([40, 41], 4, 64, 1, "joint", dtype)


@pytest.mark.parametrize("page", [16, 33, 64, 96, 128])
@pytest.mark.parametrize("T", [1, 2, 3, 5])
def test_logits(T, page):
    rng = np.random.default_rng(T + page)
    tp.check_logits(rng, [0, 2, 127, 128, 129, 1000], T, page)
    tp.check_logits(rng, [200, 300], T, page, clean=False, holes=True, layout="heads")
    tp.check_logits(rng, [200, 100], T, page, N=201, ld=207, layout="joint")
    tp.check_logits(rng, rng.integers(0, 90, 700), T, page)


def test_logits_of_long_rows():
    tp.check_logits(np.random.default_rng(3), [60001, 50000], 2, 64)


@pytest.mark.parametrize("dtype,kind", tp.TYPES)
@pytest.mark.parametrize("dim", [64, 128])
def test_attention(dtype, kind, dim):
    rng = np.random.default_rng(dim)
    tp.check_attention(rng, [0, 2, 31, 32, 33, 500], 8, 2, dim, 16, dtype, kind)
    tp.check_attention(rng, [300, 129, 10], 8, 4, dim, 32, dtype, kind, layout="joint", holes=True, fused=True)
    tp.check_attention(rng, [300, 129, 10], 8, 4, dim, 32, dtype, kind, layout="heads", holes=True, select=64)
    tp.check_attention(rng, [900] * 5, 8, 2, dim, 48, dtype, kind, select=513, shared=True)


@pytest.mark.parametrize("kind", [F8, None])
def test_attention_split_and_in_every_layout(kind):
    rng = np.random.default_rng(9)
    tp.check_attention(rng, [30011], 8, 1, 128, 64, kind=kind)
    tp.check_attention(rng, [9001, 3, 0, 5000], 16, 4, 128, 100, kind=kind)
    tp.test_attention_head_layouts(40, 5, kind)
    tp.test_attention_key_heads_side_by_side(12, 4, 128, torch.bfloat16, kind)
    tp.test_attention_groups_that_share_a_ring(32, 1, 64, torch.bfloat16, kind)
    tp.test_attention_groups_that_share_a_ring(256, 2, 128, torch.bfloat16, kind)


def test_no_pages_and_nothing_selected():
    tp.test_no_pages_at_all()
    tp.test_attention_selected_nothing_and_twice()


# ------------------------------------------------------------------------------------ what is short is recorded

def calls(page):
    """Each operator on inputs that reach the last byte of most of their memory."""
    rng = np.random.default_rng(1)
    B, cols = 3, 4
    pages = B * cols
    kd, ks = cache(rng, pages, page, 2, 128)
    vd, vs = cache(rng, pages, page, 2, 128)
    xd, xs = cache(rng, pages, page, 1, 128)
    table = torch.arange(pages, dtype=torch.int32, device="cuda").view(B, cols)
    n = cols * page
    lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
    x = torch.randn(pages * page, 2, 128, device="cuda").to(torch.bfloat16)
    slots = torch.arange(pages * page, dtype=torch.int32, device="cuda")
    starts = torch.arange(B + 1, dtype=torch.int32, device="cuda") * n
    q = torch.randn(B, 8, 128, device="cuda").to(torch.bfloat16)
    q8 = torch.randn(B, 1, 32, 128, device="cuda").to(F8)
    w = torch.randn(B, 1, 32, device="cuda")
    indices = torch.arange(n, dtype=torch.int32, device="cuda").expand(B, n).contiguous()
    attend = dict(k_scale=ks, v_scale=vs, return_lse=True)
    return {"write": lambda: fm.cache_write(slots, x, kd, ks, x.clone(), vd, vs),
            "read": lambda: fm.cache_read(kd, ks, table, starts, B * n),
            "read16": lambda: fm.cache_read(kd, ks, table, starts, B * n, dtype=torch.float16),
            "logits": lambda: fm.logits_paged(q8, xd, xs, w, table, lens),
            "fill": lambda: fm.logits_paged(q8, xd, xs, w, table, lens - 2 * page, max_len=n + 77),
            "attend": lambda: fm.attention_paged(q, kd, vd, table, lens, **attend),
            "selected": lambda: fm.attention_paged(q, kd, vd, table, lens, indices=indices, **attend)}


REACHED = {"write": ["slots", "rows", "rows2", "data", "data2", "scale", "scale2"],
           "read": ["table", "lens", "data", "scale", "out", "out_scale"],
           "read16": ["table", "lens", "data", "scale", "out"],
           "logits": ["table", "lens", "data", "scale", "q", "w", "out"],
           "fill": ["out"],
           "attend": ["table", "lens", "data", "data2", "scale", "scale2", "q", "out", "out_scale"],
           "selected": ["indices", "table", "lens", "data", "data2", "scale", "scale2", "q", "out", "out_scale"]}


def recorded(call, kind, short):
    lib = fm.lib()
    lib.fp8_mqa_debug_bounds_short(KINDS[kind], short)
    try:
        call()
        return fm.check_error()
    finally:
        lib.fp8_mqa_debug_bounds_short(KINDS[kind], 0)


@pytest.mark.parametrize("page", [64, 16])
@pytest.mark.parametrize("name", REACHED)
def test_memory_that_is_a_byte_short(name, page):
    call = calls(page)[name]
    call()
    assert fm.check_error() == 0
    for kind in REACHED[name]:
        assert recorded(call, kind, 1) == BOUNDS, kind
        assert fm.check_error() == 0            # cleared by the read
        call()
        assert fm.check_error() == 0


@pytest.mark.parametrize("page", [64, 16])
def test_memory_that_is_not_there(page):
    every = calls(page)
    for name, kinds in REACHED.items():
        # (the rows of pages of 16 are one tile each: none is split)
        for kind in kinds + (["splits"] + ["partial"] * (page == 64) if name in ("attend", "selected") else []):
            assert recorded(every[name], kind, 2 ** 62) == BOUNDS, (name, kind)
