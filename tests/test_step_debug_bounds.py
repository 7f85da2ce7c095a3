"""Page tables, norms with rotation and 4-bit caches in the bounds-checking build: small parity cases record nothing,
and memory that is taken to be a byte shorter than it is, or not there, is recorded and not accessed (see
test_paged_debug_bounds.py)."""
import ctypes

import numpy as np
import pytest
import torch

import fp8_mqa_logits_02_gb300 as fm
import test_norm_rotate as tn
import test_paged4 as t4
import test_pages as tp
from test_paged4 import F4, cache

pytestmark = pytest.mark.gpu

BOUNDS = -8
KINDS = {"slots": 1, "rows": 2, "rows2": 3, "data": 4, "data2": 5, "scale": 6, "scale2": 7, "table": 8, "lens": 9,
         "change": 10, "q": 11, "out": 13, "out_scale": 14, "splits": 15, "partial": 16, "groups": 17, "groups2": 18,
         "positions": 19, "freq": 20, "weight": 21, "weight2": 22, "out2": 23, "out_scale2": 24, "free": 25, "n_free": 26,
         "starts": 27}


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


# ------------------------------------------------------------------------------------ nothing is recorded

@pytest.mark.parametrize("B,page,cols", [(1, 64, 8), (33, 48, 9), (1025, 100, 3)])
def test_pages(B, page, cols):
    tp.test_steps(B, page, cols)


def test_odd_pages():
    tp.test_the_stack_runs_out_in_order()
    tp.test_rows_that_are_full_and_odd_arguments()
    tp.test_empty_calls()
    tp.test_many_tokens_in_a_few_requests()


@pytest.mark.parametrize("dtype", tn.TYPES)
def test_norms(dtype):
    for interleaved in (False, True):
        tn.test_sizes(7, 8, 1, 64, 48, interleaved, dtype)
        tn.test_sizes(33, 0, 2, 64, 32, interleaved, dtype)
        tn.test_sizes(257, 12, 4, 128, 112, interleaved, dtype)
    tn.test_many_heads_a_group(dtype)
    tn.test_unaligned_rows(dtype)


def test_norms_in_place():
    tn.test_in_place_and_into_strided_results()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_writes_and_reads(dtype):
    t4.test_write_pair_is_exact(7, 8, 64, 1, dtype)
    t4.test_write_pair_is_exact(130, 2, 64, 100, dtype)
    t4.test_write_unaligned_rows(dtype)
    t4.test_write_one_into_strided_cache("heads")
    t4.test_read_is_exact([0, 3, 0, 0, 70, 1, 0], 2, 64, 16, "plain", dtype)
    t4.test_read_is_exact([129, 64, 1], 8, 128, 33, "heads", dtype)


@pytest.mark.parametrize("dim", [64, 128])
def test_attention(dim):
    rng = np.random.default_rng(dim)
    t4.check_attention(rng, [0, 2, 31, 32, 33, 500], 8, 2, dim, 16)
    t4.check_attention(rng, [64, 65, 127, 300], 8, 2, dim, 32)
    t4.test_attention_layouts_holes_and_selected(dim, torch.bfloat16)
    t4.test_attention_head_layouts(40, 5, dim)
    t4.test_attention_groups_that_share_a_ring(64, 1, dim)
    t4.check_attention(rng, [9001, 3, 0, 5000], 16, 4, dim, 64)


# ------------------------------------------------------------------------------------ what is short is recorded

def calls(page):
    rng = np.random.default_rng(1)
    B, cols = 3, 4
    pages, n = B * cols, cols * page
    (kc, kg, ks), (vc, vg, vs) = cache(rng, pages, page, 2, 128), cache(rng, pages, page, 2, 128)
    table = torch.arange(pages, dtype=torch.int32, device="cuda").view(B, cols)
    lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
    x = torch.randn(pages * page, 2, 128, device="cuda").to(torch.bfloat16)
    slots = torch.arange(pages * page, dtype=torch.int32, device="cuda")
    starts = torch.arange(B + 1, dtype=torch.int32, device="cuda") * n
    q = torch.randn(B, 8, 128, device="cuda").to(torch.bfloat16)
    indices = torch.arange(n, dtype=torch.int32, device="cuda").expand(B, n).contiguous()
    attend = dict(k_scale=ks, v_scale=vs, k_groups=kg, v_groups=vg, return_lse=True)
    pos, f = torch.arange(pages * page, dtype=torch.int64, device="cuda"), tn.freq(128)
    w = torch.ones(128, dtype=torch.bfloat16, device="cuda")
    y = torch.randn(pages * page, 5, 128, device="cuda").to(torch.bfloat16)

    def update(way):
        # every page is free and taken, to the last column and the last token; or all of them come back
        held = torch.full((B,), 0 if way > 0 else n, dtype=torch.int32, device="cuda")
        count = torch.full((1,), pages if way > 0 else 0, dtype=torch.int32, device="cuda")
        fm.pages_update(table.clone(), held, torch.full_like(held, way * n), torch.arange(pages, dtype=torch.int32, device="cuda"),
                        count, page, B * n if way > 0 else 0)

    return {"write": lambda: fm.cache_write(slots, x, kc.view(F4), ks, x.clone(), vc.view(F4), vs, k_groups=kg, v_groups=vg),
            "read": lambda: fm.cache_read(kc.view(F4), ks, table, starts, B * n, dtype=torch.float16, groups=kg),
            "attend": lambda: fm.attention_paged(q, kc.view(F4), vc.view(F4), table, lens, **attend),
            "selected": lambda: fm.attention_paged(q, kc.view(F4), vc.view(F4), table, lens, indices=indices, **attend),
            "grow": lambda: update(1), "shrink": lambda: update(-1),
            "rotate": lambda: fm.norm_rotate(x, y, pos, f, w, w),
            "rotate8": lambda: fm.norm_rotate(x, y, pos, f, w, w, dtype=torch.float8_e4m3fn)}


ROTATE = ["rows", "rows2", "positions", "freq", "weight", "weight2", "out", "out2"]
REACHED = {"write": ["slots", "rows", "rows2", "data", "data2", "scale", "scale2", "groups", "groups2"],
           "read": ["table", "lens", "data", "scale", "groups", "out"],
           "attend": ["table", "lens", "data", "data2", "scale", "scale2", "groups", "groups2", "q", "out", "out_scale"],
           "selected": ["change", "table", "lens", "data", "data2", "scale", "scale2", "groups", "groups2", "q", "out",
                        "out_scale"],
           "grow": ["table", "lens", "change", "free", "n_free", "slots", "positions", "rows", "starts", "out"],
           "shrink": ["table", "lens", "change", "free", "n_free", "starts", "out"],
           "rotate": ROTATE, "rotate8": ROTATE + ["out_scale", "out_scale2"]}


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
def test_memory_that_is_a_byte_short_or_not_there(name, page):
    call = calls(page)[name]
    call()
    assert fm.check_error() == 0
    for kind in REACHED[name]:
        assert recorded(call, kind, 1) == BOUNDS, kind
        assert recorded(call, kind, 2 ** 62) == BOUNDS, kind
        assert fm.check_error() == 0            # cleared by the read
        call()
        assert fm.check_error() == 0
