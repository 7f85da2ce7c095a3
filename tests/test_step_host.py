"""The host code of page tables and of norms with rotation against a stand-in for the CUDA runtime (no GPU, no kernel
runs): which calls it refuses, and what it launches for the others."""
import ctypes
import os
import shutil
import struct
import subprocess

import numpy as np
import pytest

import fp8_mqa_logits_02_gb300 as fm
from fp8_mqa_logits_02_gb300 import nvcc_build
from test_paged_host import CALLS

HERE = os.path.dirname(os.path.abspath(__file__))
OK, INVALID, UNSUPPORTED, LAUNCH = 0, -1, -2, -5
E4M3, BF16, F32, E2M1 = 0, 1, 3, 4
LOOK = """
#include "overlap.h"
#include <cuda_runtime.h>
namespace {
int g_attributes, g_fail;
}
// In the place of the stand-in's own: counts, and fails where it is told to.
extern "C" cudaError_t __wrap_cudaFuncSetAttribute(const void*, cudaFuncAttribute, int)
{
    return ++g_attributes == g_fail ? cudaErrorInvalidValue : cudaSuccess;
}
extern "C" int attributes_set(int fail)
{
    const int n = g_attributes;
    g_attributes = 0;
    g_fail = fail;
    return n;
}
extern "C" int places_meet(const int64_t* a, const int64_t* b)
{
    const auto of = [](const int64_t* p) {
        return fp8mqa::Places{reinterpret_cast<const void*>(p[0]), p[1], p[2], p[3], p[4], p[5]};
    };
    return fp8mqa::meet(of(a), of(b));
}
"""


@pytest.fixture(scope="module")
def built(tmp_path_factory):
    nvcc = nvcc_build.nvcc_path()
    d = tmp_path_factory.mktemp("host")
    (d / "look.cpp").write_text(LOOK)
    common = [nvcc, "-std=c++17", "-Xcompiler", "-fPIC", "-I", os.path.join(nvcc_build.ROOT, "include"),
              "-I", nvcc_build.CSRC, "-c"]
    sources = [os.path.join(nvcc_build.CSRC, "step.cu"), os.path.join(nvcc_build.CSRC, "paged.cu"),
               os.path.join(HERE, "fake_runtime.cpp"), str(d / "look.cpp")]
    objects = [str(d / (os.path.basename(s) + ".o")) for s in sources]
    # the kernels are not assembled, nor optimised
    virtual = ["-gencode", "arch=compute_103a,code=compute_103a", "-Xcicc", "-O0"]
    more = {"step.cu": virtual, "paged.cu": virtual, "fake_runtime.cpp": ["-D__wrap_cudaFuncSetAttribute=not_this_one"]}
    running = [subprocess.Popen(common + more.get(os.path.basename(s), []) + ["-o", o, s], stdout=subprocess.PIPE,
                                stderr=subprocess.STDOUT, text=True) for s, o in zip(sources, objects)]
    for p in running:
        out, _ = p.communicate()
        assert p.returncode == 0, out
    wraps = [x for c in CALLS for x in ("-Xlinker", f"--wrap={c}")]
    subprocess.run([nvcc, "-shared", "-o", str(d / "host.so"), *objects, *wraps], check=True)
    return str(d / "host.so")


@pytest.fixture
def lib(built, tmp_path):
    """A library of its own, with the state of a fresh process."""
    path = str(tmp_path / "host.so")
    shutil.copy(built, path)
    handle = ctypes.CDLL(path)
    for name, (res, args) in fm.SIGNATURES.items():
        fn = getattr(handle, name, None)
        if fn is not None:
            fn.restype, fn.argtypes = res, args
    handle.fake_set(0, 0, 0)
    return handle


# ------------------------------------------------------------------------------------ memory that is shared

def test_pieces_meet_where_their_bytes_do(lib):
    rng = np.random.default_rng(1)
    hits = 0
    for _ in range(4000):
        steps = rng.integers(-40, 41, (2, 2))
        steps[1] = np.where(rng.random(2) < 0.5, steps[0], steps[1])     # half of them alike
        places, bytes_ = [], []
        for s in steps:
            n0, n1 = rng.integers(0, 6, 2)
            p = np.array([10000 + rng.integers(0, 120), n0, s[0], n1, s[1], rng.integers(0, 20)], np.int64)
            places.append(p)
            bytes_.append({int(p[0] + i * p[2] + j * p[4] + k) for i in range(n0) for j in range(n1) for k in range(p[5])})
        want = bool(bytes_[0] & bytes_[1])
        hits += want
        at = [p.ctypes.data_as(ctypes.POINTER(ctypes.c_int64)) for p in places]
        assert lib.places_meet(at[0], at[1]) == lib.places_meet(at[1], at[0]) == want, places
    assert 500 < hits < 3500


BASE, T, DIM = 1 << 20, 50, 128


def heads(x, n=4, row=9 * DIM, head=DIM, out=None, out_row=None, out_head=None, weight=0, scale=0, weight_type=F32):
    return struct.pack("@PPPPqqqqii", x, weight, x if out is None else out, scale, row, head, row if out_row is None else out_row,
                       head if out_head is None else out_head, n, weight_type)


def rotate(lib, q, k=None, to=BF16, pos=8 << 20, freq=9 << 20, T=T, rotated=64):
    launched = lib.fake_launches()
    rc = lib.fp8_mqa_norm_rotate(q, k, BF16, to, T, DIM, pos, 4, freq, rotated, 0, 1e-6, None)
    assert (lib.fake_launches() - launched == 1) == (rc == OK)
    return rc


def at(h, t=0):     # bfloat16 [T, 9, 128] from BASE on
    return BASE + 2 * DIM * (h + 9 * t)


def test_results_in_place_or_apart_are_taken(lib):
    far = 4 << 20
    assert rotate(lib, heads(at(0)), heads(at(5), n=2)) == OK                             # both in place
    assert rotate(lib, heads(at(0), out=far), heads(at(5), n=2, out=far + 8 * DIM)) == OK   # slices of another tensor
    assert rotate(lib, heads(at(0), out=at(5)), heads(at(4), n=1)) == OK                  # into heads that nobody reads
    # heads side by side: q, k and v of each in turn
    assert rotate(lib, heads(at(0), n=3, head=3 * DIM), heads(at(1), n=3, head=3 * DIM)) == OK
    assert rotate(lib, heads(at(0), n=3, head=3 * DIM, out=at(2)), heads(at(1), n=3, head=3 * DIM)) == OK
    # heads before tokens, in place
    assert rotate(lib, heads(BASE, row=DIM, head=T * DIM), heads(BASE + 8 * T * DIM, row=DIM, head=T * DIM)) == OK
    # strides of dimensions of one are never used
    assert rotate(lib, heads(at(0), n=1, head=DIM, out_head=7)) == OK
    assert rotate(lib, heads(at(0), row=5, out_row=77), heads(at(4)), T=1) == OK
    # no heads, no rotation: what is not read does not count
    assert rotate(lib, heads(at(0), n=0), heads(at(0))) == OK
    assert rotate(lib, heads(at(0)), pos=at(1), freq=at(2), rotated=0) == OK
    # to E4M3, beside one another
    assert rotate(lib, heads(at(0), out=far, out_row=512, out_head=128, scale=far + 1024 * T),
                  heads(at(4), out=far + (1 << 19), out_row=512, out_head=128, scale=far + 1024 * T + 16 * T), to=E4M3) == OK


@pytest.mark.parametrize("name,q,k,kw", [
    ("each into the other's place", heads(at(0), out=at(4)), heads(at(4), out=at(0)), {}),
    ("q into k", heads(at(0), out=at(4)), heads(at(4), out=4 << 20), {}),
    ("k into q", heads(at(0), out=4 << 20), heads(at(4), out=at(0)), {}),
    ("q over a shared tensor's k", heads(at(0)), heads(at(3), out=4 << 20), {}),
    ("one head on", heads(at(0), out=at(1)), None, {}),
    ("one token on", heads(at(0), out=at(0, 1)), None, {}),
    ("one value on", heads(at(0), out=at(0) + 16), None, {}),
    ("another stride", heads(at(0), n=3, out_head=2 * DIM), None, {}),
    ("both results in one place", heads(at(0), out=4 << 20), heads(at(4), out=4 << 20), {}),
    ("the last head", heads(at(0), out=4 << 20), heads(at(4), out=(4 << 20) + 6 * DIM), {}),
    ("rows on one another", heads(at(0), out=4 << 20, out_row=3 * DIM), None, {}),
    ("heads on one another", heads(at(0), out=4 << 20, out_head=0), None, {}),
    ("in turn, a head on", heads(at(0), n=3, head=3 * DIM, out=at(1)), heads(at(1), n=3, head=3 * DIM, out=4 << 20), {}),
    ("a weight", heads(at(0), weight=at(3)), None, {}),
    ("the other's weight", heads(at(0)), heads(at(5), out=4 << 20, weight=at(3)), {}),
    ("the last position", heads(at(0)), None, dict(pos=at(3, T - 1) + 2 * DIM - 4)),
    ("the frequencies", heads(at(0)), None, dict(freq=at(2, 7))),
    ("in place, to E4M3", heads(at(0), scale=4 << 20), None, dict(to=E4M3)),
    ("a scale", heads(at(0), out=4 << 20, out_row=512, scale=at(1)), None, dict(to=E4M3)),
    ("a scale and its values", heads(at(0), out=4 << 20, out_row=512, scale=(4 << 20) + 512 * T - 128), None, dict(to=E4M3)),
    ("one scale for both", heads(at(0), out=4 << 20, out_row=512, scale=5 << 20),
     heads(at(4), out=6 << 20, out_row=512, scale=5 << 20), dict(to=E4M3))])
def test_results_that_share_memory_are_refused(lib, name, q, k, kw):
    assert rotate(lib, q, k, **kw) == INVALID


ARRAYS = {"table": 4 * 20 * 9, "lens": 4 * 20, "change": 4 * 20, "free": 4 * 33, "n_free": 4, "slots": 4 * 50, "positions": 4 * 50,
          "rows": 4 * 50, "starts": 4 * 21, "changed": 4 * 20}      # bytes (20 requests, rows of 7 pages 9 apart)


def update(lib, B=20, cols=7, pitch=9, capacity=33, total=50, **at):
    where = {name: (i + 1) << 20 for i, name in enumerate(ARRAYS)} | at
    launched = lib.fake_launches()
    rc = lib.fp8_mqa_pages_update(where["table"], pitch, cols, 64, where["lens"], where["change"], B, where["free"], capacity,
                                  where["n_free"], total, where["slots"], where["positions"], where["rows"], where["starts"],
                                  where["changed"], None)
    assert (lib.fake_launches() > launched) == (rc == OK)
    return rc


def test_page_tables_arrays_beside_one_another_are_taken(lib):
    ends, at = {}, 1 << 16
    for name, size in ARRAYS.items():
        ends[name] = at
        at += size
    assert update(lib) == update(lib, **ends) == OK
    # between the rows of a table that lie further apart than they are long
    assert update(lib, n_free=(1 << 20) + 4 * 8, table=1 << 20) == OK
    # what is empty is nowhere
    assert update(lib, total=0, slots=1 << 20, positions=1 << 20, rows=1 << 20) == OK
    assert update(lib, B=0, table=9 << 20, lens=9 << 20, changed=9 << 20, change=9 << 20) == OK
    assert update(lib, capacity=0, free=1 << 20) == OK


@pytest.mark.parametrize("i", range(1, 10))
def test_page_tables_arrays_that_overlap_are_refused(lib, i):
    names = list(ARRAYS)
    for j in range(i):
        a, b = names[i], names[j]
        assert update(lib, **{a: 32 << 20, b: 32 << 20}) == INVALID
        # the last entry of one (of a table: past its last row there is nothing) is the first of the other
        last = ARRAYS[b] - (12 if b == "table" else 4)
        assert update(lib, **{b: 32 << 20, a: (32 << 20) + last}) == INVALID
        assert update(lib, **{b: 32 << 20, a: (32 << 20) + last + 4}) == OK


def test_shared_memory_for_many_requests_is_set_up_once(lib):
    def many():
        return update(lib, B=8192, total=0, table=1 << 30, lens=1 << 25, change=2 << 25, starts=3 << 25, changed=4 << 25)
    assert update(lib) == OK and lib.attributes_set(1) > 0      # (that of the paged operators' kernels)
    assert many() == LAUNCH and lib.attributes_set(0) == 1      # it fails, and is tried again
    assert many() == OK and lib.attributes_set(0) == 1
    assert many() == many() == update(lib) == OK and lib.attributes_set(0) == 0


# ------------------------------------------------------------------------------------ many heads

def cache(heads, dim, type, row):
    """One token of many heads."""
    return struct.pack("@PPqiiiiqqqqqqPqqq", BASE, BASE, 1, 1, heads, dim, type, heads * row, heads * row, row, heads, heads, 1,
                       BASE if type == E2M1 else 0, heads * dim // 16, heads * dim // 16, dim // 16)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("type,to,size", [(E4M3, E4M3, 1), (E4M3, BF16, 2), (E4M3, F32, 4), (E2M1, BF16, 2), (E2M1, F32, 4)])
def test_reads_of_more_heads_than_a_block_counts_are_refused(lib, type, to, size, dim):
    # a block counts the 16-byte pieces of a row of its output in 32 bits
    most = 2 ** 34 // (dim * size)

    def read(heads):
        launched = lib.fake_launches()
        c = cache(heads, dim, type, dim if type == E4M3 else dim // 2)
        rc = lib.fp8_mqa_cache_read(c, BASE, 1, 1, BASE, 1, 1, to, BASE, BASE if to == E4M3 else None, None)
        assert (lib.fake_launches() > launched) == (rc == OK)
        return rc
    assert read(most) == OK
    assert read(most + 1) == read(2 * most) == read(2 ** 31 - 1) == UNSUPPORTED


@pytest.mark.parametrize("heads_", [2 ** 31 - 1, 2 ** 31 - 9, 2 ** 30 + 1, 2 ** 20 + 7])
@pytest.mark.parametrize("other", [0, 1])
def test_norms_of_very_many_heads(lib, heads_, other):
    # one token: groups of 16 lanes that take up to 10 heads each, eight groups a block
    many = heads(BASE, n=heads_ - other, row=0)
    one = heads(1 << 50, n=other, row=0)
    grid = (ctypes.c_uint * 3)()
    for q, k in ((many, one), (one, many)):
        lib.fake_set(0, 0, 0)
        assert rotate(lib, q, k, T=1, pos=1 << 51, freq=1 << 52) == OK
        lib.fake_grid(0, grid)
        assert grid[0] == -(-(-(-(heads_ - other) // 10) + other) // 8)
