"""The paged operators' host code against a stand-in for the CUDA runtime: what a call returns, and what
it launches afterwards, when one of its calls fails.  No GPU and no kernel is involved."""
import ctypes
import os
import shutil
import struct
import subprocess

import pytest

import fp8_mqa_logits_02_gb300 as fm
from fp8_mqa_logits_02_gb300 import nvcc_build

HERE = os.path.dirname(os.path.abspath(__file__))
OK, UNSUPPORTED, LAUNCH, CUDA = 0, -2, -5, -7
E4M3, BF16 = 0, 1
P = 0x1000  # an aligned address that is never read
CALLS = ("cudaGetDevice", "cudaDeviceGetAttribute", "cudaFuncSetAttribute", "cudaMalloc", "cudaFree", "cudaMemset",
         "cudaMemcpy", "cudaGetLastError", "cudaLaunchKernelExC")


@pytest.fixture(scope="module")
def built(tmp_path_factory):
    nvcc = nvcc_build.nvcc_path()
    d = tmp_path_factory.mktemp("host")
    common = [nvcc, "-std=c++17", "-Xcompiler", "-fPIC", "-I", os.path.join(nvcc_build.ROOT, "include"),
              "-I", nvcc_build.CSRC, "-c"]
    jobs = [
        # the kernels are not assembled: nothing here runs them
        common + ["-gencode", "arch=compute_103a,code=compute_103a", "-o", str(d / "paged.o"),
                  os.path.join(nvcc_build.CSRC, "paged.cu")],
        common + ["-o", str(d / "fake.o"), os.path.join(HERE, "fake_runtime.cpp")]]
    running = [subprocess.Popen(j, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True) for j in jobs]
    for p in running:
        out, _ = p.communicate()
        assert p.returncode == 0, out
    wraps = [x for c in CALLS for x in ("-Xlinker", f"--wrap={c}")]
    subprocess.run([nvcc, "-shared", "-o", str(d / "host.so"), str(d / "paged.o"), str(d / "fake.o"), *wraps], check=True)
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


def cache(pages=4000, page=64, heads=1, dim=128, type=E4M3):
    s = (page * heads * dim, heads * dim, dim, page * heads, heads, 1)
    return struct.pack("@PPqiiiiqqqqqq", P, P if type == E4M3 else 0, pages, page, heads, dim, type, *s)


def attention(lib, B=1, heads=8, cols=2000, c=None):
    c = c or cache()
    return lib.fp8_mqa_attention_paged(P, BF16, B, heads, heads * 128, 128, c, c, P, cols, cols, P, None, 0, -1, 1.0, P, P, P,
                                       1 << 40, None)


def calls(lib):
    """Each operator, called once."""
    c = cache()
    return {"write": lambda: lib.fp8_mqa_cache_write(P, 9, BF16, P, 128, 128, c, None, 0, 0, None, None),
            "read": lambda: lib.fp8_mqa_cache_read(c, P, 9, 9, P, 2, 90, BF16, P, None, None),
            "logits": lambda: lib.fp8_mqa_logits_paged(P, P, 2, 1, 32, 128, c, P, 9, 9, P, P, 576, 576, 1, None),
            "attention": lambda: attention(lib)}


def test_attention_launches_the_join_after_its_first_kernel(lib):
    assert attention(lib) == OK and lib.fake_launches() == 2


def test_a_refused_attention_kernel_is_not_followed_by_the_join(lib):
    # the join takes rows and slots from the workspace, which nobody wrote
    lib.fake_set(1, 0, 0)
    assert attention(lib) == LAUNCH
    assert lib.fake_launches() == 1
    assert attention(lib) == OK and lib.fake_launches() == 3


def test_a_refused_join_is_reported(lib):
    lib.fake_set(2, 0, 0)
    assert attention(lib) == LAUNCH and lib.fake_launches() == 2


@pytest.mark.parametrize("name", ["write", "read", "logits", "attention"])
def test_a_refused_launch_is_reported_and_not_left_behind(lib, name):
    call = calls(lib)[name]
    assert call() == OK
    lib.fake_set(1, 0, 0)
    assert call() == LAUNCH
    assert lib.fake_last() == 0     # the caller's next look at the last error does not find this one
    assert call() == OK


@pytest.mark.parametrize("name", ["write", "read", "logits", "attention"])
def test_an_older_error_is_not_taken_for_a_launch(lib, name):
    call = calls(lib)[name]
    assert call() == OK
    lib.fake_set(0, 0, 700)          # some earlier call of the program failed
    assert call() == OK and lib.fake_launches() >= 1
    assert lib.fake_last() == 700    # and its error is still there to be seen


def test_a_set_up_that_failed_is_tried_again(lib):
    # say, in a stream capture or with the memory used up: the calls after it work
    lib.fake_set(0, 1, 0)
    assert attention(lib) == CUDA and lib.fake_launches() == 0
    assert lib.fake_last() == 0
    assert attention(lib) == OK and lib.fake_launches() == 2
    assert all(call() == OK for call in calls(lib).values())


@pytest.mark.parametrize("page", [1, 64, 1024])
def test_attention_counts_positions_in_32_bits(lib, page):
    # rows that end within a few steps of 2^31 positions: the places past their end would not be counted
    c = cache(pages=4, page=page)
    most = (2 ** 31 - 1025) // page
    assert attention(lib, cols=most, c=c) == OK and lib.fake_launches() == 2
    for cols in (most + 1, (2 ** 31 - 1) // page):
        assert attention(lib, cols=cols, c=c) == UNSUPPORTED and lib.fake_launches() == 2

    def selected(n):
        return lib.fp8_mqa_attention_paged(P, BF16, 1, 8, 1024, 128, c, c, P, 9, 9, P, P, n, n, 1.0, P, P, P, 1 << 40, None)
    assert selected(2 ** 31 - 1025) == OK
    assert selected(2 ** 31 - 1024) == selected(2 ** 31 - 1) == UNSUPPORTED
