"""Keys and values written in one call into caches of different page counts: a slot on a page that only one of them has
goes into that one, and nothing else of either changes."""
import numpy as np
import pytest
import torch

import fp8_mqa_logits_02_gb300 as fm
import test_paged as t8
import test_paged4 as t4
from oracle import paged, step
from test_paged import f64, gpu, same

pytestmark = pytest.mark.gpu

PAGE = 16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    fm.build()
    fm.lib()


def held(kind, c):
    """A cache's data, groups (4 bits) and scales."""
    if kind == "4 bits":
        codes = c[0].cpu().numpy()
        return [step.unpack(codes) if codes.size else np.empty(codes.shape[:3] + (codes.shape[3] * 2,)), f64(c[1]), f64(c[2])]
    return [f64(c[0]), f64(c[1])]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("k_pages,v_pages", [(2, 4), (4, 2), (1, 3), (3, 1), (0, 2), (2, 0)])
@pytest.mark.parametrize("kind", ["4 bits", "e4m3"])
def test_pages_of_one_cache_only(kind, k_pages, v_pages, dim, dtype):
    rng = np.random.default_rng(k_pages * 10 + v_pages)
    heads, most = 3, max(k_pages, v_pages)
    T = most * PAGE
    make = t4.cache if kind == "4 bits" else t8.cache
    caches = [make(rng, n, PAGE, heads, dim) for n in (k_pages, v_pages)]
    # (numpy's empty arrays have strides of 0)
    caches = [tuple(x if x.numel() else torch.empty(x.shape, dtype=x.dtype, device="cuda") for x in c) for c in caches]
    k, v = (torch.from_numpy(rng.standard_normal((T + 3, heads, dim))).to(dtype).cuda() for _ in range(2))
    slots = np.concatenate([rng.permutation(T), [-1, T, T + PAGE]]).astype(np.int32)    # every slot once, and some outside
    quantise = step.quantise4 if kind == "4 bits" else paged.quantise32
    want = []
    for x, c, pages in ((k, caches[0], k_pages), (v, caches[1], v_pages)):
        ok = (slots >= 0) & (slots < pages * PAGE)
        now = held(kind, c)
        for to, new in zip(now, quantise(x.float().cpu().numpy())):
            to[slots[ok] // PAGE, slots[ok] % PAGE] = new[ok]
        want.append(now)
    if kind == "4 bits":
        (kc, kg, ks), (vc, vg, vs) = caches
        fm.cache_write(gpu(slots), k, kc.view(t4.F4), ks, v, vc.view(t4.F4), vs, k_groups=kg, v_groups=vg)
    else:
        (kc, ks), (vc, vs) = caches
        fm.cache_write(gpu(slots), k, kc, ks, v, vc, vs)
    for c, now in zip(caches, want):
        for got, w in zip(held(kind, c), now):
            assert same(got, w)
