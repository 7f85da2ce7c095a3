"""Small softmax weights over long caches: a first position that takes nearly all of the softmax, with values
of zero in half of its channels, leaves those channels of the output to tens of thousands of weights near
2^-25 of it.

A weight goes to the second product in 16 bits, relative to a reference.  In f16 a weight that is the reference
itself is held as 2^7, so those under 2^-14 are held to half a unit of 2^-24, 2^-32 of the reference; n of them
are off by n 2^-32 at most, next to the terms of tests/test_paged.py.
"""
import numpy as np
import pytest
import torch

import fp8_mqa_logits_02_gb300 as fm
from oracle import paged as plain
from test_paged import F8, U, as_rows, f64, gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    fm.build()
    fm.lib()


@pytest.mark.parametrize("dtype,kind", [(torch.float16, torch.float16), (torch.float16, F8), (torch.bfloat16, F8),
                                        (torch.bfloat16, torch.bfloat16)])
def test_weights_far_below_the_first_are_not_lost(dtype, kind):
    page, pages, dim, heads = 64, 512, 64, 8
    n = page * pages
    k = torch.zeros(pages, page, 1, dim)
    k[0, 0] = 1.0
    v = torch.ones(pages, page, 1, dim)
    v[0, 0, 0, ::2] = 0.0
    kd, vd = k.to(kind).cuda(), v.to(kind).cuda()
    scale = torch.ones(pages, page, 1, device="cuda") if kind == F8 else None
    # rows enough that a CTA takes whole ones; all of them alike, over one sequence
    B = 6 * torch.cuda.get_device_properties(0).multi_processor_count
    q1 = torch.full((1, heads, dim), 2.203125).to(dtype).cuda()     # a score of 17.625: 2^-25.4 for the others
    table = np.arange(pages, dtype=np.int32)[None]
    lens = gpu(np.full(B, n, np.int32))
    got = fm.attention_paged(q1.expand(B, -1, -1), kd, vd, gpu(table).expand(B, -1), lens, k_scale=scale, v_scale=scale)
    assert (got == got[0]).all()
    got = got[:1].double().cpu().numpy()
    want, _, size, dots = plain.attention(f64(q1), as_rows(kd, scale), as_rows(vd, scale), table, [n], dim ** -0.5)
    assert (want[..., ::2] < 1e-3).all() and (want[..., ::2] > 5e-4).all()
    dx = (dim + 8) * U * dots
    bits = 2.0 ** -8 if kind == torch.bfloat16 else 2.0 ** -11
    last = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -11
    tol = (2 * dx[..., None] + 2.0 ** -20 + bits) * size + n * 2.0 ** -32 + last * np.abs(want) + 2.0 ** -25
    assert np.all(np.abs(got - want) <= tol), (np.abs(got - want) / tol).max()
