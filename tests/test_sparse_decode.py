"""The example that runs the paged operators together: its last step against a plain 64-bit one."""
import os
import sys

import numpy as np
import pytest
import torch

import fp8_mqa_logits_02_gb300 as fm
from oracle import paged as plain

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def test_sparse_decode_example():
    import sparse_decode as ex
    fm.build()
    prompt, steps, top = (300, 70, 1), 3, 32
    layer, logits, out = ex.main(prompt, steps, top, seed=3)
    lens = [n + steps for n in prompt]
    assert layer.lens.tolist() == lens and out.shape == (3, ex.Q_HEADS, ex.DIM)
    assert torch.isfinite(out.float()).all()
    # the prompt's logits are causal within each request
    want = np.zeros((sum(prompt), sum(prompt)), bool)
    at = 0
    for n in prompt:
        want[at:at + n, at:at + n] = np.tril(np.ones((n, n), bool))
        at += n
    assert np.array_equal(np.isfinite(logits.cpu().numpy()), want)

    # one more step, against the plain forms on the same caches
    gen = torch.Generator(device="cuda").manual_seed(9)
    q = torch.randn((3, ex.Q_HEADS, ex.DIM), generator=gen, device="cuda").to(torch.bfloat16)
    q8 = torch.randn((3, 1, 32, 128), generator=gen, device="cuda").to(torch.float8_e4m3fn)
    w = torch.randn((3, 1, 32), generator=gen, device="cuda") / 64
    got = layer.step(q, q8, w, top).double().cpu().numpy()
    values = plain.e4m3_values()

    def f64(t):
        return values[t.cpu().view(torch.uint8).numpy()] if t.dtype == torch.float8_e4m3fn else t.cpu().double().numpy()

    table = layer.table.cpu().numpy()
    N = layer.cols * ex.PAGE
    scores, _ = plain.logits(f64(q8), f64(w), f64(layer.index)[:, :, 0], f64(layer.index_scale)[:, :, 0], table, lens, N)
    k, v = f64(layer.k) * f64(layer.k_scale)[..., None], f64(layer.v) * f64(layer.v_scale)[..., None]
    for b, n in enumerate(lens):
        # the selection of the 64-bit scores; a near-tie at its edge may differ, and is then left out
        order = np.argsort(-scores[b, :n], kind="stable")
        if n > top and scores[b, order[top - 1]] - scores[b, order[top]] < 1e-5:
            continue
        idx = np.full((1, top), -1)
        idx[0, :min(n, top)] = order[:top]
        want, _, size, _ = plain.attention(f64(q)[b:b + 1], k, v, table[b:b + 1], [n], ex.DIM ** -0.5, idx)
        # weights of 11 bits, a result of 8 (see tests/test_paged.py)
        tol = (2.0 ** -10) * size + 2.0 ** -14 * size.max(-1, keepdims=True) + 2.0 ** -8 * np.abs(want) + 1e-6
        assert np.all(np.abs(got[b:b + 1] - want) <= tol)
