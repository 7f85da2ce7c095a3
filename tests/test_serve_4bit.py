"""The example that runs page tables, norms with rotation and 4-bit caches together: its state and its last step against
the plain forms."""
import os
import sys

import numpy as np
import pytest
import torch

import fp8_mqa_logits_02_gb300 as fm
from oracle import paged as plain
from oracle import step as plain_step
from test_paged4 import U

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu
VALUES = plain.e4m3_values()


def f64(t):
    return VALUES[t.cpu().view(torch.uint8).numpy()] if t.dtype == torch.float8_e4m3fn else t.cpu().double().numpy()


def rows(codes, groups, scale):
    return plain_step.unpack(codes.cpu().view(torch.uint8).numpy()) * np.repeat(f64(groups), 16, -1) * f64(scale)[..., None]


def test_serve_4bit_example():
    import serve_4bit as ex
    fm.build()
    prompt, steps, top = (300, 70, 1), 6, 32
    layer, step, out = ex.main(prompt, steps, top, seed=3)
    lens = [300 + 3, 70 + 6, 1 + 6]
    assert layer.lens.tolist() == lens and torch.isfinite(out.float()).all()
    # every page is held once, or free
    table = layer.table.cpu().numpy()
    held = [int(p) for b, n in enumerate(lens) for p in table[b, :-(-n // ex.PAGE)]]
    free = layer.free[:layer.n_free.item()].tolist()
    assert sorted(held + free) == list(range(layer.k.shape[0]))
    assert step.new.positions.tolist() == [n - 1 for n in lens] and step.new.changed.tolist() == [1, 1, 1]

    # the last step's new rows are what was written, and the slots are the tables'
    slots = step.new.slots.cpu().numpy()
    at = (slots // ex.PAGE, slots % ex.PAGE)
    assert slots.tolist() == [table[b, (n - 1) // ex.PAGE] * ex.PAGE + (n - 1) % ex.PAGE for b, n in enumerate(lens)]
    q, k, v = step.qkv.split([ex.Q_HEADS, ex.KV_HEADS, ex.KV_HEADS], dim=1)
    pos, freq = step.new.positions.cpu().numpy(), f64(layer.inv_freq)
    want_k, size = plain_step.norm_rotate(f64(k), f64(layer.k_weight), pos, freq, 1e-6, False)
    K, V = rows(layer.k, layer.k_groups, layer.k_scale), rows(layer.v, layer.v_groups, layer.v_scale)
    by = layer.v_scale[at].cpu().numpy()
    values, groups, scale = plain_step.quantise4(v.float().cpu().numpy())
    assert np.array_equal(by, scale) and np.array_equal(V[at], values * np.repeat(groups, 16, -1) * scale.astype(np.float64)[..., None])
    # a key, rounded to bfloat16 and to 4 bits of its group's largest value m: off by (1 + 2^-4) m / 6 at most (half the
    # step of 2 from 4 to 6, or what is cut off where the group's scale was rounded down), and 2^-7 of it before that
    m = np.repeat(np.abs(want_k).reshape(3, ex.KV_HEADS, -1, 16).max(-1), 16, -1)
    assert np.all(np.abs(K[at] - want_k) <= (1 + 2.0 ** -4) * m / 6 + 2.0 ** -7 * size.max(-1, keepdims=True))

    # the attention of the last step: on the cache as it is, over the positions that the logits select
    want_q, q_size = plain_step.norm_rotate(f64(q), f64(layer.q_weight), pos, freq, 1e-6, False)
    (index_q, index_by), _ = fm.norm_rotate(step.index_q, None, step.new.positions, layer.index_freq, interleaved=True,
                                            dtype=torch.float8_e4m3fn)
    w = f64(step.w * index_by)[:, None]
    scores, _ = plain.logits(f64(index_q)[:, None], w, f64(layer.index)[:, :, 0], f64(layer.index_scale)[:, :, 0], table, lens,
                             table.shape[1] * ex.PAGE)
    got = f64(out)
    for b, n in enumerate(lens):
        order = np.argsort(-scores[b, :n], kind="stable")
        if n > top and scores[b, order[top - 1]] - scores[b, order[top]] < 1e-5:
            continue                                    # a near-tie at the edge of the selection
        idx = np.full((1, top), -1)
        idx[0, :min(n, top)] = order[:top]
        want, _, size, dots = plain.attention(want_q[b:b + 1], K, V, table[b:b + 1], [n], ex.DIM ** -0.5, idx)
        # q is rounded to bfloat16 (2^-8 of it), and that moves the scores by as much of their absolute terms
        dx = (2.0 ** -8 + (ex.DIM + 24) * U) * dots[..., None] * (q_size[b:b + 1].max(-1, keepdims=True) / np.abs(want_q[b:b + 1]).max(-1, keepdims=True))
        tol = (np.exp(2 * dx) - 1 + 2.0 ** -10) * size + 2.0 ** -14 * size.max(-1, keepdims=True) + 2.0 ** -8 * np.abs(want) + 1e-6
        assert np.all(np.abs(got[b:b + 1] - want) <= tol)
