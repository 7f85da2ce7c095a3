"""Results of norm_rotate that share memory with an argument or with one another are refused; slices of one tensor beside
one another are not."""
import pytest
import torch

import fp8_mqa_logits_02_gb300 as fm
from test_norm_rotate import freq

pytestmark = pytest.mark.gpu

T, DIM = 70, 128


@pytest.fixture(scope="module", autouse=True)
def _lib():
    fm.build()
    fm.lib()


def make():
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(T, 9, DIM, generator=gen, device="cuda").bfloat16()
    return x, torch.arange(T, dtype=torch.int32, device="cuda"), freq(64), torch.rand(DIM, generator=gen, device="cuda") + 0.5


@pytest.mark.parametrize("what,call", [
    ("k", lambda x, p, f, w: fm.norm_rotate(x[:, :4], x[:, 4:8], p, f, q_out=x[:, 4:8], k_out=x[:, :4])),
    ("k", lambda x, p, f, w: fm.norm_rotate(x[:, :4], x[:, 4:8], p, f, q_out=x[:, 4:8])),
    ("q", lambda x, p, f, w: fm.norm_rotate(x[:, :4], x[:, 4:8], p, f, k_out=x[:, :4])),
    ("k", lambda x, p, f, w: fm.norm_rotate(x[:, :4], x[:, :4], p, f, q_out=x[:, :4])),
    ("q", lambda x, p, f, w: fm.norm_rotate(x[:, :4], None, p, f, q_out=x[:, 1:5])),
    ("q", lambda x, p, f, w: fm.norm_rotate(x[1:, :4], None, p[1:], f, q_out=x[:-1, :4])),
    ("q", lambda x, p, f, w: fm.norm_rotate(x[:, :4], None, p, f, q_out=x[:, :7:2])),
    ("k", lambda x, p, f, w: fm.norm_rotate(x[:, :4], x[:, 4:8], p, f, k_out=x[:, 5:9])),
    ("q_out", lambda x, p, f, w: [y := torch.empty_like(x), fm.norm_rotate(x[:, :4], x[:, 4:8], p, f, q_out=y[:, :4], k_out=y[:, 3:7])]),
    ("q_weight", lambda x, p, f, w: fm.norm_rotate(x[:, :4], None, p, f, x[3, 2], q_out=x[:, :4])),
    ("k_weight", lambda x, p, f, w: fm.norm_rotate(x[:, :4], x[:, 4:8], p, f, None, x[T - 1, 0], q_out=x[:, :4])),
    ("positions", lambda x, p, f, w: fm.norm_rotate(x[:, :4], None, x[5, :2].flatten()[:140].view(torch.int32), f, q_out=x[:, :4])),
    ("inv_freq", lambda x, p, f, w: fm.norm_rotate(x[:, :4], None, p, x[9, 3, :64].view(torch.float32), q_out=x[:, :4]))])
def test_refused(what, call):
    x, *rest = make()
    before = x.clone()
    with pytest.raises(ValueError, match=f"_out must not overlap {what}( |$)"):
        call(x, *rest)
    assert torch.equal(x, before)


def test_beside_one_another():
    x, p, f, w = make()
    want = fm.norm_rotate(x[:, :4], x[:, 4:6], p, f, w, w)

    def same(got):
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    same(fm.norm_rotate(x[:, :4], x[:, 4:6], p, f, w, w, q_out=torch.empty_like(x)[:, 2:6], k_out=torch.empty_like(x)[:, :2]))
    to = torch.zeros(T, 6, DIM, dtype=x.dtype, device="cuda")
    same(fm.norm_rotate(x[:, :4], x[:, 4:6], p, f, w, w, q_out=to[:, 2:], k_out=to[:, :2]))
    # into heads of the same tensor that are not read
    y = x.clone()
    same(fm.norm_rotate(y[:, :4], y[:, 4:6], p, f, w, w, q_out=y[:, :4], k_out=y[:, 7:]))
    assert torch.equal(y[:, 4:7], x[:, 4:7])
    # q, k and v of each head in turn, q and k in place
    y = x.clone()
    q, k = y[:, 0::3], y[:, 1::3]
    want = fm.norm_rotate(q, k, p, f, w, w)
    same(fm.norm_rotate(q, k, p, f, w, w, q_out=q, k_out=k))
    assert torch.equal(y[:, 2::3], x[:, 2::3])
