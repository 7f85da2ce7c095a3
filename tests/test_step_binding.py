"""What the Python side of page tables, norms with rotation and 4-bit caches refuses before the library is called."""
import types

import pytest
import torch

import fp8_mqa_logits_02_gb300 as fm

F4, F8 = torch.float4_e2m1fn_x2, torch.float8_e4m3fn


@pytest.mark.parametrize("name,n", [("pages_update", 7), ("norm_rotate", 4)])
def test_a_stream_of_another_device_is_refused(name, n, monkeypatch):
    made = []
    compiled = types.SimpleNamespace(**{name: lambda *a: made.append(a)})
    monkeypatch.setattr(fm.paged, "_binding", lambda: compiled)
    tensors = [types.SimpleNamespace(device=torch.device("cuda:0"))] * n
    with pytest.raises(ValueError, match="stream is on cuda:1, expected cuda:0"):
        getattr(fm, name)(*tensors, stream=types.SimpleNamespace(device=torch.device("cuda:1")))
    assert not made
    getattr(fm, name)(*tensors)
    assert len(made) == 1


def raises(kind, match, call):
    with pytest.raises(kind, match=match):
        call()


def ints(*shape):
    return torch.zeros(shape, dtype=torch.int32, device="cuda")


@pytest.mark.gpu
@pytest.mark.parametrize("total", [2 ** 31, 2 ** 61, 2 ** 62, 2 ** 63 - 1])
def test_more_new_tokens_than_are_counted_are_refused_before_anything_is_allocated(total):
    fm.build()
    held = torch.cuda.memory_reserved()
    raises(ValueError, "total", lambda: fm.pages_update(ints(2, 4), ints(2), ints(2), ints(9), ints(1), 64, total))
    assert torch.cuda.memory_reserved() - held < 1 << 30


@pytest.mark.gpu
def test_pages_update_refusals():
    fm.build()

    def f(table=ints(2, 4), lens=ints(2), change=ints(2), free=ints(9), n_free=ints(1), page=64, total=2):
        return fm.pages_update(table, lens, change, free, n_free, page, total)
    assert isinstance(f(), fm.PagesStep) and f().slots.tolist() == [-1, -1]
    raises(TypeError, "table must be int32", lambda: f(table=ints(2, 4).long()))
    raises(TypeError, "must be a torch.Tensor", lambda: f(lens=[1, 2]))
    raises(ValueError, "lens must be", lambda: f(lens=ints(3)))
    raises(ValueError, "change must be", lambda: f(change=ints(1)))
    raises(ValueError, "n_free must be", lambda: f(n_free=ints(2)))
    raises(ValueError, "lens must be contiguous", lambda: f(lens=ints(2, 2)[:, 0]))
    raises(ValueError, "CUDA", lambda: f(free=ints(9).cpu()))
    raises(ValueError, "overlap", lambda: f(table=ints(1, 4).expand(2, 4)))
    raises(ValueError, "page_size", lambda: f(page=0))
    raises(ValueError, "page_size", lambda: f(page=2 ** 31))
    raises(ValueError, "total", lambda: f(total=-1))
    raises(fm.Fp8MqaError, "UNSUPPORTED", lambda: f(table=ints(8193, 1), lens=ints(8193), change=ints(8193)))
    raises(fm.Fp8MqaError, "UNSUPPORTED", lambda: f(page=2 ** 30))


@pytest.mark.gpu
def test_norm_rotate_refusals():
    fm.build()
    x = torch.ones(3, 2, 128, device="cuda", dtype=torch.bfloat16)
    w = torch.ones(128, device="cuda")

    def f(q=x, k=x, pos=ints(3), freq=torch.zeros(64, device="cuda"), **kw):
        return fm.norm_rotate(q, k, pos, freq, **kw)
    assert len(f()) == 2
    raises(TypeError, "q must be bfloat16", lambda: f(q=x.double()))
    raises(TypeError, "k must be", lambda: f(k=x.half()))
    raises(TypeError, "dtype must be", lambda: f(dtype=torch.float16))
    raises(TypeError, "dtype must be", lambda: f(dtype=3))
    raises(TypeError, "positions must be", lambda: f(pos=ints(3).float()))
    raises(TypeError, "inv_freq must be", lambda: f(freq=torch.zeros(64, device="cuda").double()))
    raises(TypeError, "q_weight must be", lambda: f(q_weight=w.half()))
    raises(ValueError, "q must be", lambda: f(q=x[0]))
    raises(ValueError, "heads of 64 or 128", lambda: f(q=x[..., :96]))
    raises(ValueError, "k must be", lambda: f(k=x[:2]))
    raises(ValueError, "k must be", lambda: f(k=x[..., :64].contiguous()))
    raises(ValueError, "contiguous", lambda: f(q=torch.ones(3, 128, 2, device="cuda").transpose(1, 2), k=None))
    raises(ValueError, "positions must be", lambda: f(pos=ints(4)))
    raises(ValueError, "inv_freq must be", lambda: f(freq=torch.zeros(60, device="cuda")))
    raises(ValueError, "inv_freq must be", lambda: f(freq=torch.zeros(72, device="cuda")))
    raises(ValueError, "q_weight must be", lambda: f(q_weight=w[:64]))
    raises(ValueError, "go with k", lambda: f(k=None, k_weight=w))
    raises(ValueError, "does not go with", lambda: f(dtype=F8, q_out=x.clone()))
    raises(ValueError, "q_out must be", lambda: f(q_out=x.float()))
    raises(ValueError, "overlap", lambda: f(q_out=x[:1].expand(3, 2, 128)))
    raises(ValueError, "overlap", lambda: f(q_out=torch.zeros(1024, device="cuda").bfloat16().as_strided((3, 2, 128), (128, 128, 1))))
    by_heads = torch.zeros(2, 3, 128, device="cuda", dtype=torch.bfloat16).transpose(0, 1)
    assert torch.equal(f(q_out=by_heads)[0], f()[0])
    raises(ValueError, "CUDA", lambda: f(q=x.cpu()))
    raises(ValueError, "CUDA", lambda: f(freq=torch.zeros(64)))


@pytest.mark.gpu
def test_4_bit_cache_refusals():
    fm.build()
    data = torch.zeros(4, 16, 2, 64, dtype=torch.uint8, device="cuda").view(F4)
    e4m3 = torch.zeros(4, 16, 2, 128, device="cuda").to(F8)
    groups = torch.zeros(4, 16, 2, 8, device="cuda").to(F8)
    scale = torch.ones(4, 16, 2, device="cuda")
    x, q = (torch.ones(3, n, 128, device="cuda", dtype=torch.bfloat16) for n in (2, 8))

    def write(data=data, scale=scale, groups=groups, **kw):
        fm.cache_write(ints(3), x, data, scale, k_groups=groups, **kw)

    def read(data=data, scale=scale, groups=groups, dtype=torch.bfloat16):
        return fm.cache_read(data, scale, ints(1, 4), torch.tensor([0, 3], dtype=torch.int32, device="cuda"), 3, dtype, groups=groups)

    def attend(k=data, v=data, kg=groups, vg=groups, ks=scale, vs=scale):
        return fm.attention_paged(q, k, v, ints(3, 4), ints(3) + 5, k_scale=ks, v_scale=vs, k_groups=kg, v_groups=vg)
    write()
    assert read().shape == (3, 2, 128) and attend().shape == (3, 8, 128)
    for call in (write, read):
        raises(TypeError, "groups must be a torch.Tensor", lambda: call(groups=None))
        raises(ValueError, "groups must be float8", lambda: call(groups=groups.float()))
        raises(ValueError, "groups must be float8", lambda: call(groups=groups[..., :4]))
        raises(ValueError, "groups must be contiguous", lambda: call(groups=groups.repeat_interleave(2, -1)[..., ::2]))
        raises(ValueError, "groups go with float4", lambda: call(data=e4m3))
        raises(ValueError, "scale must be float32", lambda: call(scale=scale.half()))
        raises(TypeError, "data must be", lambda: call(data=data.view(torch.uint8)))
    raises(ValueError, "v, v_data and v_scale go together", lambda: write(v_groups=groups))
    raises(TypeError, "k data's type", lambda: write(v=x, v_data=e4m3, v_scale=scale))
    raises(TypeError, "16|float32", lambda: read(dtype=F8))
    raises(TypeError, "16|float32", lambda: read(dtype=F4))
    raises(TypeError, "groups must be a torch.Tensor", lambda: attend(vg=None))
    raises(ValueError, "one shape and type", lambda: attend(v=e4m3, vg=None))
    raises(TypeError, "scale must be a torch.Tensor", lambda: attend(ks=None))
    one = torch.zeros(4, 16, 1, 64, dtype=torch.uint8, device="cuda").view(F4)
    with pytest.raises((TypeError, ValueError)):      # the indexer's keys stay e4m3
        fm.logits_paged(torch.zeros(1, 1, 32, 128, device="cuda").to(F8), one, scale[:, :, :1], torch.ones(1, 1, 32, device="cuda"),
                        ints(1, 4), ints(1))
