"""What the paged operators' Python side refuses before the library is called."""
import types

import pytest
import torch

import fp8_mqa_logits_02_gb300 as fm

CALLS = {"cache_write": 4, "cache_read": 5, "logits_paged": 6, "attention_paged": 5}   # arguments without a default


@pytest.mark.parametrize("name", CALLS)
def test_a_stream_of_another_device_is_refused(name, monkeypatch):
    # the kernels run on the tensors' device, where the stream that was asked for does not exist
    made = []
    compiled = types.SimpleNamespace(**{n: lambda *a: made.append(a) for n in CALLS})
    monkeypatch.setattr(fm.paged, "_binding", lambda: compiled)
    tensors = [types.SimpleNamespace(device=torch.device("cuda:0"))] * CALLS[name]
    with pytest.raises(ValueError, match="stream is on cuda:1, expected cuda:0"):
        getattr(fm, name)(*tensors, stream=types.SimpleNamespace(device=torch.device("cuda:1")))
    assert not made
    getattr(fm, name)(*tensors)
    assert len(made) == 1


@pytest.mark.gpu
def test_tables_and_lists_of_2_to_32_columns_are_refused():
    # the C interface counts columns in 32 bits: 2^32 + 1 of them would pass for one
    n = 2 ** 32 + 1
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB of device memory")
    fm.build()
    wide = torch.empty(n, dtype=torch.int32, device="cuda").view(1, n)     # never read
    f8 = torch.float8_e4m3fn
    kd, ks = torch.zeros(1, 64, 1, 128, device="cuda").to(f8), torch.ones(1, 64, 1, device="cuda")
    table, lens = torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.ones(1, dtype=torch.int32, device="cuda")
    q = torch.ones(1, 4, 128, device="cuda").bfloat16()
    starts = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    for call in (lambda: fm.attention_paged(q, kd, kd, table, lens, k_scale=ks, v_scale=ks, indices=wide),
                 lambda: fm.attention_paged(q, kd, kd, wide, lens, k_scale=ks, v_scale=ks),
                 lambda: fm.logits_paged(torch.ones(1, 1, 32, 128, device="cuda").to(f8), kd, ks, torch.ones(1, 1, 32, device="cuda"),
                                         wide, lens, max_len=64),
                 lambda: fm.cache_read(kd, ks, wide, starts, 1)):
        with pytest.raises(ValueError, match="too large"):
            call()
