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
