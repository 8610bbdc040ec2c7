"""Prepared calls, without a device."""
import pytest
import torch


def test_prepared_call_refuses_another_device(monkeypatch):
    """The library launches on the current device: a call prepared on another
    one would hand it pointers it cannot read."""
    import gqa_flash_attention_prefill_gb300 as pkg
    current, issued = [0], []
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[0])
    monkeypatch.setattr(torch.cuda, "device_count", lambda: 2)
    op = pkg.PreparedOp(lambda *a: issued.append(a) or 0, (1, 2), "gqa_rope", None)
    op()
    current[0] = 1
    with pytest.raises(ValueError, match="prepared on cuda:0"):
        op()
    current[0] = 0
    op()
    assert issued == [(1, 2)] * 2
