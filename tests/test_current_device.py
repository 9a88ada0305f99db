"""Calls on tensors of another device than the current one: refused before anything is launched
(the current device is a stand-in here)."""
import pytest
import torch

from selective_state_space_sscan_amd import sscan


def test_stream_of_another_device(monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 0x1000 + i, raising=False)
    assert sscan._stream(torch.device("cuda", 1)).value == 0x1001
    with pytest.raises(ValueError, match="current device is cuda:1"):
        sscan._stream(torch.device("cuda", 0))


@pytest.mark.gpu
def test_calls_are_refused(monkeypatch):
    x, w = torch.randn(2, 6, 64, device="cuda"), torch.ones(64, device="cuda")
    state, packed = torch.zeros(2, 64, device="cuda"), sscan.pack8(x)
    calls = [lambda: sscan.rec_fwd(x, x), lambda: sscan.rec_fwd(x, x, keep=True), lambda: sscan.rec_bwd(x, x, x),
             lambda: sscan.rec_step(state, x[:, 0], x[:, 0]), lambda: sscan.gated_recurrence(x, x), lambda: sscan.pack8(x),
             lambda: sscan.unpack8(packed), lambda: sscan.layer_norm(x, w), lambda: sscan.layer_norm_bwd(x, x, w),
             lambda: sscan.gated_norm(x, x, w), lambda: sscan.add_norm(x, None, w)]
    for call in calls:
        call()
    held = state.clone()
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1)
    for call in calls:
        with pytest.raises(ValueError, match="current device"):
            call()
    assert torch.equal(state, held)
