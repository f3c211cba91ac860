"""The binding of include/glr.h refuses tensors and streams of a device that is not the current one,
on which it would launch. One GPU, or none, is enough: the current device is what a stub says."""
import types

import pytest
import torch

from state_space_sequence_gb300 import glr


def test_the_tensors_device_is_the_current_one(monkeypatch):
    monkeypatch.setattr(glr, "_current_device", lambda: 0)
    with pytest.raises(ValueError, match="cuda:1.*cuda:0"):
        glr._stream(None, 1)
    with pytest.raises(ValueError, match="cuda:1.*cuda:0"):
        glr._stream(types.SimpleNamespace(device_index=1, cuda_stream=5), 1)


def test_the_streams_device_is_the_tensors(monkeypatch):
    monkeypatch.setattr(glr, "_current_device", lambda: 1)
    with pytest.raises(ValueError, match="stream"):
        glr._stream(types.SimpleNamespace(device_index=0, cuda_stream=5), 1)
    assert glr._stream(types.SimpleNamespace(device_index=1, cuda_stream=5), 1) == 5


@pytest.mark.gpu
def test_every_call_refuses_another_device(monkeypatch):
    """And writes nothing: the state that a step would have replaced is as it was."""
    x = torch.randn(2, 4, 16, device="cuda")
    rows, h, w = x.view(8, 16), torch.ones(2, 16, device="cuda"), torch.ones(16, device="cuda")
    one = torch.ones(1, device="cuda")
    _, _, states = glr.glr_scan(x, x, x, w, save_states=True)
    kept = glr.glr_ckpt_pack(rows)
    side = torch.cuda.Stream()
    calls = [lambda s: glr.glr_scan(x, x, x, w, stream=s),
             lambda s: glr.glr_scan_backward(x, x, x, w, x, states, stream=s),
             lambda s: glr.glr_step(x[:, 0], x[:, 0], x[:, 0], w, h, stream=s),
             lambda s: glr.glr_join(rows, rows, rows, w, one, w, stream=s),
             lambda s: glr.glr_join_backward(rows, rows, rows, rows, rows, w, one, w, stream=s),
             lambda s: glr.glr_ckpt_pack(rows, stream=s),
             lambda s: glr.glr_ckpt_unpack(kept, stream=s)]
    monkeypatch.setattr(glr, "_current_device", lambda: x.get_device() + 1, raising=False)
    for call in calls:
        for s in (None, side):
            with pytest.raises(ValueError):
                call(s)
    torch.cuda.synchronize()
    assert (h == 1).all()
