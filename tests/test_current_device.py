"""The library launches on the current device, so tensors of another one are
refused before anything is launched.  The device is a pretence here (tensors that
say which they live on, a library that only counts its calls): a launch with
another device's addresses would fault."""
import pytest
import torch

import state_space_model_sm_gb300 as ssd
from state_space_model_sm_gb300 import layer_ops


class Placed(torch.Tensor):
    """A CPU tensor that says it lives on cuda:1."""

    def get_device(self):
        return 1


class CountingLibrary:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append(name)
            return 64 if name.endswith("workspace_size") else 0
        return call


def t(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype).as_subclass(Placed)


def layer_calls():
    x, w, f = t(2, 5, 8), t(8, 4), t(8)
    x1, A, B, B1 = t(2, 8), t(8, 16), t(2, 5, 1, 16), t(2, 1, 16)
    r, o16 = t(6, 8), torch.float32
    return {
        "causal_conv_fwd": lambda: ssd.causal_conv_fwd(x, w, f),
        "causal_conv_bwd": lambda: ssd.causal_conv_bwd(x, w, f, x),
        "causal_conv_step": lambda: ssd.causal_conv_step(x1, t(2, 3, 8), w, f),
        "causal_conv_step, checked one by one":
            lambda: ssd.causal_conv_step(x1, t(2, 3, 8), w, f, out_dtype=o16),
        "selective_scan_fwd": lambda: ssd.selective_scan_fwd(x, x, f, A, B, B, f, x),
        "selective_scan_bwd": lambda: ssd.selective_scan_bwd(x, x, f, A, B, B, f, x, x),
        "selective_step": lambda: ssd.selective_step(x1, x1, f, A, B1, B1, t(2, 8, 16), f, x1),
        "selective_step, checked one by one":
            lambda: ssd.selective_step(x1, x1, f, A, B1, B1, t(2, 8, 16), f, x1, out_dtype=o16),
        "ssd_step": lambda: ssd.ssd_step(t(2, 4, 8), t(2, 4), t(4), t(4), B1, B1, t(2, 4, 8, 16)),
        "ssd_step, checked one by one":
            lambda: ssd.ssd_step(t(2, 4, 8), t(2, 4), t(4), t(4), B1, B1, t(2, 4, 8, 16),
                                 out_dtype=o16),
        "block_norm_fwd": lambda: ssd.block_norm_fwd(r, r, f, f, t(1, 8)),
        "block_norm_fwd, checked one by one": lambda: ssd.block_norm_fwd(r, r, f, f, t(2, 8)),
        "block_norm_bwd": lambda: ssd.block_norm_bwd(r, r, f, f, t(2, 8), r, r),
    }


@pytest.mark.parametrize("current", [0, 1])
@pytest.mark.parametrize("name", list(layer_calls()))
def test_layer_operators(monkeypatch, name, current):
    lib = CountingLibrary()
    monkeypatch.setattr(layer_ops, "_lib", lib)
    monkeypatch.setattr(layer_ops, "_stream", lambda dev: 0)
    monkeypatch.setattr(layer_ops, "_current_device", lambda: current, raising=False)
    call = layer_calls()[name]
    if current == 1:  # the tensors' own: one call gets through
        call()
        assert [c for c in lib.calls if not c.endswith("workspace_size")] == ["ssd_" + name.split(",")[0]
                                                                              .removeprefix("ssd_")]
    else:
        with pytest.raises(ValueError, match="cuda:1.*current device.*cuda:0"):
            call()
        assert lib.calls == []


def test_stream_of_a_device(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    with pytest.raises(ValueError, match="cuda:1.*current device.*cuda:0"):
        ssd._stream(torch.device("cuda", 1))
    with pytest.raises(ValueError, match="CUDA device"):
        ssd._stream(torch.device("cpu"))


@pytest.mark.gpu
def test_scan_and_norm(cuda_lib, monkeypatch):
    """Tensors of cuda:0 while the current device says that it is another (here it is
    not, so the launches that are to be refused would be sound)."""
    z = lambda *s: torch.zeros(*s, device="cuda:0")  # noqa: E731
    x, dt, h, B, s = z(1, 64, 2, 16), z(1, 64, 2), z(2), z(1, 64, 1, 16), z(1, 2, 16, 16)
    y, w = z(8, 64), z(64)
    calls = (lambda: ssd.ssd_fwd(x, dt, h, h, B, B, h, 64),
             lambda: ssd.ssd_bwd(x, dt, h, h, B, B, h, 64, None, x),
             lambda: ssd.ssd_final_state(x, dt, h, h, B, 64),
             lambda: ssd.ssd_dinit(x, dt, h, h, B, x, 64),
             lambda: ssd.gated_norm_fwd(y, y, w, 64),
             lambda: ssd.gated_norm_bwd(y, y, w, y, 64),
             lambda: ssd.segment_decay(dt, h, h),
             lambda: ssd.state_scan(z(2, 1, 2), torch.stack([s, s]), 0, 0))
    for call in calls:
        call()
    torch.cuda.synchronize()
    before = ssd.launch_count()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 7)
    for call in calls:
        with pytest.raises(ValueError, match="cuda:0.*current device.*cuda:7"):
            call()
    assert ssd.launch_count() == before
