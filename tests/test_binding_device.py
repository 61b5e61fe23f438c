"""The binding asks for workspace sizes on the device that the call runs on:
the plans behind them depend on that device's SMs. On the CPU, with a stand-in
for torch's device switch and for the library; the tensors are on device 1
while device 0 is current."""
import types

import pytest
import torch

from linear_attention_chunk_gb300 import binding


class FakeTensor:
    """What the binding reads of a CUDA tensor, on device 1."""

    def __init__(self, shape, dtype):
        self.shape, self.dtype, self.device = torch.Size(shape), dtype, torch.device("cuda", 1)

    def get_device(self):
        return 1

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 0x10000

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return self.dtype.itemsize


@pytest.fixture
def calls(monkeypatch):
    """(entry point, current device) of every library call."""
    seen, current = [], [0]

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.before, current[0] = current[0], self.index

        def __exit__(self, *_):
            current[0] = self.before

    class Library:
        def __getattr__(self, name):
            def f(*args):
                seen.append((name, current[0]))
                return 512 if name.endswith("_workspace_size") else binding.GLA_OK
            return f

    cuda = types.SimpleNamespace(current_device=lambda: current[0], device=Device)
    fake = types.SimpleNamespace(
        float32=torch.float32, bfloat16=torch.bfloat16, int32=torch.int32, uint8=torch.uint8, cuda=cuda,
        _C=types.SimpleNamespace(_cuda_getCurrentRawStream=lambda index: 0),
        empty=lambda shape, dtype, device: FakeTensor((shape,) if isinstance(shape, int) else shape, dtype))
    monkeypatch.setattr(binding, "_torch", lambda: fake)
    monkeypatch.setattr(binding, "lib", lambda: Library())
    monkeypatch.setattr(binding, "_entry", {})
    return seen


def bf(*shape):
    return FakeTensor(shape, torch.bfloat16)


def fp(*shape):
    return FakeTensor(shape, torch.float32)


B, T, D, N = 2, 50, 64, 16


def scan(lead):
    return bf(*lead, D), bf(*lead, D), fp(D, N), bf(*lead, N), bf(*lead, N)


CALLS = {
    "gla_ssm_fwd": lambda: binding.gla_ssm_fwd(*scan((B, T))),
    "gla_ssm_varlen": lambda: binding.gla_ssm_varlen(*scan((T,)), FakeTensor((3,), torch.int32), fp(2, D, N)),
    "gla_ssm_bwd": lambda: binding.gla_ssm_bwd(*scan((B, T)), bf(B, T, D)),
    "gla_conv1d_bwd": lambda: binding.gla_conv1d_bwd(bf(B, T, D), fp(D, 4), fp(D), bf(B, T, D)),
    "gla_rmsnorm_bwd": lambda: binding.gla_rmsnorm_bwd(bf(T, D), fp(D), bf(T, D)),
}


@pytest.mark.parametrize("name", CALLS)
def test_the_workspace_is_asked_for_on_the_calls_device(calls, name):
    CALLS[name]()
    assert calls == [(name + "_workspace_size", 1), (name, 1)]
