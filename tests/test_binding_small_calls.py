"""The binding of the drafted trees, pages and the layer norm sets nothing up
where the tensors' device and its current stream are the ones in use, and
switches to the tensors' device everywhere else. On the CPU, with a stand-in
for torch's device switch and for the library."""
import types

import pytest
import torch

from linear_attention_chunk_gb300 import binding
from test_binding_device import FakeTensor, bf, fp


class Tensor(FakeTensor):
    """With what the pages read of a pool as well."""

    @property
    def nbytes(self):
        return self.numel() * self.element_size()


def i32(*shape):
    return Tensor(shape, torch.int32)


@pytest.fixture(params=[0, 1], ids=["another device", "the current device"])
def calls(request, monkeypatch):
    """(entry point, current device, stream) of every library call; the tensors are on device 1."""
    seen, current = [], [request.param]

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
                seen.append((name, current[0]) if name.endswith("_workspace_size") else (name, current[0], args[-1]))
                return 512 if name.endswith("_workspace_size") else binding.GLA_OK
            return f

    cuda = types.SimpleNamespace(current_device=lambda: current[0], device=Device)
    fake = types.SimpleNamespace(
        Tensor=FakeTensor, float32=torch.float32, bfloat16=torch.bfloat16, int32=torch.int32, uint8=torch.uint8,
        bool=torch.bool, cuda=cuda,
        _C=types.SimpleNamespace(_cuda_getDevice=lambda: current[0],
                                 _cuda_getCurrentRawStream=lambda index: 70 + index),
        empty=lambda shape, dtype, device: Tensor((shape,) if isinstance(shape, int) else shape, dtype))
    monkeypatch.setattr(binding, "_torch", lambda: fake)
    monkeypatch.setattr(binding, "lib", lambda: Library())
    monkeypatch.setattr(binding, "_entry", {})
    return seen


T, H, D, N = 6, 2, 64, 3


def trees():
    return i32(N + 1), i32(T)


CALLS = {
    "gla_layernorm_fwd": lambda: binding.gla_layernorm(bf(T, D), fp(D), fp(D), bf(T, D)),
    "gla_layernorm_bwd": lambda: binding.gla_layernorm_bwd(bf(T, D), fp(D), bf(T, D)),
    "gla_tree_fwd": lambda: binding.gla_tree_fwd(bf(T, H, D), bf(T, H, D), bf(T, H, D), fp(H), *trees(), fp(N, H, D, D)),
    "gla_tree_fwd_gated": lambda: binding.gla_tree_fwd_gated(bf(T, H, D), bf(T, H, D), bf(T, H, D), fp(T, H), *trees(),
                                                             fp(N, H, D, D), i32(N)),
    "gla_tree_commit": lambda: binding.gla_tree_commit(bf(T, H, D), bf(T, H, D), fp(H), *trees(), i32(N),
                                                       fp(N, H, D, D), x=bf(T, 48), win_pool=fp(N, 4, 48)),
    "gla_conv1d_tree": lambda: binding.gla_conv1d_tree(bf(T, D), fp(D, 4), fp(D), *trees(), fp(N, 4, D)),
    "gla_pages_copy": lambda: binding.gla_pages_copy([Tensor((N, 8), torch.float32)] * 2, i32(2), i32(2)),
    "gla_pages_clear": lambda: binding.gla_pages_clear(Tensor((N, 8), torch.float32), i32(1)),
    "gla_pages_compact": lambda: binding.gla_pages_compact(Tensor((N, 8), torch.float32), Tensor((N,), torch.bool)),
}


@pytest.mark.parametrize("name", CALLS)
def test_the_call_runs_on_its_tensors_device(calls, name):
    CALLS[name]()
    assert calls[-1] == (name, 1, 71)


def test_the_layer_norms_workspace_is_asked_for_on_its_device(calls):
    CALLS["gla_layernorm_bwd"]()
    assert calls == [("gla_layernorm_bwd_workspace_size", 1), ("gla_layernorm_bwd", 1, 71)]


def test_heads_of_no_width_reach_the_librarys_refusal(calls):
    binding.gla_tree_fwd(bf(T, H, 0), bf(T, H, 0), bf(T, H, D), fp(H), *trees(), fp(N, H, 0, D))
    assert calls[-1][0] == "gla_tree_fwd"
