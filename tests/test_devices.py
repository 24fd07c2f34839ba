"""Tensors of another device than the current one are refused before anything is launched with their
addresses. A tensor without memory stands for one on a second GPU, so one GPU is enough, or none for
the functions whose checks are in Python."""
import pytest
import torch

import combine_ep_get_05_gb300 as ep
from combine_ep_get_05_gb300 import _lib

T, H, k, E, R, M = 4, 256, 2, 8, 4, 5


class OnSecond(torch.Tensor):
    @staticmethod
    def __new__(cls, t):
        return torch.Tensor._make_wrapper_subclass(cls, t.shape, dtype=t.dtype, device=torch.device("cuda:1"))

    @classmethod
    def __torch_dispatch__(cls, func, types, args=(), kwargs=None):
        raise NotImplementedError(func)


def on_second(t):
    return OnSecond(t)


@pytest.fixture
def first_of_two(monkeypatch):
    monkeypatch.setattr(_lib, "_only_device", False)
    monkeypatch.setattr(torch.cuda, "device_count", lambda: 2)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)


def test_check_refuses_a_tensor_of_another_device(first_of_two):
    t = on_second(torch.empty((T, H), dtype=torch.bfloat16))
    for shape in (None, (T, H), (T, 1)):
        with pytest.raises(ValueError, match="y must be on the current device, cuda:0, got cuda:1"):
            _lib._check("y", t, torch.bfloat16, shape)
    with pytest.raises(ValueError, match="y must be on the current device"):
        ep.ep_combine(on_second(torch.empty((R, M, H), dtype=torch.bfloat16)), torch.empty((T, R), dtype=torch.int32), M, None)


def test_check_accepts_the_current_device(first_of_two, monkeypatch):
    t = on_second(torch.empty((T, H), dtype=torch.bfloat16))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    _lib._check("y", t, torch.bfloat16, (T, H))
    assert not _lib._only_device
    monkeypatch.setattr(torch.cuda, "device_count", lambda: 1)
    _lib._check("y", t, torch.bfloat16, (T, H))
    assert _lib._only_device


@pytest.mark.gpu
def test_binding_refuses_tensors_of_another_device():
    from test_gpu_refusals import arguments

    ep.build_library()
    for f, base in arguments().items():
        for name, t in base.items():
            if isinstance(t, torch.Tensor):
                with pytest.raises(ValueError, match=f"{name} must be on the current device, cuda:0, got cuda:1"):
                    f(**{**base, name: on_second(t)})
        f(**base)
    torch.cuda.synchronize()
