"""The buffer helpers with `stream`: every allocation and fill happens on that stream, the kernel is
given it, and what is returned is also known to the caller's stream. CPU only: streams are stood in
for, and the entry points only note what they were called with."""
import contextlib
import dataclasses

import pytest
import torch

import combine_ep_get_05_gb300 as ep
from combine_ep_get_05_gb300 import _lib, api

T, H, E, k, R, M = 4, 256, 8, 2, 4, 5


class FakeStream:
    cuda_stream = 7


@pytest.fixture
def world(monkeypatch):
    """Notes [what, stream] of every allocation and entry point, and tensors recorded on another stream."""
    side, now, notes, recorded = FakeStream(), ["callers"], [], []

    @contextlib.contextmanager
    def stream(s):
        now.append(s)
        yield
        now.pop()

    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: now[-1])
    monkeypatch.setattr(torch.cuda, "Stream", FakeStream)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: recorded.append((t.data_ptr(), s)), raising=False)
    for name in ("empty", "zeros", "full", "empty_like", "zeros_like"):
        def made(*a, _f=getattr(torch, name), _n=name, **kw):
            notes.append((_n, now[-1]))
            return _f(*a, **kw)
        monkeypatch.setattr(api.torch, name, made)
    for name in _lib.EXPORTS:
        if hasattr(_lib, name) and "size" not in name:
            monkeypatch.setattr(_lib, name, lambda *a, _n=name: notes.append((_n, a[-1])))
    monkeypatch.setattr(_lib, "ep_layout_workspace_size", lambda *a: 256)
    monkeypatch.setattr(_lib, "ep_expert_layout_workspace_size", lambda *a: 256)
    monkeypatch.setattr(_lib, "ep_rmsnorm_bwd_workspace_size", lambda *a: 256)
    return side, notes, recorded


def calls():
    bf, f32, i32 = (lambda *s: torch.ones(s, dtype=torch.bfloat16)), torch.ones, lambda *s: torch.ones(
        s, dtype=torch.int32)
    idx, w = torch.ones((T, k), dtype=torch.int64), f32(T, k)
    expert = api.ExpertLayout(i32(E + 1), i32(T, k), i32(1), i32(1), E)
    ranks = api.Layout(i32(E), i32(R), None, i32(T, R), None, i32(T, R), i32(1), i32(1), E, R, 0)
    return {
        "get_layout": (api.get_layout, (idx, E, R)),
        "dispatch": (api.dispatch, (bf(T, H), idx, w, ranks, M)),
        "combine": (api.combine, (bf(R, M, H), ranks, M)),
        "rmsnorm": (api.rmsnorm, (bf(T, H), bf(H), 1e-6, f32(T, H), True, True)),
        "rmsnorm_bwd": (api.rmsnorm_bwd, (bf(T, H), f32(T, H), bf(H), 1e-6)),
        "get_expert_layout": (api.get_expert_layout, (idx, E)),
        "dispatch_permuted": (api.dispatch_permuted, (bf(T, H), idx, w, expert, R, M)),
        "dispatch_permuted fp8": (api.dispatch_permuted, (bf(T, H), idx, w, expert, R, M, f32(T, 2))),
        "dispatch_permuted_bwd": (api.dispatch_permuted_bwd, (bf(R, M, H), idx, expert, f32(R, M))),
        "combine_permuted": (api.combine_permuted, (bf(R, M, H), idx, w, expert)),
        "combine_permuted_bwd": (api.combine_permuted_bwd, (bf(T, H), bf(R, M, H), idx, w, expert)),
    }


def tensors(out):
    if isinstance(out, torch.Tensor):
        return [out]
    if dataclasses.is_dataclass(out):
        out = [getattr(out, f.name) for f in dataclasses.fields(out)]
    return [t for t in out if isinstance(t, torch.Tensor)]


@pytest.mark.parametrize("name", sorted(calls()))
def test_allocations_are_on_the_given_stream(world, name):
    side, notes, recorded = world
    helper, args = calls()[name]
    notes.clear(), recorded.clear()
    out = helper(*args, stream=side)
    made = [(n, s) for n, s in notes if not n.startswith("ep_")]
    entries = [(n, s) for n, s in notes if n.startswith("ep_")]
    assert made and all(s is side for _, s in made), made
    assert len(entries) == 1 and entries[0][1] is side
    known = {p for p, s in recorded if s == "callers"}
    inputs = {t.data_ptr() for t in args if isinstance(t, torch.Tensor)}
    assert {t.data_ptr() for t in tensors(out)} - inputs <= known
    assert not known & inputs


@pytest.mark.parametrize("name", sorted(calls()))
def test_without_a_stream_the_current_one_stays(world, name):
    side, notes, recorded = world
    helper, args = calls()[name]
    notes.clear(), recorded.clear()
    helper(*args)
    assert all(s == "callers" for n, s in notes if not n.startswith("ep_"))
    assert [s for n, s in notes if n.startswith("ep_")] == [None] and not recorded
    assert ep.rmsnorm is api.rmsnorm
