"""The compiled binding around the experts' products: tensors of another device are refused, inputs are only
read, other Python threads run during a call, errors of the library are raised."""
import ctypes
import subprocess
import threading

import pytest
import torch

import combine_ep_get_05_gb300 as ep
from combine_ep_get_05_gb300 import _lib, build
from test_devices import on_second
from test_gpu_binding import STUB

pytestmark = pytest.mark.gpu

R, M, E, H, F = 2, 24, 4, 64, 128


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ep.build_library()


def arguments():
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    off = torch.tensor([0, 3, 3, 20, 24], dtype=torch.int32, device="cuda")
    q = lambda: torch.zeros((R, M, 2 * F), dtype=torch.float8_e4m3fn, device="cuda")  # noqa: E731
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    return {
        ep.ep_expert_gate_up: dict(x=z(R, M, H), w_gate_up=z(E, 2 * F, H), expert_offsets=off, act=0, h=z(R, M, F),
                                   pre=z(R, M, 2 * F), pre_q=q(), pre_scales=z(R, M, 2 * F // 128), status=status),
        ep.ep_expert_down: dict(h=z(R, M, F), w_down=z(E, H, F), expert_offsets=off, y=z(R, M, H), status=status),
        ep.ep_expert_down_bwd: dict(dy=z(R, M, H), w_down=z(E, H, F), pre=None, pre_q=q(),
                                    pre_scales=z(R, M, 2 * F // 128), expert_offsets=off, act=1, dpre=z(R, M, 2 * F),
                                    h=z(R, M, F), status=status),
        ep.ep_expert_gate_up_bwd: dict(dpre=z(R, M, 2 * F), w_gate_up=z(E, 2 * F, H), expert_offsets=off,
                                       dx=z(R, M, H), status=status),
        ep.ep_expert_wgrad: dict(dout=z(R, M, 2 * F), rows=z(R, M, H), expert_offsets=off, dw=z(E, 2 * F, H),
                                 status=status),
    }


INPUTS = {"ep_expert_gate_up": {"x", "w_gate_up", "expert_offsets"}, "ep_expert_down": {"h", "w_down", "expert_offsets"},
          "ep_expert_down_bwd": {"dy", "w_down", "pre_q", "pre_scales", "expert_offsets"},
          "ep_expert_gate_up_bwd": {"dpre", "w_gate_up", "expert_offsets"},
          "ep_expert_wgrad": {"dout", "rows", "expert_offsets"}}


def test_tensors_of_another_device_are_refused():
    for f, base in arguments().items():
        for name, t in base.items():
            if isinstance(t, torch.Tensor):
                with pytest.raises(ValueError, match=f"{name} must be on the current device, cuda:0, got cuda:1"):
                    f(**{**base, name: on_second(t)})
        f(**base)
    torch.cuda.synchronize()


def test_inputs_that_are_lazy_clones_stay_so():
    for f, args in arguments().items():
        f(**args)
        cloned = {n: torch._lazy_clone(v) if isinstance(v, torch.Tensor) else v for n, v in args.items()}
        tensors = {n for n, v in cloned.items() if isinstance(v, torch.Tensor)}
        f(**cloned)
        torch.cuda.synchronize()
        assert {n for n in tensors if torch._C._is_cow_tensor(cloned[n])} == INPUTS[f.__name__]


def test_other_python_threads_run_during_a_call(tmp_path):
    source, library = tmp_path / "stub.c", tmp_path / "stub.so"
    source.write_text(STUB)
    subprocess.run([build.host_compiler(), "-x", "c", "-shared", "-fPIC", str(source), "-o", str(library)], check=True)
    stub = ctypes.CDLL(str(library))
    go = ctypes.c_int32.in_dll(stub, "g_go")
    native = _lib._native()
    calls = arguments()
    real = {f.__name__: ctypes.cast(getattr(_lib.lib(), f.__name__), ctypes.c_void_p).value for f in calls}
    try:
        native.bind({n: ctypes.cast(stub.waits, ctypes.c_void_p).value for n in real})  # the others stay bound
        for f, args in calls.items():
            go.value = 0
            setter = threading.Timer(0.02, lambda: setattr(go, "value", 1))
            setter.start()
            f(**args)  # raises EpError where the flag was not seen
            setter.join()
    finally:
        native.bind(real)
    for f, args in calls.items():
        f(**args)
    ep.ep_rmsnorm(torch.ones((2, 64), dtype=torch.bfloat16, device="cuda"), None,
                  torch.ones(64, device="cuda"), 1e-6, None, torch.empty((2, 64), dtype=torch.bfloat16, device="cuda"))
    torch.cuda.synchronize()


def test_two_host_threads_at_once():
    """Calls of two host threads, each on a stream of its own, as in one."""
    def results(stream):
        torch.cuda.set_device(0)
        with torch.cuda.stream(stream):
            g = torch.Generator(device="cuda").manual_seed(3)
            x, w = (torch.randn(s, generator=g, device="cuda").to(torch.bfloat16) for s in ((R, M, H), (E, 2 * F, H)))
            off = torch.tensor([0, 3, 3, 20, 24], dtype=torch.int32, device="cuda")
            for _ in range(50):
                h = torch.zeros((R, M, F), dtype=torch.bfloat16, device="cuda")
                dw = torch.empty((E, F, H), dtype=torch.bfloat16, device="cuda")
                ep.ep_expert_gate_up(x, w, off, 0, h)
                ep.ep_expert_wgrad(h, x, off, dw)
            stream.synchronize()
            return h, dw

    want = results(torch.cuda.Stream())
    got = [None, None]
    streams = [torch.cuda.Stream() for _ in got]

    def worker(i):
        got[i] = results(streams[i])

    threads = [threading.Thread(target=worker, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for g in got:
        assert torch.equal(g[0], want[0]) and torch.equal(g[1], want[1])
