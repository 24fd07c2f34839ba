"""What the compiled binding does to the process around a call. A function in C stands for the library's
entry points where the call itself is looked at: nothing is launched then."""
import ctypes
import subprocess
import threading

import pytest
import torch

import combine_ep_get_05_gb300 as ep
from combine_ep_get_05_gb300 import _lib, build
from test_gpu_refusals import arguments

pytestmark = pytest.mark.gpu

STUB = """
#include <stdint.h>
#include <time.h>
volatile int32_t g_go;
int32_t waits(void) { /* up to 2 s for g_go; 0 if it came */
    for (int i = 0; i < 2000 && !g_go; ++i) {
        struct timespec ms = {0, 1000000};
        nanosleep(&ms, 0);
    }
    return !g_go;
}
"""


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ep.build_library()


def test_other_python_threads_run_during_a_call(tmp_path):
    """Every entry point waits for a flag that another Python thread sets."""
    source, library = tmp_path / "stub.c", tmp_path / "stub.so"
    source.write_text(STUB)
    subprocess.run([build.host_compiler(), "-x", "c", "-shared", "-fPIC", str(source), "-o", str(library)], check=True)
    stub = ctypes.CDLL(str(library))
    go = ctypes.c_int32.in_dll(stub, "g_go")
    native = _lib._native()
    calls = arguments()
    real = {f.__name__: ctypes.cast(getattr(_lib.lib(), f.__name__), ctypes.c_void_p).value for f in calls}
    try:
        native.bind({n: ctypes.cast(stub.waits, ctypes.c_void_p).value for n in real})
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
    torch.cuda.synchronize()


INPUTS = {"ep_rmsnorm": {"x", "residual", "weight"}, "ep_rmsnorm_bwd": {"dy", "z", "weight", "dz_in"},
          "ep_dispatch_permuted_fp8": {"x_q", "x_scales", "topk_idx", "topk_w", "expert_offsets", "expert_slot"},
          "ep_dispatch_permuted_fp8_ll": {"x_q", "x_scales", "topk_idx", "topk_w"},
          "ep_dispatch_permuted_bwd": {"dperm_x", "dperm_w", "dx_in", "topk_idx", "expert_offsets", "expert_slot"},
          "ep_combine_permuted_bwd": {"dout", "y", "topk_idx", "topk_w", "expert_offsets", "expert_slot"}}


def test_inputs_that_are_lazy_clones_stay_so():
    """A call only reads its inputs, so none of them gets memory of its own; outputs do."""
    for f, args in arguments().items():
        f(**args)
        cloned = {n: torch._lazy_clone(v) if isinstance(v, torch.Tensor) else v for n, v in args.items()}
        tensors = {n for n, v in cloned.items() if isinstance(v, torch.Tensor)}
        assert all(torch._C._is_cow_tensor(cloned[n]) for n in tensors)
        f(**cloned)
        torch.cuda.synchronize()
        assert {n for n in tensors if torch._C._is_cow_tensor(cloned[n])} == INPUTS[f.__name__]
