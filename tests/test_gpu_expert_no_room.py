"""Slabs without any rows: every row is dropped, and the flag says so."""
import pytest
import torch

import combine_ep_get_05_gb300 as ep
from expert_cases import SENTINEL, Rows, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ep.build_library()


H, F = 64, 128


@pytest.mark.parametrize("counts,R", [([0, 0, 0, 1], 1), ([0, 0, 3, 0], 2), ([2], 1), ([0] * 4, 2), ([0] * 2999 + [1], 8)],
                         ids=["last", "second", "dense", "none", "many"])
def test_rows_without_a_slab_are_dropped_with_the_flag(counts, R):
    rows = Rows(counts, R, 0)
    E, off = rows.E, rows.offsets
    want = ep.FLAG_CAPACITY if sum(counts) else 0

    def z(width, dtype=torch.bfloat16):
        return torch.empty((R, 0, width), dtype=dtype, device="cuda")

    w1, w2 = (torch.zeros(s, dtype=torch.bfloat16, device="cuda") for s in ((E, 2 * F, H), (E, H, F)))
    dw = torch.full((E, F, H), SENTINEL, dtype=torch.bfloat16, device="cuda")
    calls = {
        "gate_up": lambda status: ep.ep_expert_gate_up(z(H), w1, off, 0, z(F), status=status),
        "gate_up 8bit": lambda status: ep.ep_expert_gate_up(z(H), w1, off, 0, z(F), None, z(2 * F, torch.uint8),
                                                            z(2 * F // 128), status),
        "down": lambda status: ep.ep_expert_down(z(F), w2, off, z(H), status),
        "down_bwd": lambda status: ep.ep_expert_down_bwd(z(H), w2, z(2 * F), None, None, off, 0, z(2 * F), None, status),
        "gate_up_bwd": lambda status: ep.ep_expert_gate_up_bwd(z(2 * F), w1, off, z(H), status),
        "wgrad": lambda status: ep.ep_expert_wgrad(z(F), z(H), off, dw, status),
    }
    for name, call in calls.items():
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        call(status)
        assert ep.read_flags(status) == want, name
        call(None)
    assert not dw.any()


def test_a_captured_call_reads_the_offsets_of_its_replay():
    off = torch.zeros(5, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    h, y, w = (torch.empty(s, dtype=torch.bfloat16, device="cuda") for s in ((1, 0, F), (1, 0, H), (4, H, F)))
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        ep.ep_expert_down(h, w, off, y, status)
    g.replay()
    assert ep.read_flags(status) == 0
    off.copy_(torch.tensor([0, 0, 2, 2, 2], dtype=torch.int32))
    g.replay()
    assert ep.read_flags(status) == ep.FLAG_CAPACITY


def test_a_captured_gradient_of_weights_is_cleared_and_reported():
    off = torch.tensor([0, 3], dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    dout, x = (torch.empty((1, 0, n), dtype=torch.bfloat16, device="cuda") for n in (F, H))
    dw = torch.empty((1, F, H), dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        ep.ep_expert_wgrad(dout, x, off, dw, status)
    dw.fill_(SENTINEL)
    g.replay()
    assert not dw.any() and ep.read_flags(status) == ep.FLAG_CAPACITY
