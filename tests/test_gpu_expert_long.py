"""One expert with as many rows as its slab may have: offsets of rows and sums of them past 2^31 elements."""
import pytest
import torch

import combine_ep_get_05_gb300 as ep
from expert_cases import SENTINEL, act_of, close, normal, product

pytestmark = pytest.mark.gpu

MOST = 2 ** 31 - 512
# rows that are looked at: at both ends, and around 2^30
PLACES = [(0, 300), (2 ** 30 - 200, 2 ** 30 + 200), (MOST - 300, MOST)]


@pytest.fixture(scope="module", autouse=True)
def slabs():
    """Two slabs of 34 GB, the first of zeros but for PLACES."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("less than 80 GB of the GPU are free")
    ep.build_library()
    x = torch.zeros((1, MOST, 8), dtype=torch.bfloat16, device="cuda")
    for i, (a, b) in enumerate(PLACES):
        x[0, a:b] = normal(i + 1, b - a, 8)
    yield x, torch.empty_like(x)
    del x
    torch.cuda.empty_cache()


@pytest.fixture
def offsets():
    return torch.tensor([0, MOST], dtype=torch.int32, device="cuda")


def test_rows(slabs, offsets):
    x, out = slabs
    w = normal(7, 1, 16, 8, scale=0.3)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out.fill_(SENTINEL)
    ep.ep_expert_down(x, w[:, :8].contiguous(), offsets, out, status)
    for a, b in PLACES:
        close(out[0, a:b], *product(x[0, a:b], w[0, :8]), ("y", a))
    assert not out[0, 300:10 ** 6].any() and not out[0, MOST - 10 ** 6:MOST - 300].any()
    out.fill_(SENTINEL)
    ep.ep_expert_gate_up(x, w, offsets, ep.ACT_SILU, out, status=status)
    for a, b in PLACES:
        c, err = product(x[0, a:b], w[0])
        v, _ = act_of("silu", c[:, :8])
        # slopes below 1.13, and 2^-18 of the fast power and reciprocal
        bound = (1.01 * (1.13 * err[:, :8] * c[:, 8:].abs() + v.abs() * err[:, 8:]) + 1.13 * err[:, :8] * err[:, 8:]
                 + 2.0 ** -18 * (c[:, :8] * c[:, 8:]).abs())
        close(out[0, a:b], v * c[:, 8:], bound, ("h", a))
    assert not out[0, 300:10 ** 6].any() and not out[0, MOST - 10 ** 6:MOST - 300].any()
    assert ep.read_flags(status) == 0


def test_weights_gradient_of_one_long_tile(slabs, offsets):
    """One tile, whose finishing warps wait several seconds for its sums: no wait gives up while stages are
    filled. Rows that are zero in one operand add nothing."""
    x, out = slabs
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out.zero_()
    for i, (a, b) in enumerate(PLACES):
        out[0, a + 7:b] = normal(i + 11, b - a - 7, 8)
    dw = torch.full((1, 8, 8), SENTINEL, dtype=torch.bfloat16, device="cuda")
    ep.ep_expert_wgrad(out, x, offsets, dw, status)
    d, v = (torch.cat([t[0, a:b] for a, b in PLACES]) for t in (out, x))
    close(dw[0], *product(d.T, v.T), "dw")
    assert ep.read_flags(status) == 0
