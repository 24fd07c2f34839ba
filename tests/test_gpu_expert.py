"""The experts' feed-forward block against its definition in 64 bits: experts without rows, with one,
around every tile's edge and with many; odd widths; dropped rows; NaN in rows that no expert owns."""
import pytest
import torch

import combine_ep_get_05_gb300 as ep
from expert_cases import (ACTS, SENTINEL, Rows, check_down, check_down_bwd, check_gate_up, check_gate_up_bwd,
                          check_wgrad, decode, normal, out, slab)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ep.build_library()


# counts per expert, ranks, rows of a slab, H, F
SHAPES = [
    ([1], 1, 1, 8, 8),
    ([0, 1, 0, 2], 2, 3, 64, 128),
    ([5, 0, 0, 0], 4, 8, 72, 200),                      # all rows on one expert, three without any
    ([0] * 8, 2, 4, 128, 256),                          # no rows at all
    ([3, 31, 32, 33], 1, 100, 136, 128),
    ([127, 128, 129, 1], 2, 257, 256, 384),
    ([255, 256, 257, 17], 4, 258, 200, 264),
    ([300, 0, 40, 90], 2, 200, 1032, 120),              # the first rank's rows run past its slab
    ([513, 700], 1, 1300, 512, 640),
    ([2, 1, 0, 3] * 16, 16, 9, 1024, 512),              # many experts, few rows
    ([1, 0, 1, 1, 1, 1, 0, 1, 1, 0, 1, 0, 0, 0, 0, 1], 4, 8, 2048, 1024),  # one decoded token
    ([9, 60, 16, 8, 24, 15, 70, 33], 8, 70, 520, 1000),
    ([1500], 1, 1500, 776, 512),                        # a dense layer
]
IDS = [f"E{len(c)}R{r}M{m}H{h}F{f}" for c, r, m, h, f in SHAPES]


def weights(E, H, F, seed=3):
    return normal(seed, E, 2 * F, H, scale=H ** -0.5), normal(seed + 1, E, H, F, scale=F ** -0.5)


def flags(rows, status):
    assert ep.read_flags(status) == (ep.FLAG_CAPACITY if rows.dropped else 0)


def zero_status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("counts,R,M,H,F", SHAPES, ids=IDS)
def test_gate_up(counts, R, M, H, F, act):
    rows, status = Rows(counts, R, M), zero_status()
    x, (w, _) = slab(rows, 1, H, 2.0), weights(rows.E, H, F)
    for save in ("none", "bf16") + (("8bit", "both") if F % 128 == 0 else ()):
        h = out(rows, F)
        pre = out(rows, 2 * F) if save in ("bf16", "both") else None
        q = out(rows, 2 * F, torch.float8_e4m3fn) if save in ("8bit", "both") else None
        scales = out(rows, 2 * F // 128) if save in ("8bit", "both") else None
        ep.ep_expert_gate_up(x, w, rows.offsets, ACTS[act], h, pre, q, scales, status)
        check_gate_up(x, w, rows, act, h, pre, q, scales)
    flags(rows, status)


@pytest.mark.parametrize("counts,R,M,H,F", SHAPES, ids=IDS)
def test_down(counts, R, M, H, F):
    rows, status = Rows(counts, R, M), zero_status()
    h, (_, w), y = slab(rows, 1, F), weights(rows.E, H, F), out(rows, H)
    ep.ep_expert_down(h, w, rows.offsets, y, status)
    check_down(h, w, rows, y)
    flags(rows, status)


def checkpoint(c):
    blocks = c.float().view(*c.shape[:-1], -1, 128)
    s = (blocks.abs().amax(-1) / 448).to(torch.bfloat16)
    return (blocks / s.float()[..., None]).to(torch.float8_e4m3fn).view(c.shape), s


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("counts,R,M,H,F", SHAPES, ids=IDS)
def test_down_bwd(counts, R, M, H, F, act):
    rows, status = Rows(counts, R, M), zero_status()
    dy, (_, w), pre = slab(rows, 1, H, 0.1), weights(rows.E, H, F), slab(rows, 2, 2 * F, 3.0)
    dpre, h = out(rows, 2 * F), out(rows, F)
    ep.ep_expert_down_bwd(dy, w, pre, None, None, rows.offsets, ACTS[act], dpre, h, status)
    check_down_bwd(dy, w, pre, rows, act, dpre, h)
    if F % 128 == 0:
        q, s = checkpoint(pre)
        dpre, h = out(rows, 2 * F), out(rows, F)
        ep.ep_expert_down_bwd(dy, w, None, q, s, rows.offsets, ACTS[act], dpre, h, status)
        check_down_bwd(dy, w, decode(q, s), rows, act, dpre, h)
        again = out(rows, 2 * F)
        ep.ep_expert_down_bwd(dy, w, None, q.view(torch.uint8), s, rows.offsets, ACTS[act], again, None, status)
        assert torch.equal(again, dpre)
    flags(rows, status)


@pytest.mark.parametrize("counts,R,M,H,F", SHAPES, ids=IDS)
def test_gate_up_bwd(counts, R, M, H, F):
    rows, status = Rows(counts, R, M), zero_status()
    dpre, (w, _), dx = slab(rows, 1, 2 * F, 0.1), weights(rows.E, H, F), out(rows, H)
    ep.ep_expert_gate_up_bwd(dpre, w, rows.offsets, dx, status)
    check_gate_up_bwd(dpre, w, rows, dx)
    flags(rows, status)


@pytest.mark.parametrize("counts,R,M,H,F", SHAPES, ids=IDS)
def test_wgrad(counts, R, M, H, F):
    rows, status = Rows(counts, R, M), zero_status()
    for n, m in ((2 * F, H), (H, F)):
        dout, x = slab(rows, 1, n, 0.1), slab(rows, 2, m)
        dw = torch.full((rows.E, n, m), SENTINEL, dtype=torch.bfloat16, device="cuda")
        ep.ep_expert_wgrad(dout, x, rows.offsets, dw, status)
        check_wgrad(dout, x, rows, dw)
    flags(rows, status)


# One round of tiles takes them 32 rows high, then 64, 128 and 256, with as many stages as fit.
@pytest.mark.parametrize("counts", [[40], [1100], [2300], [4600], [5000], [900, 700], [33, 1, 65, 200]],
                         ids=lambda c: "x".join(map(str, c)))
def test_tiles_of_every_height(counts):
    H, F = 1544, 512
    rows, status = Rows(counts, 1, sum(counts) + 3), zero_status()
    (w13, w2), x = weights(rows.E, H, F), slab(rows, 1, H)
    h, q, s = out(rows, F), out(rows, 2 * F, torch.float8_e4m3fn), out(rows, 2 * F // 128)
    ep.ep_expert_gate_up(x, w13, rows.offsets, ACTS["silu"], h, None, q, s, status)
    check_gate_up(x, w13, rows, "silu", h, None, q, s)
    a, y = slab(rows, 2, F), out(rows, H)
    ep.ep_expert_down(a, w2, rows.offsets, y, status)
    check_down(a, w2, rows, y)
    dy, pre, dpre = slab(rows, 3, H, 0.1), slab(rows, 4, 2 * F, 3.0), out(rows, 2 * F)
    ep.ep_expert_down_bwd(dy, w2, pre, None, None, rows.offsets, ACTS["silu"], dpre, None, status)
    check_down_bwd(dy, w2, pre, rows, "silu", dpre)
    d, dx = slab(rows, 5, 2 * F, 0.1), out(rows, H)
    ep.ep_expert_gate_up_bwd(d, w13, rows.offsets, dx, status)
    check_gate_up_bwd(d, w13, rows, dx)
    flags(rows, status)
