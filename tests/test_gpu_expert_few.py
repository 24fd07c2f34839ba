"""The experts' products for few rows: slabs that hold up to 8, 16 or a few more rows an expert, in every
way their kernel takes them, and the bounds between it and the general one."""
import math

import pytest
import torch

import combine_ep_get_05_gb300 as ep
from expert_cases import ACTS, SENTINEL, Rows, check_down, check_gate_up, normal, out, slab
from gpu_helpers import GUARD

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ep.build_library()


def run(x, w1, w2, rows, act, h, y, status=None, stream=None):
    ep.ep_expert_gate_up(x, w1, rows.offsets, ACTS[act], h, status=status, stream=stream)
    ep.ep_expert_down(h, w2, rows.offsets, y, status, stream)


def weights(E, H, F, seed=3):
    return normal(seed, E, 2 * F, H, scale=H ** -0.5), normal(seed + 1, E, H, F, scale=F ** -0.5)


CASES = [
    ([1], 1, 1, 8, 8),
    ([8], 1, 8, 520, 1000),             # one pass of eight rows
    ([7], 1, 9, 4096, 24),              # sixteen at once, seven there
    ([16], 1, 16, 136, 264),
    ([17], 1, 17, 136, 264),            # 32 at once
    ([29, 4], 1, 32, 520, 104),         # dropped rows
    ([50], 1, 64, 264, 48),             # the general kernel
    ([20], 1, 24, 4096, 1032),          # 32 at once; down, heavier: the general kernel
    ([11, 0, 48, 5], 1, 64, 520, 104),  # light: sixteen at once, three passes
    ([65], 1, 65, 136, 264),            # the general kernel
    ([3, 0, 12, 1], 1, 16, 2048, 80),
    ([9, 0, 7], 1, 16, 1032, 200),      # sixteen at once
    ([20, 0, 0, 0], 4, 16, 72, 40),     # dropped rows
    ([0, 0, 0, 0, 0, 0, 0, 64], 8, 64, 264, 48),   # general: 512 rows of room
    ([30, 0, 1, 0, 2, 0, 0, 1], 1, 34, 264, 48),   # several passes of eight
    ([1, 9, 8, 16, 0, 2, 3, 5], 1, 44, 264, 48),   # sixteen at once
    ([0] * 16, 4, 4, 64, 64),
    ([1] * 152 + [2] * 152, 16, 64, 64, 16),       # more units than CTAs, one slice each
    ([2, 0, 1] * 64, 1, 192, 1024, 8),
]


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("counts,R,M,H,F", CASES, ids=[f"E{len(c[0])}R{c[1]}M{c[2]}H{c[3]}F{c[4]}" for c in CASES])
def test_against_64_bits(counts, R, M, H, F, act):
    rows = Rows(counts, R, M)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    x, (w1, w2) = slab(rows, 1, H, 2.0), weights(rows.E, H, F)
    h, y = out(rows, F), out(rows, H)
    run(x, w1, w2, rows, act, h, y, status)
    check_gate_up(x, w1, rows, act, h)
    check_down(h, w2, rows, y)
    assert ep.read_flags(status) == (ep.FLAG_CAPACITY if rows.dropped else 0)


def test_many_experts():
    g = torch.Generator().manual_seed(4)
    counts = (torch.rand(8192, generator=g) < 0.3).int().tolist()
    rows = Rows(counts, 256, 40)
    x, (w1, w2) = slab(rows, 1, 16), weights(8192, 16, 24)
    h, y = out(rows, 24), out(rows, 16)
    run(x, w1, w2, rows, "silu", h, y)
    check_gate_up(x, w1, rows, "silu", h)
    check_down(h, w2, rows, y)


def test_nothing_is_written_outside_the_outputs():
    for counts, R, M in (([5], 1, 5), ([13], 1, 13), ([1, 0, 2, 1], 2, 4)):
        rows = Rows(counts, R, M)
        H, F = 72, 40
        x, (w1, w2) = slab(rows, 1, H), weights(rows.E, H, F)
        backing = [torch.full((R * M * n + 2 * GUARD,), SENTINEL, dtype=torch.bfloat16, device="cuda") for n in (F, H)]
        h, y = (b[GUARD:-GUARD].view(R, M, -1) for b in backing)
        run(x, w1, w2, rows, "gelu", h, y)
        check_gate_up(x, w1, rows, "gelu", h)
        check_down(h, w2, rows, y)
        for b in backing:
            assert bool((b[:GUARD] == SENTINEL).all()) and bool((b[-GUARD:] == SENTINEL).all())


def test_repeated_concurrent_and_replayed_calls():
    """Chained calls repeat bit for bit, on two streams at a time and in a graph whose offsets change."""
    H, F, E, R, M = 1024, 520, 16, 4, 8
    first, second = Rows([1, 0, 1, 0] * 4, R, M), Rows([0, 3, 0, 1] * 4, R, M)
    sets = []
    for i in range(2):
        w1, w2 = weights(E, H, F, seed=20 + i)
        sets.append((normal(i, R, M, H), w1, w2, out(first, F), out(first, H)))

    def calls(s, stream=None):
        x, w1, w2, h, y = s
        ep.ep_expert_gate_up(x, w1, off, 0, h, stream=stream)
        ep.ep_expert_down(h, w2, off, y, stream=stream)

    off = first.offsets.clone()
    want = []
    for s in sets:
        calls(s)
        check_gate_up(s[0], s[1], first, "silu", s[3])
        check_down(s[3], s[2], first, s[4])
        want.append((s[3].clone(), s[4].clone()))
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, stream in zip(sets, streams):
            calls(s, stream)
    torch.cuda.synchronize()
    for s, (h, y) in zip(sets, want):
        assert torch.equal(s[3], h) and torch.equal(s[4], y)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        calls(sets[0])
    off.copy_(second.offsets)
    sets[0][3].fill_(SENTINEL)
    sets[0][4].fill_(SENTINEL)
    g.replay()
    check_gate_up(sets[0][0], sets[0][1], second, "silu", sets[0][3])
    check_down(sets[0][3], sets[0][2], second, sets[0][4])


def test_values_that_are_not_finite_stay_in_their_row():
    rows = Rows([6], 1, 6)
    x, (w1, w2) = slab(rows, 1, 128), weights(1, 128, 64)
    good, y = out(rows, 64), out(rows, 128)
    run(x, w1, w2, rows, "silu", good, y)
    x[0, 2, 9], x[0, 4, 3] = math.nan, math.inf
    h = out(rows, 64)
    run(x, w1, w2, rows, "silu", h, y)
    assert torch.equal(h[0, [0, 1, 3, 5]], good[0, [0, 1, 3, 5]])
    assert bool(h[0, 2].isnan().all()) and not bool(torch.isfinite(h[0, 4]).any())


def test_weights_past_2_31_elements():
    E, H, F = 40, 8192, 3584  # the last expert's weights begin at element 2.3e9
    rows = Rows([0] * 39 + [3], 1, 4)
    w1 = torch.zeros((E, 2 * F, H), dtype=torch.bfloat16, device="cuda")
    w1[39] = normal(2, 2 * F, H, scale=H ** -0.5)
    x, h = slab(rows, 1, H), out(rows, F)
    ep.ep_expert_gate_up(x, w1, rows.offsets, 0, h)
    check_gate_up(x, w1, rows, "silu", h)


@pytest.mark.parametrize("offsets", [[0, 50, 20, 90, 64], [-40, -30, 5, 6, 7], [2 ** 31 - 1, -2 ** 31, 2 ** 31 - 1, 0, 5]])
def test_offsets_that_are_wrong_stay_inside_the_slabs(offsets):
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    x, (w1, _) = normal(1, 2, 8, 64), weights(4, 64, 128)
    g = torch.full((2 * 8 * 128 + 2 * GUARD,), SENTINEL, dtype=torch.bfloat16, device="cuda")
    ep.ep_expert_gate_up(x, w1, off, 0, g[GUARD:-GUARD].view(2, 8, 128))
    assert bool((g[:GUARD] == SENTINEL).all()) and bool((g[-GUARD:] == SENTINEL).all())
