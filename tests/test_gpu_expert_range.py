"""The experts' activations, their gradients and the 8-bit checkpoint over the whole range of bf16: gates far
from zero, outputs near the smallest numbers, quotients beside the midpoints of codes, small scales.

One channel of x, or of dy, selects what a sum is: every other product is zero, so that sums are exact."""
import math

import pytest
import torch

import combine_ep_get_05_gb300 as ep
from expert_cases import ACTS, BF16, Rows, act_of, decode, out

pytestmark = pytest.mark.gpu

# sigmoid: a few 2^-22 from the fast power and reciprocal, and p's own roundings, three of 2^-24 |p| with
# |p| < 110 where the result is no zero: below 2^-15 in all. Half a step of bf16's smallest numbers is 2^-134.
NEAR = BF16 + 2.0 ** -14
SMALLEST = 2.0 ** -134


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ep.build_library()


def bf(values):
    return torch.tensor(values, dtype=torch.float64).to(torch.bfloat16).cuda()


def near(got, want, what):
    got, want = got.double(), want.double()
    assert bool(torch.isfinite(got).all()), (what, got)
    over = (got - want).abs() - (NEAR * want.abs() + SMALLEST)
    i = int(over.argmax())
    assert float(over.max()) <= 0, (what, float(got.flatten()[i]), float(want.flatten()[i]))


FAR = [s * v for v in (0.0, 30.0, 1e4, 1.2e13, 1e15, 1.8e19, 2e19, 1e30, 3e38) for s in (1, -1)]


def gradients(gates, ups, act, eight=None):
    """dgate, dup and h where dh is 1: a row, all of whose channels are given."""
    F = gates.shape[-1]
    rows = Rows([1], 1, 1)
    dy = torch.zeros((1, 1, 8), dtype=torch.bfloat16, device="cuda")
    w = torch.zeros((1, 8, F), dtype=torch.bfloat16, device="cuda")
    dy[0, 0, 0], w[0, 0] = 1.0, 1.0
    dpre, h = out(rows, 2 * F), out(rows, F)
    if eight is None:
        pre, q, s = torch.cat([gates, ups])[None, None].contiguous(), None, None
    else:
        pre, (q, s) = None, eight
    ep.ep_expert_down_bwd(dy, w, pre, q, s, rows.offsets, ACTS[act], dpre, h)
    return dpre[0, 0, :F], dpre[0, 0, F:], h[0, 0]


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gradient_at_gates_far_from_zero(act):
    gates = bf(FAR + [0.0] * (-len(FAR) % 8))
    dgate, dup, h = gradients(gates, torch.ones_like(gates), act)
    v, dv = act_of(act, gates.double())
    near(dgate, dv, "dgate")
    near(dup, v, "dup")
    near(h, v, "h")


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("scale", [2.0 ** 40, 2.0 ** 60, 2.0 ** 118])
def test_gradient_at_gates_far_from_zero_from_the_8_bit_checkpoint(act, scale):
    q = torch.zeros((1, 1, 256), device="cuda")
    q[0, 0, :128] = torch.arange(128, device="cuda") - 64
    q[0, 0, 128:] = 1.0
    q, s = q.to(torch.float8_e4m3fn), bf([[[scale, 1.0]]])
    gates = decode(q, s)[0, 0, :128]
    dgate, dup, h = gradients(gates, None, act, (q, s))
    v, dv = act_of(act, gates)
    near(dgate, dv, "dgate")
    near(dup, v, "dup")
    near(h, v, "h")


def act_below(name, v):
    """The same as act_of, for v far below zero, where 1 + tanh(u) cancels in 64 bits, too: it is 2 sigmoid(2u)."""
    a = 2 * math.sqrt(2 / math.pi)
    p, dp = (v, 1.0) if name == "silu" else (a * (v + 0.044715 * v ** 3), a * (1 + 3 * 0.044715 * v * v))
    s, rest = 1 / (1 + torch.exp(-p)), 1 / (1 + torch.exp(p))
    return v * s, s + v * s * rest * dp


# p(v) from about -80 to -104: the activation falls to bf16's smallest number
LOW = {"silu": [-80 - 0.5 * i for i in range(48)], "gelu": [-9.5 - i / 16 for i in range(24)]}


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("path", ["few", "general", "8bit"])
def test_activation_down_to_the_smallest_numbers(act, path):
    gates = bf(LOW[act])
    n, F = len(gates), 128
    rows = Rows([n], 1, 64 if path == "few" else n)
    x = torch.zeros((1, rows.max_rows, 8), dtype=torch.bfloat16, device="cuda")
    x[0, :n, 0], x[0, :n, 1] = gates, 1.0
    w = torch.zeros((1, 2 * F, 8), dtype=torch.bfloat16, device="cuda")
    w[0, :F, 0], w[0, F:, 1] = 1.0, 1.0
    h = out(rows, F)
    pre = out(rows, 2 * F) if path == "general" else None
    q, s = (out(rows, 2 * F, torch.float8_e4m3fn), out(rows, 2)) if path == "8bit" else (None, None)
    ep.ep_expert_gate_up(x, w, rows.offsets, ACTS[act], h, pre, q, s)
    v, _ = act_below(act, gates.double())
    near(h[0, :n], v[:, None].expand(n, F), "h")


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gradient_down_to_the_smallest_numbers(act):
    gates = bf(LOW[act])
    dgate, dup, h = gradients(gates, torch.ones_like(gates), act)
    v, dv = act_below(act, gates.double())
    near(dup, v, "dup")
    near(h, v, "h")
    near(dgate, dv, "dgate")


def midpoints():
    """Halfway between neighbouring codes from 2^-9 on, ten bits of mantissa and fewer."""
    codes = torch.arange(1, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    return (codes[1:] + codes[:-1]) / 2


def checkpoint_of(scales, nudge, least=0.0):
    """Rows whose blocks have the scales, and values at midpoints times them, plus nudge of that size."""
    m = midpoints()
    m = m[m >= least]
    F, n = 128, len(scales)
    w = torch.zeros((1, 2 * F, 8), dtype=torch.float64)
    w[0, :len(m), 0] = m
    w[0, :len(m), 1] = m
    w[0, F:F + len(m), 0] = -m
    w[0, F:F + len(m), 1] = -m
    w[0, 127, 0], w[0, 255, 0] = 448.0, -448.0
    x = torch.zeros((1, n, 8), dtype=torch.float64)
    x[0, :, 0] = scales
    x[0, :, 1] = scales.sign() * torch.exp2(torch.floor(torch.log2(scales))) * nudge
    assert bool((x == x.to(torch.bfloat16).double()).all()) and bool((w == w.to(torch.bfloat16).double()).all())
    c = torch.einsum("rh,ch->rc", x[0], w[0])
    assert bool((c == c.float().double()).all())
    rows = Rows([n], 1, n)
    h, q, s = out(rows, F), out(rows, 2 * F, torch.float8_e4m3fn), out(rows, 2)
    ep.ep_expert_gate_up(x.to(torch.bfloat16).cuda(), w.to(torch.bfloat16).cuda(), rows.offsets, 0, h, None, q, s)
    return c, q[0].cpu(), s[0].cpu().double()


def codes_of(c, scales):
    """E4M3 of the exact quotients: c has 24 bits and a scale 8, so c / scale is exactly a midpoint or farther
    from it than half a step of fp32, and to round it to fp32 first changes no code."""
    q = c / scales.repeat_interleave(128, dim=1)
    return q.clamp(-448, 448).float().to(torch.float8_e4m3fn)


MANTISSAS = 1.0 + torch.arange(128, dtype=torch.float64) / 128


@pytest.mark.parametrize("exponent", [0, -20, -60, 100])
@pytest.mark.parametrize("nudge", [0.0, 2.0 ** -11, -2.0 ** -11, 2.0 ** -13, -2.0 ** -13, 2.0 ** -15, -2.0 ** -15])
def test_codes_are_rounded_once(nudge, exponent):
    scales = MANTISSAS * 2.0 ** exponent
    c, q, s = checkpoint_of(scales, nudge)
    assert torch.equal(s, scales[:, None].expand(-1, 2))
    assert torch.equal(q.view(torch.uint8), codes_of(c, s).view(torch.uint8))


@pytest.mark.parametrize("exponent", [-92, -101, -116, -117])
@pytest.mark.parametrize("nudge", [0.0, 2.0 ** -8, -2.0 ** -8])
def test_codes_of_small_scales(nudge, exponent):
    """Down to 2^-117, where the smallest code, 2^-9, stands for fp32's smallest normal number."""
    scales = MANTISSAS * 2.0 ** exponent
    c, q, s = checkpoint_of(scales, nudge, least=1.0)
    assert torch.equal(s, scales[:, None].expand(-1, 2))
    assert torch.equal(q.view(torch.uint8), codes_of(c, s).view(torch.uint8))


def test_blocks_below_the_smallest_scale_are_zeros():
    c, q, s = checkpoint_of(MANTISSAS * 2.0 ** -118, 0.0, least=1.0)
    assert not s.any() and not q.float().any()
