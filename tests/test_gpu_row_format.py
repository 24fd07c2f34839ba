"""The E4M3 row format at its edges: scales so small that a corrected quotient would underflow,
infinite and zero scales, NaN codes. The FP8 dispatch is compared with the oracle bit for bit, the
norm with the fp32 division on the host: its rows have a mean square of exactly 1 and eps is 0,
so v is the weight, or twice the weight, without rounding."""
import numpy as np
import pytest
import torch

import combine_ep_get_05_gb300 as ep
import oracle
from gpu_helpers import dev_bf16, host_bits
from workloads import bf16_bits

pytestmark = pytest.mark.gpu

CODES = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
MIDPOINTS = (CODES[:-1] + CODES[1:]) / 2


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ep.build_library()


def dispatched(bits):
    """Codes and scales of bf16 rows through the FP8 dispatch, every row to one rank in order."""
    T, H = bits.shape
    topk = torch.zeros((T, 1), dtype=torch.int64, device="cuda")
    lay = ep.get_layout(topk, 1, 1)
    d = ep.dispatch(dev_bf16(bits), topk, torch.ones((T, 1), device="cuda"), lay, T, fp8=True)
    return host_bits(d.recv_x[0]), host_bits(d.recv_scales[0])


def quantised_by_oracle(bits):
    rows = [oracle.quantize_row_e4m3(r) for r in bits]
    return np.stack([q for q, _ in rows]), np.stack([s for _, s in rows])


@pytest.mark.parametrize("H", [16384, 16256])  # through shared memory; through registers
def test_fp8_dispatch_rounds_codes_once_where_scales_are_small(H):
    """Every bf16 amax from 2^-119 to 2^-84 in a block with the bf16 value nearest to each midpoint of
    two codes: where the residual of a corrected quotient underflows, the neighbouring code shows."""
    exponents, mantissas = np.meshgrid(np.arange(-119, -84), np.arange(128), indexing="ij")
    amax = ((1 + mantissas / 128) * 2.0 ** exponents).reshape(-1).astype(np.float32)
    scale = amax / np.float32(448.0)
    blocks = np.empty((amax.size, 128), np.float32)
    blocks[:, :126] = torch.from_numpy(MIDPOINTS * scale[:, None].astype(np.float64)).to(torch.bfloat16).float()
    blocks[:, 126] = -amax
    blocks[:, 127] = 0.0
    per = H // 128
    blocks = blocks[:amax.size // per * per]
    bits = bf16_bits(blocks.reshape(-1, H))
    q, s = dispatched(bits)
    want_q, want_s = quantised_by_oracle(bits)
    assert np.array_equal(s, want_s)
    assert np.array_equal(q, want_q)


@pytest.mark.parametrize("H", [1024, 1152])  # through shared memory; through registers
def test_fp8_dispatch_of_infinite_values(H):
    """A block with an infinity has an infinite scale: 0 for its finite values, NaN for infinities."""
    x = np.random.default_rng(41).standard_normal((5, H)).astype(np.float32)
    x[1, 3], x[2, 200], x[2, 201], x[3, H - 1] = np.inf, -np.inf, np.inf, -np.inf
    bits = bf16_bits(x)
    q, s = dispatched(bits)
    with np.errstate(invalid="ignore"):
        want_q, want_s = quantised_by_oracle(bits)
    assert np.isinf(want_s).sum() == 3
    assert np.array_equal(s, want_s)
    nan = (want_q & 0x7F) == 0x7F
    assert nan.sum() == 4 and np.all((q[nan] & 0x7F) == 0x7F)
    assert np.array_equal(q[~nan], want_q[~nan])


def normed(weight, carry, T=3, quarter=False):
    """Codes and scales of v = +-weight, or of v in {0, +-2 weight} (a quarter of the channels is
    2, the others 0), and v itself in fp32."""
    H = weight.size
    rng = np.random.default_rng(42)
    z = np.where(rng.random((T, H)) < 0.5, -1.0, 1.0).astype(np.float32)
    if quarter:
        z *= np.where(np.arange(H) % 4 == 1, 2.0, 0.0).astype(np.float32)
    q = torch.empty((T, H), dtype=torch.uint8, device="cuda")
    s = torch.empty((T, H // 128), device="cuda")
    ep.ep_rmsnorm(None, torch.from_numpy(z).cuda().to(carry), torch.from_numpy(weight).cuda(), 0.0, None, None, q, s)
    with np.errstate(over="ignore", invalid="ignore"):
        v = z * weight
    return host_bits(q), host_bits(s), v


def by_division(v):
    """The stated format: scale = amax / 448, code = e4m3(v / scale), saturated; where the scale is 0
    every value's own code; NaN takes no part in amax (its code stands as 0x7F here)."""
    blocks = v.reshape(v.shape[0], -1, 128)
    with np.errstate(invalid="ignore", over="ignore"):
        s = np.fmax.reduce(np.abs(blocks), axis=2, initial=np.float32(0)) / np.float32(448.0)
        quotient = blocks / np.where(s > 0, s, np.float32(1.0))[:, :, None]
    q = torch.from_numpy(np.clip(quotient, -448.0, 448.0)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    return np.where(np.isnan(quotient), np.uint8(0x7F), q).reshape(v.shape), s


@pytest.mark.parametrize("carry", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("H", [1024, 7168])
def test_norm_of_blocks_that_overflow(carry, H):
    """Products above the largest fp32 number: scale infinity, 0 for the block's finite values."""
    weight = np.random.default_rng(43).uniform(0.5, 1.0, H).astype(np.float32)
    weight[130], weight[133], weight[300], weight[641] = 3e38, 3e38, -3e38, np.inf
    weight[H - 127] = 1e38  # twice that is finite
    q, s, v = normed(weight, carry, quarter=True)
    want_q, want_s = by_division(v)
    assert np.isinf(want_s).any(0).sum() == 2  # channels 133 and 641 are among the quarter, 130 and 300 are not
    assert np.array_equal(s, want_s)
    nan = (want_q & 0x7F) == 0x7F
    assert nan.any() and np.all((q[nan] & 0x7F) == 0x7F)
    assert np.array_equal(q[~nan], want_q[~nan])


@pytest.mark.parametrize("carry", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("H", [1024, 7168])
def test_norm_of_blocks_whose_scale_rounds_to_zero(carry, H):
    """amax up to 224 * 2^-149 over 448 is 0 in fp32: the values' own codes (signed zeros), no
    division by 0; one step above it the scale is 2^-149."""
    rng = np.random.default_rng(44)
    weight = rng.uniform(0.5, 1.0, H).astype(np.float32)
    for b, most in ((1, 1), (2, 224), (4, 225), (5, 2000), (6, 3)):
        steps = rng.integers(0, most + 1, 128)
        steps[::7] = 0
        steps[3] = most
        weight[128 * b:128 * (b + 1)] = np.ldexp(steps.astype(np.float64), -149).astype(np.float32)
    q, s, v = normed(weight, carry)
    want_q, want_s = by_division(v)
    assert np.all(want_s[:, [1, 2, 6]] == 0) and np.all(want_s[:, 4] == np.float32(2.0 ** -149))
    assert np.array_equal(s, want_s)
    assert np.array_equal(q, want_q)


@pytest.mark.parametrize("carry", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H", [(4, 128), (4, 7168), (2000, 256), (1000, 1024)])  # a row per CTA; the ring
def test_norm_writes_one_nan_code(carry, T, H):
    """0xFF for a NaN of either sign; the FP8 dispatch writes 0x7F."""
    weight = np.random.default_rng(45).uniform(0.5, 1.0, H).astype(np.float32)
    weight[5::11], weight[7::11] = np.nan, -np.nan
    q, s, v = normed(weight, carry, T)
    want_q, want_s = by_division(v)
    nan = np.isnan(v)
    assert nan.any() and np.all(q[nan] == 0xFF)
    assert np.array_equal(q[~nan], want_q[~nan]) and np.array_equal(s, want_s)
    bits = np.full((2, 512), 0x3F80, np.uint16)
    bits[0, 3], bits[1, 9] = 0x7FC0, 0xFFC0
    codes, _ = dispatched(bits)
    assert codes[0, 3] == 0x7F and codes[1, 9] == 0x7F
