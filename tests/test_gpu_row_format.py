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
