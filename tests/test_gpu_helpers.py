"""The buffer helpers in every form of the operators behind them."""
import numpy as np
import pytest
import torch

import combine_ep_get_05_gb300 as ep

pytestmark = pytest.mark.gpu

T, H, E, k, R, M = 70, 264, 8, 3, 2, 210


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ep.build_library()


def rand(shape, seed, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def routing():
    idx = np.random.default_rng(51).permuted(np.tile(np.arange(E), (T, 1)), axis=1)[:, :k].astype(np.int64)
    idx[3, 1] = idx[9, :] = -1
    return torch.from_numpy(np.ascontiguousarray(idx)).cuda()


def test_gradient_of_the_unweighted_return():
    """Rows back without weights: every counted entry's row of dy is dout, and there is no dtopk_w."""
    idx = routing()
    lay = ep.get_expert_layout(idx, E)
    y = rand((R, M, H), 53)
    dout = rand((T, H), 54)
    assert ep.combine_permuted(y, idx, None, lay).shape == (T, H)
    dy, dw = ep.combine_permuted_bwd(dout, y, idx, None, lay)
    assert dw is None
    assert torch.equal(dy, ep.dispatch_permuted(dout, idx, None, lay, R, M).perm_x)  # the sort's adjoint
    weighted, dw = ep.combine_permuted_bwd(dout, y, idx, torch.ones((T, k), device="cuda"), lay)
    assert torch.equal(weighted, dy) and dw.shape == (T, k)
    assert torch.equal(ep.dispatch_permuted_bwd(dy, idx, lay)[0], ep.combine_permuted(dy, idx, None, lay))


@pytest.mark.parametrize("carry", [torch.bfloat16, torch.float32])
def test_norm_of_the_stream_alone(carry):
    """A norm without an addition in front of it (a model's last one): the stream goes in as it is."""
    stream, weight = rand((T, 1024), 55, carry), rand((1024,), 56)
    n = ep.rmsnorm(None, weight, 1e-6, stream, fp8=True)
    assert n.residual is stream
    zero = ep.rmsnorm(torch.zeros((T, 1024), dtype=torch.bfloat16, device="cuda"), weight, 1e-6, stream, fp8=True)
    assert torch.equal(n.y, zero.y) and torch.equal(n.y_scales, zero.y_scales)
    assert torch.equal(n.y_q.view(torch.uint8), zero.y_q.view(torch.uint8))
    with pytest.raises(ValueError, match="x or residual is required"):
        ep.rmsnorm(None, weight, 1e-6)
