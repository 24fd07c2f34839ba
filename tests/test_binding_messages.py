"""Refusals of the compiled binding name the argument that they are about. CPU only: tensors without memory."""
import pytest
import torch

import combine_ep_get_05_gb300 as ep


@pytest.fixture(scope="module", autouse=True)
def built():
    ep.build_library()


def test_a_residual_that_is_too_wide_is_named():
    wide = torch.empty((1, 1 << 31), dtype=torch.bfloat16, device="meta")
    with pytest.raises(ValueError, match="^residual is too large"):
        ep.ep_rmsnorm(None, wide, None, 1e-6)
    with pytest.raises(ValueError, match="^x is too large"):
        ep.ep_rmsnorm(wide, None, None, 1e-6)
    with pytest.raises(ValueError, match="^residual must have 2 dimensions, got 3"):
        ep.ep_rmsnorm(None, wide[None], None, 1e-6)
