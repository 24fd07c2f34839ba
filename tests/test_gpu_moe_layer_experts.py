"""The example layer with its experts' 8-bit checkpoint: it runs, and its gradients are the fp32 layer's up to
the checkpoint's rounding (2^-4 of an element at most, in gate and in up) and those between the operators."""
import os
import sys

import pytest
import torch

import combine_ep_get_05_gb300 as ep

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import moe_layer  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,H,E,k,R", [(64, 256, 8, 2, 2), (200, 512, 16, 4, 4)])
def test_training_step_with_the_8_bit_checkpoint(T, H, E, k, R):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ep.build_library()
    for name, d in moe_layer.train(T, H, E, k, R, save="8bit").items():
        assert d < 0.04 + 2 * 2.0 ** -4, (name, d)
