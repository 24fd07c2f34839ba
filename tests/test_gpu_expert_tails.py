"""The gradient of the weights takes an expert's rows as its sums' k: rows behind the last of them, the next
expert's, are in the same copies and have to be cleared, in both CTAs of a pair, before they are multiplied."""
import math

import pytest
import torch

import combine_ep_get_05_gb300 as ep
from expert_cases import SENTINEL, Rows, close, normal, product

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("I,J", [(256, 256), (512, 264), (48, 128)])
def test_rows_of_the_next_expert_are_not_added(I, J):
    """Every second expert's rows are NaN: the others' gradients are finite, right, and the same every time."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ep.build_library()
    E = 300
    counts = [1 + (37 * e) % 130 for e in range(E)]
    rows = Rows(counts, 1, sum(counts))
    dout, x = normal(1, 1, rows.max_rows, I), normal(2, 1, rows.max_rows, J)
    for e, (_, a, b) in enumerate(rows.spans):
        if e % 2:
            dout[0, a:b], x[0, a:b] = math.nan, math.nan
    first = None
    for _ in range(10):
        dw = torch.full((E, I, J), SENTINEL, dtype=torch.bfloat16, device="cuda")
        ep.ep_expert_wgrad(dout, x, rows.offsets, dw)
        if first is None:
            first = dw
        assert torch.equal(dw[::2], first[::2]) and bool(dw[1::2].isnan().all())
    for e, (_, a, b) in enumerate(rows.spans):
        if e % 2 == 0:
            close(first[e], *product(dout[0, a:b].T, x[0, a:b].T), ("dw", e))
