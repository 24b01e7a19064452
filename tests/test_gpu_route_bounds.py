"""GPU: expert routing at the edges of its error bounds -- sums that round one
way, choices closer than their errors, rows beside padded ones."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import route as oracle_route

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from wide_bf16_row_gb300 import build
    build.build()


@pytest.mark.parametrize("tokens", [70, 1301])
@pytest.mark.parametrize("with_bias", [True, False])
@pytest.mark.parametrize("experts,step", [(256, 4), (256, 8), (128, 4), (96, 3), (1024, 32)])
def test_a_softmax_sum_that_rounds_one_way(tokens, with_bias, experts, step):
    """Four experts at logit 0, the others' exponentials a little over half a unit of 1: every addition to a sum of 1
    rounds up.  The bound that the choice counts on: 50 u of the score (a sum of at most 36 u, exp2, the rounded
    exponent of a logit of 0, a reciprocal, a product)."""
    import torch

    from wide_bf16_row_gb300 import topk
    x = torch.full((tokens, experts), float(np.log(0.505 * 2.0 ** -23)))
    lead = torch.arange(4) * step
    x[:, lead] = 0
    bias = torch.zeros(experts) if with_bias else None
    idx, weight = topk.route_experts(x.cuda(), 4, bias=None if bias is None else bias.cuda(), renormalize=False)
    assert torch.equal(idx.cpu(), lead.int().expand(tokens, 4))
    p = np.exp(x[0].double().numpy())
    assert (np.abs(weight.double().cpu().numpy() * p.sum() - 1) <= 50 * U).all()
