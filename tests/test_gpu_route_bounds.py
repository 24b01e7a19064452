"""GPU: expert routing at the edges of its error bounds -- sums that round one
way, choices closer than their errors, rows beside padded ones."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import route as oracle_route

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
# four lanes per token take over at 40 tokens per SM at the latest
MANY = 6505


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from wide_bf16_row_gb300 import build
    build.build()


@pytest.mark.parametrize("tokens", [70, 1301, MANY])
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


@pytest.mark.parametrize("k", [1, 2, 3, 4, 5, 6])
def test_a_near_tie_behind_the_next_choice(k):
    """The k-th choice and the one behind it are small scores with large biases and known to 2 u; the one behind that
    is a score of nearly 1, known less well, and in truth before both: its softmax sum rounds one way (as above), so
    that in 32 bits it comes out 13 u too low."""
    import torch

    from wide_bf16_row_gb300 import topk
    x = torch.full((MANY, 256), float(np.log(0.55 * 2.0 ** -23)))
    x[:, 0] = 0
    p = np.exp(x[0].double().numpy())
    p /= p.sum()
    bias = torch.full((256,), -10.0)
    bias[10:10 * k:10] = torch.arange(k, 1, -1).float()
    bias[10 * k] = 1.0
    bias[100] = 1.0 - 5 * U
    bias[0] = 1.0 + p[100] + 1e-8 - p[0]
    idx, _ = topk.route_experts(x.cuda(), k, bias=bias.cuda())
    expected, _, _ = oracle_route.route(x[:1].numpy(), k, bias.numpy())
    assert expected[0, k - 1] == 0
    assert np.array_equal(idx.cpu().numpy(), np.repeat(expected, MANY, 0))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("k", [3, 8, 12])
def test_a_token_does_not_see_its_neighbours(score, k):
    """Weights and gradients of a token are the same bits alone, beside tokens without experts and beside tokens whose
    scores underflow."""
    import torch

    from wide_bf16_row_gb300 import topk
    g = torch.Generator().manual_seed(k)
    tokens, experts = 64, 40
    x = torch.randn(tokens, experts, generator=g)
    grad = torch.randn(tokens, k, generator=g)
    how = {"score": score, "scale": 2.5}
    idx, weight = topk.route_experts(x.cuda(), k, **how)
    d = topk.route_experts_grad(x.cuda(), idx, grad.cuda(), **how)
    for other in (-float("inf"), -120.0):
        mixed = torch.full((4 * tokens, experts), other)
        mixed[::4] = x
        grads = torch.ones(4 * tokens, k)
        grads[::4] = grad
        idx2, weight2 = topk.route_experts(mixed.cuda(), k, **how)
        d2 = topk.route_experts_grad(mixed.cuda(), idx2, grads.cuda(), **how)
        assert torch.equal(idx2[::4], idx) and torch.equal(weight2[::4], weight) and torch.equal(d2[::4], d)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
def test_nothing_flows_to_experts_out_of_reach(score, renorm, bad):
    """A gradient that overflowed stays with the experts that have a part in the weights: logits of -inf and NaN get 0,
    and the other tokens what they get without it."""
    import torch

    from wide_bf16_row_gb300 import topk
    g = torch.Generator().manual_seed(2)
    x = torch.randn(50, 40, generator=g)
    x[:, 3::5] = -float("inf")
    x[:, 4::7] = float("nan")
    how = {"score": score, "renormalize": renorm}
    idx, _ = topk.route_experts(x.cuda(), 4, **how)
    grad = torch.randn(50, 4, generator=g).cuda()
    want = topk.route_experts_grad(x.cuda(), idx, grad, **how)
    grad[::3, 1] = bad
    d = topk.route_experts_grad(x.cuda(), idx, grad, **how)
    assert (d.cpu()[~(x > -float("inf"))] == 0).all()
    rest = torch.arange(50) % 3 != 0
    assert torch.equal(d[rest], want[rest])
    assert not torch.isfinite(d[::3]).all()


def test_heavy_near_ties_left_out():
    """More than 32 candidates, eight of them one choice eight times over, and one that in 32 bits falls just below
    them, at the border of a short key, and in truth lies above: its score times the inverse sum, rounded or not
    before the bias is added, gives one key or the other."""
    import torch

    from wide_bf16_row_gb300 import topk
    for shift in range(12):
        x = torch.full((1301, 256), float(np.log(0.55 * 2.0 ** -23)))
        x[:, 0] = 0
        x[:, 1] = float(np.float32(-0.3 - 0.01 * shift)) + torch.arange(-650, 651) * 2.0 ** -25
        x[:, 200:240] = -40
        p = np.exp(x[650].double().numpy())
        p /= p.sum()
        bias = torch.full((256,), -10.0)
        bias[200:208] = 0.75
        bias[208:240] = 0.75 - 2e-6 - 2e-7 * torch.arange(32)
        bias[1] = 0.75 - p[1]
        idx, _ = topk.route_experts(x.repeat(5, 1).cuda(), 8, bias=bias.cuda())
        expected = np.tile(oracle_route.route(x.numpy(), 8, bias.numpy())[0], (5, 1))
        bad = np.flatnonzero((idx.cpu().numpy() != expected).any(1))
        assert not len(bad), (shift, bad[:5], idx[int(bad[0])], expected[bad[0]])


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("experts,groups,kept,k,best,with_bias", [
    (256, 8, 4, 8, 2, True), (256, 16, 15, 8, 1, False), (240, 5, 2, 1, 2, True), (255, 1, 1, 8, 2, True),
    (256, 1, 1, 7, 2, False), (128, 8, 3, 7, 2, False), (126, 2, 1, 8, 2, True), (100, 4, 3, 1, 1, True),
    (91, 7, 6, 6, 2, False), (64, 4, 2, 6, 2, True), (61, 1, 1, 5, 2, True), (32, 2, 1, 3, 1, True),
    (22, 2, 1, 8, 2, True), (15, 15, 7, 8, 2, False), (4, 2, 1, 8, 2, True), (1, 1, 1, 1, 2, True)])
def test_many_tokens_in_every_layout(dtype, score, experts, groups, kept, k, best, with_bias):
    """Enough tokens that four lanes take each, with a bias and groups too: 271 rows -- masked experts, empty rows,
    coarse ones with ties, equal ones -- 24 times over and one row more, against the 64-bit oracle."""
    import torch

    from wide_bf16_row_gb300 import topk
    g = torch.Generator().manual_seed(experts + k)
    x = 1.5 * torch.randn(271, experts, generator=g)
    x[torch.rand(271, experts, generator=g) < 0.1] = -float("inf")
    x[torch.rand(271, experts, generator=g) < 0.02] = float("nan")
    x[::11] = -float("inf")
    x[5::7] = (x[5::7] * 2).round() / 2
    x[6::7] = 0.5
    x = x.to({"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[dtype])
    bias = 0.1 * torch.randn(experts, generator=g) if with_bias else None
    many = torch.cat([x.repeat(24, 1), x[:1]])
    load = torch.zeros(experts, dtype=torch.int32, device="cuda")
    idx, weight = topk.route_experts(many.cuda(), k, bias=None if bias is None else bias.cuda(), score=score, groups=groups,
                                     groups_kept=kept, group_best=best, scale=1.5, load=load)
    ref_idx, ref_weight, _ = oracle_route.route(x.float().numpy(), k, None if bias is None else bias.numpy(), score, groups,
                                                kept, best, True, 1.5)
    ref_idx, ref_weight = (np.concatenate([np.tile(r, (24, 1)), r[:1]]) for r in (ref_idx, ref_weight))
    assert np.array_equal(idx.cpu().numpy(), ref_idx)
    np.testing.assert_allclose(weight.cpu().numpy(), ref_weight, rtol=1e-5, atol=1e-37)
    assert np.array_equal(load.cpu().numpy(), np.bincount(ref_idx[ref_idx >= 0], minlength=experts))


@pytest.mark.parametrize("tokens", [70, MANY])
@pytest.mark.parametrize("with_bias", [True, False])
def test_small_softmax_scores_are_within_their_bound(tokens, with_bias):
    """Scores down to exp(-86), whose exponents' roundings count: 253 u of the score, which the choice allows for."""
    import torch

    from wide_bf16_row_gb300 import topk
    g = torch.Generator().manual_seed(7)
    x = -86 * torch.rand(tokens, 8, generator=g)
    x[:, 0] = 0
    bias = torch.zeros(8, device="cuda") if with_bias else None
    idx, weight = topk.route_experts(x.cuda(), 8, bias=bias, renormalize=False)
    p = torch.softmax(x.double(), 1).gather(1, idx.cpu().long())
    assert ((weight.cpu().double() / p - 1).abs() <= 253 * U).all()
    assert torch.equal(idx.cpu(), x.sort(dim=1, descending=True, stable=True).indices.int())
