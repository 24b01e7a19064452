"""The operators together, as a drafter with a mixture layer uses them.

A training step: router logits -> route_experts -> the chosen experts' products
(torch) -> head_loss_bf16 -> head_loss_grad_bf16 -> the routing weights'
gradient -> route_experts_grad.  Everything is checked against 64 bits from the
same hidden states; the bound of the router's gradient is the head gradient's
bound (see test_gpu_head_loss) carried through the linear steps in between.

Serving: head_topk_bf16 picks the draft tokens, head_loss_bf16 gives their
log-probabilities."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import head_loss as oracle_loss
from oracle import route as oracle_route
from tests.test_gpu_head_loss import HALF, check_grad, check_loss, logit_error
from tests.test_gpu_route import RTOL

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from wide_bf16_row_gb300 import build
    build.build()


@pytest.mark.parametrize("score,renorm,groups,kept", [("sigmoid", True, 4, 2), ("softmax", True, 1, 1),
                                                      ("softmax", False, 1, 1)])
def test_training_step_of_a_mixture_drafter(score, renorm, groups, kept):
    import torch

    from wide_bf16_row_gb300 import topk
    rows, dim, vocab, experts, k = 300, 64, 1500, 16, 4
    gen = torch.Generator().manual_seed(5)
    x = torch.randn(rows, dim, generator=gen).cuda()
    router = (torch.randn(experts, dim, generator=gen) / 8).cuda()
    expert = (torch.randn(experts, dim, dim, generator=gen) / 8).cuda()
    head = (torch.randn(vocab, dim, generator=gen) / 4).bfloat16().cuda()
    bias = (torch.randn(experts, generator=gen) / 10).cuda()
    target = torch.randint(0, vocab, (rows,), generator=gen).cuda()
    target[::4] = -100
    how = dict(score=score, renormalize=renorm, scale=1.5)

    logits = x @ router.T
    load = torch.zeros(experts, dtype=torch.int32, device="cuda")
    idx, weight = topk.route_experts(logits, k, bias=bias, groups=groups, groups_kept=kept, load=load, **how)
    each = torch.stack([torch.einsum("nd,nde->ne", x, expert[idx[:, i].long()]) for i in range(k)], 1)  # [rows, k, dim]
    hidden = (x + (weight[:, :, None] * each).sum(1)).bfloat16()
    loss, lse = topk.head_loss_bf16(hidden, head, target)
    valid = (target != -100).float()
    g = valid / valid.sum()
    d_hidden, d_head = topk.head_loss_grad_bf16(hidden, head, target, lse, g)
    d_weight = (d_hidden.float()[:, None, :] * each).sum(2)
    d_logits = topk.route_experts_grad(logits, idx, d_weight, **how)
    d_router = d_logits.T @ x

    def np64(t):
        return t.detach().double().cpu().numpy()

    ref_idx, ref_weight, ref_load = oracle_route.route(np64(logits), k, np64(bias), score, groups, kept, 2, renorm, 1.5)
    assert np.array_equal(idx.cpu().numpy(), ref_idx) and np.array_equal(load.cpu().numpy(), ref_load)
    np.testing.assert_allclose(np64(weight), ref_weight, rtol=RTOL)
    check_loss(hidden, head, target, loss, lse)
    check_grad(hidden, head, target, g, d_hidden, d_head)
    # the router's gradient from 64 bits, and how far the head's roundings may carry
    h, w, t = np64(hidden), np64(head), target.cpu().numpy()
    ref_h, _, G = oracle_loss.grad(h, w, t, np64(g))
    hot = np.zeros_like(G)
    hot[np.flatnonzero(t >= 0), t[t >= 0]] = 1
    entry = HALF * np.abs(G) + (2 * logit_error(h, w) + 1e-5)[:, None] * np.abs(G + hot * np64(g)[:, None])
    allow_h = entry @ np.abs(w) + (vocab / 16 + 34) * 2.0 ** -23 * (np.abs(G) @ np.abs(w)) + HALF * np.abs(ref_h)
    e = np64(each)
    ref_dw = (ref_h[:, None, :] * e).sum(2)
    # dim products and sums in fp32 beside it
    allow_dw = (allow_h[:, None, :] * np.abs(e)).sum(2) + dim * 2.0 ** -24 * (np.abs(ref_h[:, None, :]) * np.abs(e)).sum(2)
    ref_d, size = oracle_route.grad(np64(logits), ref_idx, ref_dw, score, renorm, 1.5)
    _, carried = oracle_route.grad(np64(logits), ref_idx, allow_dw, score, renorm, 1.5)
    off = np.abs(np64(d_logits) - ref_d)
    assert (off <= carried + 2 * RTOL * (size + carried) + 2.0 ** -24 * np.abs(ref_d) + 1e-30).all()
    assert d_router.shape == router.shape and torch.isfinite(d_router).all()
    assert not torch.any(d_logits[::4] != 0)  # ignored rows reach no router


def test_drafts_and_their_log_probabilities():
    """The best token of head_topk_bf16 scored by head_loss_bf16: lse - loss is
    its logit, whose bf16 rounding the selection reported."""
    import torch

    from wide_bf16_row_gb300 import topk
    gen = torch.Generator().manual_seed(6)
    hidden = torch.randn(15, 256, generator=gen).bfloat16().cuda()
    head = (torch.randn(5000, 256, generator=gen) / 16).bfloat16().cuda()
    idx, val, count, mask = topk.head_topk_bf16(hidden, head, 4)
    prob, keep = topk.nucleus_bf16(val, count, 1.0, 1.0)
    scores = []
    for i in range(4):
        loss, lse = topk.head_loss_bf16(hidden, head, idx[:, i].contiguous())
        logit = (lse - loss).double()
        v = val[:, i].double()
        slack = 2 * float(logit_error(hidden.double().cpu().numpy(), head.double().cpu().numpy()).max()) + 2e-5
        assert ((logit - v).abs() <= HALF * v.abs() + slack).all()
        scores.append(-loss)
    # the nucleus over these four is their softmax: the lse cancels
    ours = torch.softmax(torch.stack(scores, 1).double(), 1)
    step = float(HALF * val.double().abs().max()) + slack  # both logits of a ratio off by this much
    assert ((ours - prob.double()).abs() <= 2 * step).all()


def test_two_streams_at_once():
    """Calls in flight on two streams, each with workspaces of its own, leave one another alone."""
    import torch

    from wide_bf16_row_gb300 import topk
    gen = torch.Generator().manual_seed(7)
    sets = []
    for rows in (300, 520):
        hidden = torch.randn(rows, 256, generator=gen).bfloat16().cuda()
        head = (torch.randn(9000, 256, generator=gen) / 16).bfloat16().cuda()
        target = torch.randint(0, 9000, (rows,), generator=gen).cuda()
        g = torch.rand(rows, generator=gen).cuda()
        logits = torch.randn(rows * 10, 64, generator=gen).cuda()
        sets.append((hidden, head, target, g, logits))

    def all_of(hidden, head, target, g, logits, stream=None):
        loss, lse = topk.head_loss_bf16(hidden, head, target, stream=stream)
        dh, dw = topk.head_loss_grad_bf16(hidden, head, target, lse, g, stream=stream)
        idx, weight = topk.route_experts(logits, 6, score="sigmoid", groups=4, groups_kept=2, stream=stream)
        return loss, lse, dh, dw, idx, weight

    want = [all_of(*s) for s in sets]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for _ in range(4):
        for i in (0, 1):
            got[i].append(all_of(*sets[i], stream=streams[i]))
    for s in streams:
        s.synchronize()
    for i in (0, 1):
        for run in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(run, want[i]))
    assert topk.device_fault() == 0
