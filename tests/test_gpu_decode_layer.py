"""The operators of a decode step in a row, as a user calls them: routing,
order by expert, rows in 8 bits, the experts' products, the tokens' sums, the
head's product in 8 bits, penalties, top-k and top-p; checked against the
oracles, each on what the step before gave."""
from __future__ import annotations

import numpy as np
import pytest

import oracle as topk_oracle
from oracle import penalty as oracle_penalty
from oracle import route as oracle_route
from oracle import tokens as oracle

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from wide_bf16_row_gb300 import build
    build.build()


def _np(x):
    return x.double().cpu().numpy()


def _eight(shape, g):
    import torch
    w = (80 * torch.randn(*shape, generator=g)).clamp(-448, 448).to(torch.float8_e4m3fn).cuda()
    lead, (rows, dim) = shape[:-2], shape[-2:]
    return w, (torch.rand(*lead, -(-rows // 128), -(-dim // 128), generator=g) + 0.5).cuda() * (0.01 * dim ** -0.5)


def products_near(y, ref, size, blocks):
    allow = 2.0 ** -8 * np.abs(ref) + (265 + blocks) * U * 1.01 * size + 1e-38
    assert (np.abs(_np(y) - ref) <= allow).all()


@pytest.mark.parametrize("tokens", [1, 5, 300])
def test_a_decode_step(tokens):
    import torch

    from wide_bf16_row_gb300 import topk
    dim, inner, experts, k, vocab = 256, 272, 16, 4, 5003
    g = torch.Generator().manual_seed(tokens)
    x = torch.randn(tokens, dim, generator=g).bfloat16().cuda()
    router = torch.randn(tokens, experts, generator=g).cuda()
    up, up_scale = _eight((experts, inner, dim), g)
    down, down_scale = _eight((experts, dim, inner), g)
    head, head_scale = _eight((vocab, dim), g)
    said = torch.randint(0, vocab, (tokens, 50), generator=g, dtype=torch.int32).cuda()
    repetition = torch.full((tokens,), 1.3, device="cuda")

    def step():
        idx, weight = topk.route_experts(router, k, score="sigmoid")
        order = topk.sort_by_expert(idx, experts)
        q, s = topk.quantize_tokens_fp8(x, order)
        mid = topk.product_fp8(q, s, up, up_scale, offsets=order.offsets)
        q2, s2 = topk.quantize_tokens_fp8(mid)
        rows = topk.product_fp8(q2, s2, down, down_scale, offsets=order.offsets)
        hidden = topk.combine_tokens(rows, order, weight)
        q3, s3 = topk.quantize_tokens_fp8(hidden)
        logits = topk.product_fp8(q3, s3, head, head_scale)
        ready = topk.penalize_logits(logits, tokens=said, repetition=repetition)
        best = topk.select_topk(ready, 20)
        prob, keep = topk.nucleus(best[1], best[2], 0.7, 0.95)
        return idx, weight, order, q, s, mid, q2, s2, rows, hidden, q3, s3, logits, ready, *best, prob, keep

    (idx, weight, order, q, s, mid, q2, s2, rows, hidden, q3, s3, logits, ready, top, val, count, mask, prob,
     keep) = step()
    assert np.array_equal(idx.cpu().numpy(), oracle_route.route(router.cpu().numpy(), k, None, "sigmoid")[0])
    slot, source, offsets = oracle.order(idx.cpu().numpy(), experts)
    assert np.array_equal(order.slot.cpu().numpy(), slot)
    ref_q, ref_s = oracle.quantize(x.float().cpu().numpy())
    assert np.array_equal(_np(q.float()), oracle.gather(ref_q, source, k))
    assert np.array_equal(_np(s), oracle.gather(ref_s, source, k))
    products_near(mid, *oracle.product(_np(q.float()), _np(s), _np(up.float()), _np(up_scale), offsets), 2)
    assert np.array_equal(_np(q2.float()), oracle.quantize(mid.float().cpu().numpy())[0])
    products_near(rows, *oracle.product(_np(q2.float()), _np(s2), _np(down.float()), _np(down_scale), offsets), 3)
    ref, size = oracle.combine(_np(rows), slot, _np(weight))
    assert (np.abs(_np(hidden) - ref) <= 2.0 ** -8 * np.abs(ref) + k * U * 1.01 * size + 1e-38).all()
    products_near(logits, *oracle.product(_np(q3.float()), _np(s3), _np(head.float()), _np(head_scale)), 2)
    ref, size = oracle_penalty.penalize(_np(logits), said.cpu().numpy(), repetition=_np(repetition))
    assert (np.abs(_np(ready) - ref) <= 2.0 ** -8 * np.abs(ref) + U * 1.01 * size).all()
    exp = topk_oracle.topk(ready.view(torch.int16).cpu().numpy().view(np.uint16), vocab, 20)
    assert np.array_equal(top.cpu().numpy(), exp[0]) and bool((keep >= 1).all())
    assert np.allclose(prob.sum(1).cpu().numpy(), 1, atol=1e-5)

    # the same step captured once and replayed on another token
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = step()
    x.copy_(torch.randn(tokens, dim, generator=g).bfloat16())
    router.copy_(torch.randn(tokens, experts, generator=g))
    graph.replay()
    torch.cuda.synchronize()
    now = step()
    for a, b in zip(kept[5:], now[5:]):
        assert torch.equal(a.float(), b.float())
    assert topk.device_fault() == 0
