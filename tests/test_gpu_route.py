"""GPU parity of expert routing and its gradient against the 64-bit oracle.

Indices and loads are equal, ties and near-ties included.  Tolerance of the
weights, from the kernel's fp32 arithmetic (u = 2^-24): a score takes an
exponential (2 ulp = 4 u; the fast one behind a softmax's sum 2 + 1.18 |x|
ulp), the rounded difference x - max (|x - max| u relative), a sum of at most
1024 positive terms in 32 partial sums (37 u) and a division (u); over the
chosen ones another sum of at most 32 terms (6 u in a butterfly) and a
division.  With |x - max| <= 30 wherever a term is not negligible this stays
below 150 u = 9e-6 relative; the tests allow 1e-5.  Terms below fp32's normal
range add 1e-37.  The gradient is a sum of terms s (|g| + sum |g| s) each
within twice that, rounded once to its type (eps / 2)."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import route as oracle_route

pytestmark = pytest.mark.gpu

RTOL = 1e-5
TYPES = ("bf16", "fp16", "fp32")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from wide_bf16_row_gb300 import build
    build.build()


def _dtype(name):
    import torch
    return {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[name]


def _logits(tokens, experts, dtype, seed, spread=1.5, masked=0.0):
    import torch
    g = torch.Generator().manual_seed(seed)
    x = spread * torch.randn(tokens, experts, generator=g)
    if masked:
        x[torch.rand(tokens, experts, generator=g) < masked] = -float("inf")
        x[torch.rand(tokens, generator=g) < 0.1] = -float("inf")
        x[torch.rand(tokens, experts, generator=g) < masked / 4] = float("nan")
    return x.to(_dtype(dtype)).cuda()


def _bias(experts, seed, size=0.1):
    import torch
    return (size * torch.randn(experts, generator=torch.Generator().manual_seed(seed))).cuda()


def _np(x):
    return x.float().cpu().numpy()


def check(logits, k, bias=None, score="softmax", groups=1, kept=None, best=2, renorm=True, scale=1.0, seed=0):
    import torch

    from wide_bf16_row_gb300 import topk
    tokens, experts = logits.shape
    load = torch.full((experts,), 3, dtype=torch.int32, device="cuda")
    idx, weight = topk.route_experts(logits, k, bias=bias, score=score, groups=groups, groups_kept=kept,
                                     group_best=best, renormalize=renorm, scale=scale, load=load)
    x = _np(logits)
    ref_idx, ref_weight, ref_load = oracle_route.route(x, k, None if bias is None else bias.cpu().numpy(), score,
                                                       groups, kept, best, renorm, scale)
    got = idx.cpu().numpy()
    bad = np.flatnonzero((got != ref_idx).any(1))
    assert not len(bad), f"{len(bad)} rows differ, first {bad[0]}: {got[bad[0]]} expected {ref_idx[bad[0]]}"
    np.testing.assert_allclose(weight.cpu().numpy(), ref_weight, rtol=RTOL, atol=1e-37)
    assert np.array_equal(load.cpu().numpy(), ref_load + 3)
    g = torch.randn(tokens, k, generator=torch.Generator().manual_seed(seed + 1))
    g[idx.cpu() < 0] = float("nan")  # a skipped place's gradient is not used
    d = topk.route_experts_grad(logits, idx, g.cuda(), score=score, renormalize=renorm, scale=scale)
    assert d.dtype == logits.dtype and d.shape == logits.shape
    ref, size = oracle_route.grad(x, ref_idx, g.numpy(), score, renorm, scale)
    tiny = {"bf16": 1e-37, "fp16": 2.0 ** -25, "fp32": 1e-37}
    name = {torch.bfloat16: "bf16", torch.float16: "fp16", torch.float32: "fp32"}[d.dtype]
    allow = torch.finfo(d.dtype).eps / 2 * np.abs(ref) + 2 * RTOL * size + tiny[name]
    off = np.abs(d.double().cpu().numpy() - ref)
    assert (off <= allow).all(), f"gradient off by {np.max(off - allow)} at {np.argwhere(off > allow)[0]}"
    return idx, weight


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("tokens,experts,k", [(1, 8, 2), (1, 256, 8), (70, 1, 1), (67, 33, 5), (67, 60, 4), (65, 128, 8),
                                              (33, 257, 9), (9, 1000, 32), (5, 1024, 31), (40, 5, 8)])
def test_plain(dtype, score, renorm, tokens, experts, k):
    check(_logits(tokens, experts, dtype, seed=experts + k), k, score=score, renorm=renorm, scale=2.5)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("best", [1, 2])
@pytest.mark.parametrize("experts,groups,kept,k", [(256, 8, 4, 8), (256, 8, 1, 8), (64, 8, 3, 6), (60, 4, 2, 4),
                                                   (96, 32, 5, 10), (160, 5, 3, 6), (32, 32, 7, 9), (24, 2, 1, 16),
                                                   (1024, 16, 4, 32), (512, 8, 4, 8)])
@pytest.mark.parametrize("with_bias", [True, False])
def test_groups(dtype, score, best, experts, groups, kept, k, with_bias):
    bias = _bias(experts, 3) if with_bias else None
    check(_logits(41, experts, dtype, seed=experts + groups, masked=0.05), k, bias, score, groups, kept, best)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("experts,groups,kept,k,with_bias", [
    (256, 8, 4, 8, True), (256, 1, 1, 8, False), (128, 8, 3, 7, False), (100, 1, 1, 5, True), (64, 4, 2, 6, True),
    (60, 1, 1, 4, False), (32, 2, 1, 3, True), (4, 1, 1, 8, True), (240, 5, 2, 1, False), (256, 16, 15, 8, True)])
def test_enough_tokens_for_four_lanes_each(dtype, score, experts, groups, kept, k, with_bias):
    """At least eight tokens per SM: the kernel that gives a token four lanes, with masked experts, empty rows and a
    ragged last warp."""
    bias = _bias(experts, 3) if with_bias else None
    x = _logits(1301, experts, dtype, seed=experts + groups, masked=0.1)
    check(x, k, bias, score, groups, kept, 2 - k % 2, renorm=k != 8 or with_bias, scale=1.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_ties_and_extremes_with_four_lanes_each(score):
    import torch
    x = torch.zeros(1301, 64, device="cuda")
    check(x, 6, None, score)
    check(x, 6, torch.zeros(64, device="cuda"), score, 4, 2, 2)
    coarse = (_logits(1301, 64, "fp32", 5) * 2).round() / 2
    check(coarse, 6, None, score, 4, 2, 2)
    check(coarse, 6, torch.full((64,), 0.25, device="cuda"), score)
    far = _logits(1301, 64, "fp32", 6) * 200
    far[:, ::5] = float("inf")
    far[:, 1::7] = -float("inf")
    far[1::2] -= 3000
    check(far, 8, None, score)
    check(far, 8, None, score, renorm=False)
    check(far, 8, _bias(64, 9, 5.0), score, 4, 3, 2)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_masked(dtype, score, renorm):
    """Experts out of reach, rows that have fewer than k or none."""
    check(_logits(200, 40, dtype, seed=11, masked=0.9), 8, _bias(40, 5), score, renorm=renorm)
    check(_logits(200, 40, dtype, seed=12, masked=0.9), 8, None, score, 4, 2, 2, renorm=renorm)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_ties(score):
    """Equal logits: the lower expert and the lower group, with and without a bias."""
    import torch
    x = torch.zeros(20, 64, device="cuda")
    check(x, 6, None, score)
    check(x, 6, torch.zeros(64, device="cuda"), score, 8, 3, 2)
    coarse = (_logits(300, 64, "fp32", 5) * 2).round() / 2
    check(coarse, 6, None, score, 8, 3, 2)
    check(coarse, 6, torch.full((64,), 0.25, device="cuda"), score)
    signed = torch.tensor([[0.0, -0.0, 0.0, -0.0]], device="cuda")
    check(signed, 2, None, score)
    check(signed - 0.0, 3, torch.tensor([-0.5, -0.5, 0.0, -0.0], device="cuda"), score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("gap", [1e-9, 1e-8, 3e-8, 1e-7, 1e-6])
def test_near_ties(score, gap):
    """Choices that 32 bits cannot order: the bias cancels the scores' differences
    but for a few parts in 2^24."""
    import torch
    g = torch.Generator().manual_seed(int(1e9 * gap))
    x = torch.randn(1, 32, generator=g).repeat(64, 1)
    s = torch.sigmoid(x.double()) if score == "sigmoid" else torch.softmax(x.double(), 1)
    bias = (1.0 - s[0] + gap * torch.randn(32, generator=g).double()).float()
    x[1:] += 1e-7 * torch.randn(63, 32, generator=g)
    check(x.cuda(), 7, bias.cuda(), score)
    check(x.cuda(), 7, bias.cuda(), score, 4, 2, 2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_extremes(score):
    """Infinite and huge logits, scores that underflow, biases that dwarf them."""
    import torch
    inf = float("inf")
    x = torch.tensor([[inf, 1.0, inf, 2.0, -inf, 0.0], [3e38, -3e38, 3e38, 0.0, 1.0, 2.0],
                      [-200.0, -201.0, -202.0, -203.0, -204.0, -205.0], [-inf, -inf, -inf, -inf, -inf, -1e30],
                      [float("nan")] * 6, [90.0, 89.0, 88.0, 87.0, -90.0, -89.0]], device="cuda")
    check(x, 3, None, score)
    check(x, 3, None, score, renorm=False)
    check(x, 3, None, score, 3, 2, 1)
    check(x, 4, torch.tensor([1e6, -1e6, 1e6, 0.0, inf, -inf], device="cuda"), score)
    check(x, 2, torch.tensor([0.0, float("nan"), 1.0, 1.0, 1.0, 1.0], device="cuda"), score)


def test_strided_rows_and_offsets():
    import torch
    wide = torch.randn(50, 71, device="cuda")
    check(wide[:, 3:67], 6, None, "softmax")
    check(wide.bfloat16()[::3, 1:65], 6, _bias(64, 1), "sigmoid", 8, 4, 2)


def test_many_tokens():
    """More tokens than warps in flight, the load's sum."""
    import torch

    from wide_bf16_row_gb300 import topk
    x = torch.randn(40001, 64, device="cuda", dtype=torch.bfloat16)
    load = torch.zeros(64, dtype=torch.int32, device="cuda")
    idx, weight = topk.route_experts(x, 8, load=load)
    assert int(load.sum()) == 40001 * 8
    assert torch.equal(load, torch.bincount(idx.view(-1).long(), minlength=64).int())
    value, order = x.float().sort(dim=1, descending=True, stable=True)
    assert torch.equal(idx, order[:, :8].int())
    torch.testing.assert_close(weight, torch.softmax(value[:, :8].double(), 1).float(), rtol=RTOL, atol=0)


def test_twice_named_and_foreign_indices():
    """Entries out of range are skipped; an expert named twice adds up."""
    import torch

    from wide_bf16_row_gb300 import topk
    x = torch.randn(7, 10, device="cuda")
    idx = torch.tensor([[3, 3, 1], [0, -1, 0], [9, 10, 2], [-7, 4, 4], [1 << 30, 5, 6], [2, 2, 2], [-1, -1, -1]],
                       dtype=torch.int32, device="cuda")
    g = torch.randn(7, 3, device="cuda")
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            d = topk.route_experts_grad(x, idx, g, score=score, renormalize=renorm)
            ref, size = oracle_route.grad(_np(x), idx.cpu().numpy(), g.cpu().numpy(), score, renorm)
            assert (np.abs(d.double().cpu().numpy() - ref) <= 2 ** -24 * np.abs(ref) + 2 * RTOL * size).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_against_differences(score, renorm):
    """Central differences of the kernel's own weights: steps of 2^-6 leave
    fp32 noise of 1e-6 / 2^-5 and a third-order term below 2^-12 / 6 per unit of g."""
    import torch

    from wide_bf16_row_gb300 import topk
    x = torch.randn(3, 12, generator=torch.Generator().manual_seed(4)).clamp(-2, 2).cuda()
    x[:, ::4] += 4.5  # these three stay chosen: they lead by at least 0.5, and a step is 2^-6
    idx, _ = topk.route_experts(x, 3, score=score, renormalize=renorm)
    g = torch.randn(3, 3, device="cuda")
    d = topk.route_experts_grad(x, idx, g, score=score, renormalize=renorm)
    step = 2.0 ** -6
    for e in range(12):
        sides = []
        for sign in (1, -1):
            y = x.clone()
            y[:, e] += sign * step
            i, w = topk.route_experts(y, 3, score=score, renormalize=renorm)
            back = (i[:, None, :] == idx[:, :, None]).long().argmax(2)
            assert torch.equal(i.gather(1, back), idx)
            sides.append((w.gather(1, back) * g).sum(1))
        slope = (sides[0] - sides[1]) / (2 * step)
        assert (slope - d[:, e]).abs().max() <= (3.2e-5 + 2 ** -12) * g.abs().sum(1).max()


def test_streams_graphs_and_outputs():
    """Another stream than the current one, caller's outputs, a captured and replayed call."""
    import torch

    from wide_bf16_row_gb300 import topk
    x = _logits(100, 64, "bf16", 1)
    want = topk.route_experts(x, 6, score="sigmoid", groups=8, groups_kept=4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = topk.route_experts(x, 6, score="sigmoid", groups=8, groups_kept=4, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    out = (torch.zeros(100, 6, dtype=torch.int32, device="cuda"), torch.zeros(100, 6, device="cuda"))
    load = torch.zeros(64, dtype=torch.int32, device="cuda")
    g = torch.randn(100, 6, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        topk.route_experts(x, 6, score="sigmoid", groups=8, groups_kept=4, load=load, out=out)
        d = topk.route_experts_grad(x, out[0], g, score="sigmoid")
    x.copy_(_logits(100, 64, "bf16", 2))
    graph.replay()
    graph.replay()
    idx, weight, ref_load = oracle_route.route(_np(x), 6, None, "sigmoid", 8, 4, 2)
    assert np.array_equal(out[0].cpu().numpy(), idx)
    assert np.array_equal(load.cpu().numpy(), 2 * ref_load)
    assert torch.equal(d, topk.route_experts_grad(x, out[0], g, score="sigmoid"))


def test_no_tokens():
    import torch

    from wide_bf16_row_gb300 import topk
    x = torch.empty(0, 16, device="cuda")
    idx, weight = topk.route_experts(x, 2)
    assert idx.shape == (0, 2) and weight.shape == (0, 2)
    assert topk.route_experts_grad(x, idx, weight).shape == (0, 16)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tokens,experts,k,renorm", [(1, 7, 3, True), (33, 60, 4, False), (1301, 256, 8, True), (1301, 64, 6, False)])
def test_nothing_beside_the_outputs_is_written(dtype, tokens, experts, k, renorm):
    """Outputs of exactly their sizes inside larger buffers."""
    import torch

    from wide_bf16_row_gb300 import topk
    x = _logits(tokens, experts, dtype, 3)
    g = torch.randn(tokens, k, device="cuda")

    def inside(shape, kind):
        size = int(np.prod(shape)) * kind.itemsize
        block = torch.full((256 + size + 256,), 0xA5, dtype=torch.uint8, device="cuda")
        return block, block[256:256 + size].view(kind).view(shape)
    blocks, parts = zip(inside((tokens, k), torch.int32), inside((tokens, k), torch.float32),
                        inside((experts,), torch.int32), inside((tokens, experts), x.dtype))
    parts[2].zero_()
    topk.route_experts(x, k, renormalize=renorm, load=parts[2], out=parts[:2])
    topk.route_experts_grad(x, parts[0], g, renormalize=renorm, out=parts[3])
    for block in blocks:
        assert bool((block[:256] == 0xA5).all()) and bool((block[-256:] == 0xA5).all())
    idx, weight = topk.route_experts(x, k, renormalize=renorm)
    assert torch.equal(parts[0], idx) and torch.equal(parts[1], weight)
    assert torch.equal(parts[2], torch.bincount(idx.view(-1).long(), minlength=experts).int())
    assert torch.equal(parts[3], topk.route_experts_grad(x, idx, g, renormalize=renorm))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("experts,k,with_bias", [(1, 1, True), (3, 8, False), (22, 8, False), (61, 5, True), (101, 8, True),
                                                 (130, 1, True), (253, 7, False), (255, 8, True)])
def test_odd_expert_counts_with_four_lanes_each(dtype, score, experts, k, with_bias):
    """Rows that are no whole vectors; the last element of the last row ends the buffer."""
    bias = _bias(experts, 3) if with_bias else None
    check(_logits(1301, experts, dtype, seed=experts, masked=0.1), k, bias, score, renorm=k != 8 or with_bias, scale=1.5)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("stride,start,step", [(67, 0, 1), (72, 1, 1), (68, 2, 2)])
def test_rows_off_the_vectors_with_four_lanes_each(dtype, stride, start, step):
    check(_logits(1301 * step, stride, dtype, seed=stride)[::step, start:start + 64], 6, _bias(64, 1), "sigmoid", 4, 2, 2)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("experts,groups,kept,k,best", [(22, 2, 1, 8, 2), (31, 31, 9, 7, 2), (62, 31, 4, 5, 2), (100, 4, 3, 1, 1),
                                                        (216, 8, 5, 3, 2), (216, 27, 5, 6, 1), (510, 3, 2, 7, 2),
                                                        (992, 31, 9, 20, 2)])
def test_groups_across_lanes(dtype, score, experts, groups, kept, k, best):
    """Groups whose ends lie inside a lane's experts; masked experts, groups without any, near and whole ties."""
    import torch
    x = _logits(1301 if experts < 500 else 150, experts, dtype, seed=experts, masked=0.1)
    x[3::7, :experts // groups] = -float("inf")
    x[5::7] = (x[5::7] * 2).round() / 2
    x[6::7] = 0.5
    check(x, k, None, score, groups, kept, best)
    check(x, k, _bias(experts, 3), score, groups, kept, best)
    check(x, k, torch.zeros(experts, device="cuda"), score, groups, kept, best, renorm=False)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("experts,groups,kept,k,best", [(15, 15, 7, 8, 2), (4, 2, 1, 8, 2), (60, 5, 2, 5, 1), (91, 7, 6, 6, 2),
                                                        (128, 16, 3, 8, 2), (127, 1, 1, 3, 2), (126, 2, 1, 8, 2)])
def test_groups_of_any_size_with_four_lanes_each(dtype, score, experts, groups, kept, k, best):
    import torch
    x = _logits(1301, experts, dtype, seed=experts, masked=0.1)
    x[3::7, :experts // groups] = -float("inf")
    x[5::7] = (x[5::7] * 2).round() / 2
    x[6::7] = 0.5
    check(x, k, None, score, groups, kept, best)
    check(x, k, _bias(experts, 3), score, groups, kept, best)
    check(x, k, torch.zeros(experts, device="cuda"), score, groups, kept, best, renorm=False)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_an_only_choice_has_weight_scale_and_no_gradient(dtype, score):
    """Renormalised, one expert's weight is the scale whatever its logit: no rounding may leave a gradient."""
    import torch

    from wide_bf16_row_gb300 import topk
    x = _logits(1301, 33, dtype, 8)
    x[::3, 1:] = -float("inf")
    for k, rows in ((1, slice(None)), (4, slice(None, None, 3)), (12, slice(None, None, 3))):
        idx, weight = topk.route_experts(x, k, score=score, scale=2.5)
        d = topk.route_experts_grad(x, idx, torch.randn(1301, k, device="cuda"), score=score, scale=2.5)
        assert not torch.any(d[rows] != 0)
        torch.testing.assert_close(weight[rows, 0], torch.full_like(weight[rows, 0], 2.5), rtol=2 * RTOL, atol=0)
