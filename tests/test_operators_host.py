"""The head's loss and expert routing without a GPU: the argument guards of
the C ABI and of the binding (nothing is launched), and pins of their
oracles against hand-computed values, closed forms and differences."""
from __future__ import annotations

import math
import re

import numpy as np
import pytest

from oracle import head_loss as oracle_loss
from oracle import route as oracle_route
from tests.test_abi_host import FAKE, header_macros


@pytest.fixture(scope="module")
def lib():
    from wide_bf16_row_gb300 import build
    build.build()
    from wide_bf16_row_gb300 import topk
    return topk.library()


def call_loss(lib, hidden=FAKE, hs=64, weight=FAKE, ws=64, rows=4, dim=64, vocab=100, target=FAKE, tb=8, space=FAKE,
              loss=FAKE, lse=FAKE):
    return lib.tf_topk_head_loss_bf16(hidden, hs, weight, ws, rows, dim, vocab, target, tb, -100, space, 0, loss, lse,
                                      None)


def call_loss_grad(lib, hidden=FAKE, hs=64, weight=FAKE, ws=64, rows=4, dim=64, vocab=100, target=FAKE, tb=8,
                   space=FAKE, lse=FAKE, grad=FAKE, dh=FAKE, dw=FAKE):
    return lib.tf_topk_head_loss_grad_bf16(hidden, hs, weight, ws, rows, dim, vocab, target, tb, -100, lse, grad, space,
                                           0, dh, dw, None)


SHARED = [
    (dict(rows=-1), 2), (dict(rows=(1 << 20) + 1), 2), (dict(dim=0), 2), (dict(dim=12, hs=16, ws=16), 2),
    (dict(dim=4, hs=8, ws=8), 2), (dict(vocab=0), 2), (dict(vocab=2**31 - 1024), 2), (dict(hs=56), 2), (dict(ws=56), 2),
    (dict(hs=65), 2), (dict(ws=68), 2), (dict(hs=2**39), 2), (dict(ws=2**62), 2), (dict(tb=2), 9), (dict(tb=0), 9),
    (dict(hidden=None), 1), (dict(weight=None), 1), (dict(target=None), 1), (dict(space=None), 1), (dict(lse=None), 1),
    (dict(hidden=FAKE + 8), 4), (dict(weight=FAKE + 2), 4), (dict(target=FAKE + 4), 4), (dict(lse=FAKE + 2), 4),
    (dict(target=FAKE + 2, tb=4), 4),
]


@pytest.mark.parametrize("kwargs,status", SHARED + [(dict(loss=None), 1), (dict(loss=FAKE + 1), 4)])
def test_loss_guards(lib, kwargs, status):
    assert call_loss(lib, **kwargs) == status


@pytest.mark.parametrize("kwargs,status", SHARED + [
    (dict(grad=None), 1), (dict(dh=None, dw=None), 1), (dict(grad=FAKE + 2), 4), (dict(dh=FAKE + 8), 4),
    (dict(dw=FAKE + 2), 4), (dict(rows=0, dw=FAKE + 2), 4)])
def test_loss_grad_guards(lib, kwargs, status):
    assert call_loss_grad(lib, **kwargs) == status


def test_no_rows_no_launch(lib):
    assert call_loss(lib, rows=0, hidden=None, target=None, space=None, loss=None, lse=None) == 0
    assert call_loss_grad(lib, rows=0, dw=None, space=None, target=None) == 0
    assert lib.tf_topk_head_loss_bf16_workspace(0, 64, 100) == 0
    assert lib.tf_topk_head_loss_bf16_workspace(4, 60, 100) == 0
    assert lib.tf_topk_head_loss_grad_bf16_workspace(4, 64, 0, 0) == 0


def call_route(lib, logits=FAKE, dtype=0, tokens=4, experts=64, stride=64, k=6, bias=None, score=0, groups=1, kept=1,
               best=2, renorm=1, scale=1.0, idx=FAKE, weight=FAKE, load=None):
    return lib.tf_topk_route(logits, dtype, tokens, experts, stride, k, bias, score, groups, kept, best, renorm, scale,
                             idx, weight, load, None)


@pytest.mark.parametrize("kwargs,status", [
    (dict(dtype=3), 10), (dict(dtype=-1), 10), (dict(k=0), 3), (dict(k=33), 3), (dict(tokens=-1), 2),
    (dict(experts=0), 2), (dict(experts=1025, stride=1025), 2), (dict(stride=63), 2), (dict(tokens=2**40, stride=2**30), 2),
    (dict(score=2), 9), (dict(score=-1), 9), (dict(groups=0), 9), (dict(groups=3), 9), (dict(groups=64, kept=1), 9),
    (dict(groups=8, kept=0), 9), (dict(groups=8, kept=9), 9), (dict(best=0), 9), (dict(best=3), 9),
    (dict(scale=math.inf), 9), (dict(scale=math.nan), 9), (dict(logits=None), 1), (dict(idx=None), 1),
    (dict(weight=None), 1), (dict(logits=FAKE + 1), 4), (dict(logits=FAKE + 2, dtype=2), 4), (dict(bias=FAKE + 2), 4),
    (dict(idx=FAKE + 1), 4), (dict(weight=FAKE + 2), 4), (dict(load=FAKE + 2), 4), (dict(tokens=0), 0)])
def test_route_guards(lib, kwargs, status):
    assert call_route(lib, **kwargs) == status


def call_route_grad(lib, logits=FAKE, dtype=0, tokens=4, experts=64, stride=64, k=6, idx=FAKE, grad=FAKE, score=0,
                    renorm=1, scale=1.0, out=FAKE):
    return lib.tf_topk_route_grad(logits, dtype, tokens, experts, stride, k, idx, grad, score, renorm, scale, out, None)


@pytest.mark.parametrize("kwargs,status", [
    (dict(dtype=7), 10), (dict(k=0), 3), (dict(k=33), 3), (dict(tokens=-2), 2), (dict(experts=0), 2),
    (dict(stride=10), 2), (dict(score=2), 9), (dict(scale=math.nan), 9), (dict(logits=None), 1), (dict(idx=None), 1),
    (dict(grad=None), 1), (dict(out=None), 1), (dict(logits=FAKE + 1), 4), (dict(out=FAKE + 2, dtype=2), 4),
    (dict(idx=FAKE + 2), 4), (dict(grad=FAKE + 1), 4), (dict(tokens=0), 0)])
def test_route_grad_guards(lib, kwargs, status):
    assert call_route_grad(lib, **kwargs) == status


def test_constants_match_header(lib):
    from wide_bf16_row_gb300 import topk
    m = header_macros()
    assert m["TF_TOPK_ROUTE_MAX_EXPERTS"] == topk.ROUTE_MAX_EXPERTS
    assert m["TF_TOPK_ROUTE_MAX_K"] == topk.ROUTE_MAX_K
    assert m["TF_TOPK_ROUTE_MAX_GROUPS"] == topk.ROUTE_MAX_GROUPS
    assert topk.ROUTE_SCORES == {"softmax": m["TF_TOPK_ROUTE_SOFTMAX"], "sigmoid": m["TF_TOPK_ROUTE_SIGMOID"]}


def test_binding_refuses_what_it_cannot_run(lib):
    """CPU tensors, wrong types and shapes: Python errors before any call."""
    import torch

    from wide_bf16_row_gb300 import topk
    h, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(100, 64, dtype=torch.bfloat16)
    t = torch.zeros(4, dtype=torch.int64)
    for args, err in (((h, w, t), ValueError), ((h.float(), w, t), TypeError), ((h[0], w, t), ValueError)):
        with pytest.raises(err):
            topk.head_loss_bf16(*args)
        with pytest.raises(err):
            topk.head_loss_grad_bf16(*args, torch.zeros(4), torch.zeros(4))
    x = torch.zeros(4, 16)
    for args, kwargs, err in (((x, 2), {}, ValueError), ((x.double(), 2), {}, TypeError),
                              ((x, 2), {"score": "relu"}, ValueError)):
        with pytest.raises(err):
            topk.route_experts(*args, **kwargs)
    with pytest.raises(ValueError):
        topk.route_experts_grad(x, torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2))


# ------------------------------------------------------------------ oracle pins


def test_loss_oracle_by_hand():
    h, w = np.eye(2), np.array([[1.0, 0.0], [0.0, 2.0], [0.0, 0.0]])
    loss, lse = oracle_loss.loss(h, w, [0, 2])
    e = math.e
    np.testing.assert_allclose(lse, [math.log(e + 2), math.log(e**2 + 2)], rtol=1e-14)
    np.testing.assert_allclose(loss, [math.log(e + 2) - 1, math.log(e**2 + 2)], rtol=1e-14)
    loss, lse = oracle_loss.loss(h, w, [-100, 3])
    assert loss[0] == lse[0] == 0 and np.isnan(loss[1]) and np.isnan(lse[1])
    loss, _ = oracle_loss.loss([[40.0]], [[1.0], [0.0]], [0])
    np.testing.assert_allclose(loss, [math.exp(-40)], rtol=1e-14)


def test_loss_oracle_gradient_is_the_slope():
    rng = np.random.default_rng(1)
    h, w = rng.normal(size=(3, 5)), rng.normal(size=(7, 5))
    t, g = np.array([6, -100, 2]), rng.normal(size=3)
    dh, dw, G = oracle_loss.grad(h, w, t, g)
    assert not dh[1].any() and np.allclose(G.sum(1), 0, atol=1e-15)
    step = 1e-6

    def total(a, b):
        return (oracle_loss.loss(a, b, t)[0] * g).sum()

    for x, d, at in ((h, dh, (0, 3)), (h, dh, (2, 1)), (w, dw, (6, 0)), (w, dw, (1, 4))):
        up, down = x.copy(), x.copy()
        up[at] += step
        down[at] -= step
        s = (total(up, w) - total(down, w)) if x is h else (total(h, up) - total(h, down))
        assert abs(s / (2 * step) - d[at]) < 1e-8


def test_route_oracle_by_hand():
    x = np.array([[0.0, 2.0, 1.0, 2.0]])
    idx, weight, load = oracle_route.route(x, 2)
    assert idx.tolist() == [[1, 3]] and np.allclose(weight, 0.5) and load.tolist() == [0, 1, 0, 1]
    idx, weight, _ = oracle_route.route(x, 2, bias=[10.0, 0, 0, 0], score="sigmoid", renorm=False, scale=2.0)
    assert idx.tolist() == [[0, 1]]  # the bias moves the choice, not the weight
    np.testing.assert_allclose(weight, [[1.0, 2 / (1 + math.exp(-2))]], rtol=1e-14)
    # two groups of two: sums 0 + 2 against 1 + 2; with the best alone a tie, the lower group
    assert oracle_route.route(x, 2, score="sigmoid", groups=2, kept=1)[0].tolist() == [[3, 2]]
    assert oracle_route.route(x, 2, score="sigmoid", groups=2, kept=1, best=1)[0].tolist() == [[1, 0]]
    masked = np.array([[-np.inf, np.nan, 3.0, -np.inf]])
    idx, weight, _ = oracle_route.route(masked, 2)
    assert idx.tolist() == [[2, -1]] and weight.tolist() == [[1.0, 0.0]]
    assert oracle_route.route(np.full((1, 3), -np.inf), 2)[0].tolist() == [[-1, -1]]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_oracle_gradient_is_the_slope(score, renorm):
    rng = np.random.default_rng(2)
    x, g = rng.normal(size=(2, 6)), rng.normal(size=(2, 3))
    idx, _, _ = oracle_route.route(x, 3, score=score, renorm=renorm, scale=1.5)
    d, size = oracle_route.grad(x, idx, g, score, renorm, 1.5)
    assert (np.abs(d) <= size + 1e-15).all()
    step = 1e-6
    for at in np.ndindex(x.shape):
        sides = []
        for sign in (1, -1):
            y = x.copy()
            y[at] += sign * step
            i, w, _ = oracle_route.route(y, 3, score=score, renorm=renorm, scale=1.5)
            assert (i == idx).all()
            sides.append((w * g).sum())
        assert abs((sides[0] - sides[1]) / (2 * step) - d[at]) < 1e-8


def test_waits_are_bounded():
    """The new kernels' waits all count their polls."""
    from wide_bf16_row_gb300.build import PKG
    text = (PKG / "csrc" / "tf_topk_head_loss.cu").read_text()
    assert len(re.findall(r"mbarrier\.try_wait", text)) == 1 and "i < kWaitLimit" in text
    assert "try_wait" not in (PKG / "csrc" / "tf_topk_route.cu").read_text()
