"""Tokens by expert, products in 8 bits and penalties without a GPU: the
argument guards of the C ABI and of the binding (nothing is launched), and
pins of their oracles against hand-computed values, torch and differences."""
from __future__ import annotations

import math
import re

import numpy as np
import pytest

from oracle import penalty as oracle_penalty
from oracle import tokens as oracle_tokens
from tests.test_abi_host import FAKE, header_macros


@pytest.fixture(scope="module")
def lib():
    from wide_bf16_row_gb300 import build
    build.build()
    from wide_bf16_row_gb300 import topk
    return topk.library()


def call_sort(lib, idx=FAKE, tokens=4, k=2, experts=8, space=None, room=0, slot=FAKE, source=FAKE, offsets=FAKE):
    return lib.tf_topk_sort_experts(idx, tokens, k, experts, space, room, slot, source, offsets, None)


@pytest.mark.parametrize("kwargs,status", [
    (dict(k=0), 3), (dict(k=33), 3), (dict(tokens=-1), 2), (dict(tokens=2**30, k=2), 2), (dict(experts=0), 2),
    (dict(experts=1025), 2), (dict(idx=None), 1), (dict(slot=None), 1), (dict(source=None), 1),
    (dict(offsets=None), 1), (dict(tokens=0, idx=None, offsets=None), 1), (dict(idx=FAKE + 2), 4),
    (dict(slot=FAKE + 1), 4), (dict(source=FAKE + 2), 4), (dict(offsets=FAKE + 2), 4), (dict(space=FAKE + 2), 4)])
def test_sort_guards(lib, kwargs, status):
    assert call_sort(lib, **kwargs) == status


def test_sort_workspace_of_bad_arguments(lib):
    for args in ((0, 8, 16), (4, 0, 16), (4, 33, 16), (-1, 2, 16), (1000, 8, 0), (1000, 8, 1025), (16, 8, 16)):
        assert lib.tf_topk_sort_experts_workspace(*args) == 0


def call_gather(lib, x=FAKE, dtype=0, tokens=4, dim=64, stride=64, k=2, slot=FAKE, source=FAKE, out=FAKE):
    return lib.tf_topk_gather_tokens(x, dtype, tokens, dim, stride, k, slot, source, out, None)


def call_quantize(lib, x=FAKE, dtype=0, tokens=4, dim=64, stride=64, k=2, slot=FAKE, source=FAKE, out=FAKE,
                  scale=FAKE):
    return lib.tf_topk_quantize_tokens(x, dtype, tokens, dim, stride, k, slot, source, out, scale, None)


def call_combine(lib, x=FAKE, dtype=0, tokens=4, dim=64, stride=64, k=2, slot=FAKE, weight=None, out=FAKE):
    return lib.tf_topk_combine_tokens(x, dtype, tokens, dim, stride, k, slot, weight, out, None)


def call_combine_grad(lib, grad=FAKE, dtype=0, tokens=4, dim=64, stride=64, x=FAKE, row_stride=64, k=2, slot=FAKE,
                      source=FAKE, weight=FAKE, out=FAKE, out_weight=FAKE):
    return lib.tf_topk_combine_tokens_grad(grad, dtype, tokens, dim, stride, x, row_stride, k, slot, source, weight,
                                           out, out_weight, None)


ROWS = [(dict(dtype=3), 10), (dict(dtype=-1), 10), (dict(k=0), 3), (dict(k=33), 3), (dict(tokens=-1), 2),
        (dict(tokens=2**31, k=1), 2), (dict(dim=0), 2), (dict(stride=63), 2), (dict(stride=2**62), 2),
        (dict(tokens=0), 0), (dict(dim=2**30 + 16, stride=2**31), 2), (dict(x=None), 1), (dict(slot=FAKE + 2), 4), (dict(out=None), 1), (dict(x=FAKE + 1), 4),
        (dict(x=FAKE + 2, dtype=2), 4)]


@pytest.mark.parametrize("kwargs,status", ROWS + [
    (dict(slot=None), 1), (dict(source=None), 1), (dict(source=FAKE + 1), 4), (dict(out=FAKE + 2, dtype=2), 4)])
def test_gather_guards(lib, kwargs, status):
    assert call_gather(lib, **kwargs) == status


@pytest.mark.parametrize("kwargs,status", ROWS + [
    (dict(slot=None), 3), (dict(source=None), 1), (dict(scale=None), 1), (dict(dim=24, stride=24), 2),
    (dict(out=FAKE + 8), 4), (dict(scale=FAKE + 2), 4)])
def test_quantize_guards(lib, kwargs, status):
    assert call_quantize(lib, **kwargs) == status


@pytest.mark.parametrize("kwargs,status", ROWS + [
    (dict(slot=None), 1), (dict(weight=FAKE + 2), 4), (dict(out=FAKE + 1), 4)])
def test_combine_guards(lib, kwargs, status):
    assert call_combine(lib, **kwargs) == status


@pytest.mark.parametrize("kwargs,status", ROWS + [
    (dict(slot=None), 1), (dict(source=None), 1), (dict(weight=None), 1), (dict(out_weight=None), 1),
    (dict(grad=None), 1), (dict(grad=FAKE + 1), 4), (dict(row_stride=60), 2), (dict(out_weight=FAKE + 2), 4),
    (dict(weight=FAKE + 2), 4), (dict(source=FAKE + 2), 4)])
def test_combine_grad_guards(lib, kwargs, status):
    assert call_combine_grad(lib, **kwargs) == status


def call_product(lib, q=FAKE, scale=FAKE, rows=4, dim=64, weight=FAKE, wscale=FAKE, cols=32, groups=2, offsets=FAKE,
                 dtype=0, out=FAKE):
    return lib.tf_topk_product_fp8(q, scale, rows, dim, weight, wscale, cols, groups, offsets, dtype, out, None)


@pytest.mark.parametrize("kwargs,status", [
    (dict(dtype=3), 10), (dict(rows=-1), 2), (dict(rows=2**31 - 1), 2), (dict(dim=0), 2), (dict(dim=24), 2),
    (dict(dim=2**30 + 16), 2),
    (dict(cols=0), 2), (dict(cols=2**30), 2), (dict(groups=0), 2), (dict(groups=1025), 2),
    (dict(offsets=None), 2), (dict(rows=0, q=None), 0), (dict(q=None), 1), (dict(scale=None), 1),
    (dict(weight=None), 1), (dict(wscale=None), 1), (dict(out=None), 1), (dict(q=FAKE + 8), 4),
    (dict(weight=FAKE + 1), 4), (dict(scale=FAKE + 2), 4), (dict(wscale=FAKE + 2), 4), (dict(offsets=FAKE + 2), 4),
    (dict(out=FAKE + 1), 4), (dict(out=FAKE + 2, dtype=2), 4), (dict(rows=2**31 - 1000, cols=2**29), 2)])
def test_product_guards(lib, kwargs, status):
    assert call_product(lib, **kwargs) == status


def call_penalize(lib, logits=FAKE, dtype=0, rows=4, cols=100, stride=100, tokens=FAKE, ts=10, width=10, lengths=None,
                  prompts=None, rep=None, pres=None, freq=None, bt=None, bv=None, bs=0, biases=0, allowed=None, als=0,
                  out=FAKE, os=100):
    return lib.tf_topk_penalize(logits, dtype, rows, cols, stride, tokens, ts, width, lengths, prompts, rep, pres, freq,
                                bt, bv, bs, biases, allowed, als, out, os, None)


@pytest.mark.parametrize("kwargs,status", [
    (dict(dtype=3), 10), (dict(rows=-1), 2), (dict(cols=0), 2), (dict(cols=2**31, stride=2**31, os=2**31), 2),
    (dict(stride=99), 2), (dict(os=99), 2), (dict(width=-1), 2), (dict(width=2**29 + 1, ts=2**30), 2), (dict(ts=9), 2), (dict(biases=-1), 2),
    (dict(biases=65536, bs=65536, bt=FAKE, bv=FAKE), 2), (dict(biases=3, bs=2, bt=FAKE, bv=FAKE), 2),
    (dict(allowed=FAKE, als=3), 2), (dict(rows=2**31), 2), (dict(rows=2**40, stride=2**30), 2),
    (dict(rows=0, logits=None, out=None, tokens=None), 0), (dict(logits=None), 1), (dict(out=None), 1),
    (dict(tokens=None), 1), (dict(biases=3, bs=3, bt=FAKE), 1), (dict(biases=3, bs=3, bv=FAKE), 1),
    (dict(logits=FAKE + 1), 4), (dict(logits=FAKE + 2, dtype=2), 4), (dict(out=FAKE + 1), 4), (dict(tokens=FAKE + 2), 4),
    (dict(lengths=FAKE + 2), 4), (dict(prompts=FAKE + 1), 4), (dict(rep=FAKE + 2), 4), (dict(pres=FAKE + 2), 4),
    (dict(freq=FAKE + 2), 4), (dict(biases=3, bs=3, bt=FAKE + 2, bv=FAKE), 4),
    (dict(biases=3, bs=3, bt=FAKE, bv=FAKE + 2), 4), (dict(allowed=FAKE + 2, als=4), 4)])
def test_penalize_guards(lib, kwargs, status):
    assert call_penalize(lib, **kwargs) == status


def test_constants_match_header(lib):
    from wide_bf16_row_gb300 import topk
    m = header_macros()
    assert m["TF_TOPK_FP8_BLOCK"] == topk.FP8_BLOCK == oracle_tokens.BLOCK
    assert m["TF_TOPK_PENALTY_MAX_BIASES"] == topk.PENALTY_MAX_BIASES


def test_binding_refuses_what_it_cannot_run(lib):
    """CPU tensors, wrong types and shapes: Python errors before any call."""
    import torch

    from wide_bf16_row_gb300 import topk
    x, idx = torch.zeros(4, 32), torch.zeros(4, 2, dtype=torch.int32)
    order = topk.ExpertOrder(idx, torch.zeros(8, dtype=torch.int32), torch.zeros(9, dtype=torch.int32))
    with pytest.raises(TypeError):
        topk.sort_by_expert(idx.long(), 8)
    with pytest.raises(ValueError):
        topk.sort_by_expert(idx, 8)
    for call in (lambda t: topk.gather_tokens(t, order), lambda t: topk.quantize_tokens_fp8(t),
                 lambda t: topk.combine_tokens(t, order), lambda t: topk.gather_tokens_grad(t, order),
                 lambda t: topk.combine_tokens_grad(t, t, order, None), lambda t: topk.penalize_logits(t)):
        with pytest.raises(TypeError):
            call(x.double())
        with pytest.raises(ValueError):
            call(x)
    q = torch.zeros(4, 32, dtype=torch.float8_e4m3fn)
    with pytest.raises(TypeError):
        topk.product_fp8(x, x, q, x)
    with pytest.raises(ValueError):
        topk.product_fp8(q, x, q, x)


def test_waits_are_bounded():
    from wide_bf16_row_gb300.build import PKG
    text = (PKG / "csrc" / "tf_topk_product.cu").read_text()
    assert len(re.findall(r"mbarrier\.try_wait", text)) == 1 and "i < kWaitLimit" in text
    for name in ("tokens", "penalty"):
        assert "mbarrier" not in (PKG / "csrc" / f"tf_topk_{name}.cu").read_text()


# ------------------------------------------------------------------ oracle pins


def test_order_oracle_by_hand():
    slot, source, offsets = oracle_tokens.order([[2, 0], [-1, 2], [0, 9]], 3)
    assert offsets.tolist() == [0, 2, 2, 4] and source.tolist() == [1, 4, 0, 3, -1, -1]
    assert slot.tolist() == [[2, 0], [-1, 3], [1, -1]]
    rows = oracle_tokens.gather([[1.0], [2.0], [3.0]], source, 2)
    assert rows[:, 0].tolist() == [1, 3, 1, 2, 0, 0]
    out, size = oracle_tokens.combine(rows, slot, [[1.0, -2.0], [5.0, 3.0], [0.5, 7.0]])
    assert out[:, 0].tolist() == [-1, 6, 1.5] and size[:, 0].tolist() == [3, 6, 1.5]


def test_combine_oracle_gradient_is_the_slope():
    rng = np.random.default_rng(4)
    slot, _, _ = oracle_tokens.order(rng.integers(-1, 4, size=(5, 3)), 4)
    rows, weight, grad = rng.normal(size=(15, 6)), rng.normal(size=(5, 3)), rng.normal(size=(5, 6))
    d_rows, d_weight, _ = oracle_tokens.combine_grad(grad, rows, slot, weight)
    for x, d in ((rows, d_rows), (weight, d_weight)):
        for at in list(np.ndindex(x.shape))[::4]:
            kept, total = x[at], []
            for step in (1e-5, -1e-5):
                x[at] = kept + step
                total.append((oracle_tokens.combine(rows, slot, weight)[0] * grad).sum())
            x[at] = kept
            assert abs((total[0] - total[1]) / 2e-5 - d[at]) < 1e-8


def test_e4m3_oracle_is_torch_s_rounding():
    import torch
    v = np.concatenate([np.linspace(-460, 460, 40001), np.linspace(-0.1, 0.1, 40001), [0.0, 2.0 ** -9, 2.0 ** -10, math.nan]])
    v = v.astype(np.float32)
    v = np.where(np.abs(v) > 448, np.sign(v) * 448, v)
    expect = torch.from_numpy(v).to(torch.float8_e4m3fn).float().numpy()
    np.testing.assert_array_equal(oracle_tokens.e4m3(v), expect)


def test_quantize_oracle_by_hand():
    x = np.zeros((1, 144), np.float32)
    x[0, :3], x[0, 128:131] = [448.0, -17.0, 19.0], [1.0, 0.5, math.inf]
    q, scale = oracle_tokens.quantize(x)
    inv = np.float32(1 / 448)
    assert scale[0, 0] == np.float32(448) * inv and scale[0, 1] == math.inf
    assert q[0, :3].tolist() == [448, -16, 20] and np.isnan(q[0, 130]) and q[0, 128] == 0
    assert oracle_tokens.quantize(np.zeros((1, 16), np.float32))[1][0, 0] == np.float32(2.0 ** -100) * inv


def test_product_oracle_is_a_matrix_product():
    rng = np.random.default_rng(5)
    q, w = rng.integers(-8, 9, (6, 144)), rng.integers(-8, 9, (2, 130, 144))
    s, ws = rng.random((6, 2)), rng.random((2, 2, 2))
    y, size = oracle_tokens.product(q, s, w, ws, [0, 4, 5])
    r, n = 4, 129
    by_hand = sum(s[r, d // 128] * ws[1, 1, d // 128] * q[r, d] * w[1, n, d] for d in range(144))
    assert abs(y[r, n] - by_hand) < 1e-9 * size[r, n] and not y[5].any()


def test_penalty_oracle_by_hand():
    x = np.array([[1.0, -1.0, 2.0, 4.0, 0.5, math.nan]])
    tokens = np.array([[0, 1, 3, 3, 9, 5]])
    y, _ = oracle_penalty.penalize(x, tokens, [5], [2], [2.0], [0.25], [0.5], [[4, 2, 4, -1]], [[1.0, 3.0, 5.0, 9.0]],
                                   np.array([[0b110111]]))
    assert y[0, :3].tolist() == [0.5, -2.0, 5.0] and y[0, 3] == -math.inf and y[0, 4] == 5.5 and np.isnan(y[0, 5])
    y, _ = oracle_penalty.penalize(x, tokens, [4], [2], [2.0], [0.25], [0.5])
    assert y[0, 3] == 4.0 / 2 - 0.5 * 2 - 0.25
