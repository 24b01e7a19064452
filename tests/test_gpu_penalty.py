"""GPU parity of penalties, biases and masks on logits against the oracle in 64 bits.

Tolerance (u = 2^-24): at most five roundings to 32 bits (the product or quotient
with the repetition penalty, frequency times count, two differences, a sum), each
off by at most u of a magnitude that the oracle keeps as `size`; then one
rounding to the logits' type (eps / 2, and half its smallest step).  What
nothing names keeps its bits."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import penalty as oracle

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = ("bf16", "fp16", "fp32")
TINY = {"bf16": 1e-38, "fp16": 2.0 ** -25, "fp32": 1e-44}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from wide_bf16_row_gb300 import build
    build.build()


def _dtype(name):
    import torch
    return {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[name]


def logits_of(rows, cols, dtype, seed, stride=None, offset=0):
    import torch
    x = (3 * torch.randn(rows, cols, generator=torch.Generator().manual_seed(seed))).to(_dtype(dtype))
    stride = stride or cols
    flat = torch.full((offset + rows * stride + 16,), float("nan"), dtype=x.dtype, device="cuda")
    view = flat.as_strided((rows, cols), (stride, 1), offset)
    view.copy_(x)
    return view


def request(rows, cols, width=0, biases=0, mask=False, seed=0, token_stride=None):
    import torch
    g = torch.Generator().manual_seed(seed)
    r = {}
    if width:
        tokens = (cols * torch.rand(rows, width, generator=g) ** 3).int()
        tokens[torch.rand(rows, width, generator=g) < 0.02] = -1
        tokens[torch.rand(rows, width, generator=g) < 0.02] = cols
        if token_stride:
            wide = torch.zeros(rows, token_stride, dtype=torch.int32)
            wide[:, 1:1 + width] = tokens
            r["tokens"] = wide.cuda()[:, 1:1 + width]
        else:
            r["tokens"] = tokens.cuda()
        r["lengths"] = torch.randint(-1, width + 3, (rows,), generator=g, dtype=torch.int32).cuda()
        r["prompts"] = torch.randint(-1, width + 3, (rows,), generator=g, dtype=torch.int32).cuda()
        r["repetition"] = (0.7 + torch.rand(rows, generator=g)).cuda()
        r["presence"] = (torch.rand(rows, generator=g) - 0.3).cuda()
        r["frequency"] = (torch.rand(rows, generator=g) - 0.3).cuda()
        for name, none in (("repetition", 1.0), ("presence", 0.0), ("frequency", 0.0)):
            r[name][::3] = none
    if biases:
        names = torch.randint(-1, cols + 1, (rows, biases), generator=g, dtype=torch.int32)
        names[:, biases // 2] = names[:, 0]  # a column twice: the last counts
        r["bias_tokens"] = names.cuda()
        r["bias_values"] = (4 * torch.randn(rows, biases, generator=g)).cuda()
    if mask:
        words = torch.randint(-2**31, 2**31, (rows, -(-cols // 32)), generator=g, dtype=torch.int64).int()
        words[::4] = 0  # nothing is left
        words[1::4] = -1
        r["allowed"] = words.cuda()
    return r


def check(x, r, dtype, **kw):
    import torch

    from wide_bf16_row_gb300 import topk
    host = {n: t.cpu().numpy() for n, t in r.items()}
    before = x.clone()
    ref, size = oracle.penalize(x.double().cpu().numpy(), **host)
    # a result half a step or more beyond the type's largest number is rounded to infinity
    info = torch.finfo(x.dtype)
    beyond = np.abs(ref) >= info.max * (1 + info.eps / 2 / (2 - info.eps))
    ref = np.where(beyond, np.copysign(np.inf, ref), ref)
    y = topk.penalize_logits(x, **r, **kw)
    assert y.dtype == x.dtype and y.shape == x.shape
    if kw.get("out") is not x:
        assert torch.equal(x.contiguous().view(torch.uint8), before.contiguous().view(torch.uint8))
    got = y.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    fine = np.isfinite(ref)
    assert np.array_equal(got[~fine & ~np.isnan(ref)], ref[~fine & ~np.isnan(ref)])
    allow = torch.finfo(x.dtype).eps / 2 * np.abs(ref[fine]) + 5 * U * 1.01 * size[fine] + TINY[dtype]
    off = np.abs(got[fine] - ref[fine])
    assert (off <= allow).all(), f"off by {np.max(off - allow)}"
    return y


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols,width,biases,mask,stride,offset,token_stride", [
    (1, 1, 1, 1, True, None, 0, None), (3, 100, 0, 0, True, None, 0, None), (5, 1003, 50, 5, True, 1010, 3, None),
    (4, 4096, 300, 0, False, None, 0, 310), (9, 32771, 3000, 40, True, None, 0, 3005), (2, 50000, 0, 300, False, 50008, 8, None),
    (7, 98592, 20000, 3, False, None, 1, None), (330, 2049, 64, 9, True, 2056, 0, None), (1, 248320, 9000, 16, True, None, 0, None),
    (40, 16392, 7, 0, True, None, 0, None), (33, 31, 5, 2, True, 33, 1, 6)])
def test_parity(dtype, rows, cols, width, biases, mask, stride, offset, token_stride):
    x = logits_of(rows, cols, dtype, rows + cols, stride, offset)
    check(x, request(rows, cols, width, biases, mask, seed=cols, token_stride=token_stride), dtype)


@pytest.mark.parametrize("dtype", TYPES)
def test_specials(dtype):
    import math

    import torch
    x = logits_of(6, 700, dtype, 1)
    for i, v in enumerate((math.nan, math.inf, -math.inf, 0.0, -0.0, torch.finfo(x.dtype).min, torch.finfo(x.dtype).max,
                           torch.finfo(x.dtype).tiny)):
        x[:, i::16] = v
    check(x, request(6, 700, 900, 30, True, seed=3), dtype)
    y = check(x, request(6, 700, 900, 0, False, seed=3), dtype)
    # rows 0 and 3 ask for nothing: their bits stay, NaN's too
    assert torch.equal(y[::3].view(torch.uint8), x[::3].contiguous().view(torch.uint8))
    assert torch.equal(check(x, {}, dtype).view(torch.uint8), x.view(torch.uint8))


def test_each_part_alone():
    full = request(8, 3000, 400, 20, True, seed=5)
    for names in (("tokens", "repetition"), ("tokens", "lengths", "frequency"), ("tokens", "prompts", "presence"),
                  ("bias_tokens", "bias_values"), ("allowed",), ("tokens",), ("repetition", "presence", "frequency"),
                  ("tokens", "lengths", "prompts", "repetition", "allowed")):
        check(logits_of(8, 3000, "fp32", 2), {n: full[n] for n in names}, "fp32")


@pytest.mark.parametrize("dtype,stride,offset", [("bf16", None, 0), ("fp32", 1010, 1), ("fp16", 1011, 0)])
def test_in_place_and_into_strided_rows(dtype, stride, offset):
    import torch

    from wide_bf16_row_gb300 import topk
    r = request(20, 1003, 60, 6, True, seed=7)
    x = logits_of(20, 1003, dtype, 3, stride, offset)
    ref = topk.penalize_logits(x, **r)
    flat = torch.full((20 * 1040 + 9,), 3.0, dtype=x.dtype, device="cuda")
    out = flat.as_strided((20, 1003), (1040, 1), 5)
    topk.penalize_logits(x, **r, out=out)
    assert torch.equal(out, ref)
    assert bool((flat[:5] == 3).all()) and bool((flat[5:5 + 20 * 1040].view(20, 1040)[:, 1003:] == 3).all())
    assert topk.penalize_logits(x, **r, out=x) is x
    assert torch.equal(x, ref)


def test_as_many_biases_as_there_may_be():
    import torch

    from wide_bf16_row_gb300 import topk
    r = request(2, 70000, 0, topk.PENALTY_MAX_BIASES, False, seed=8)
    check(logits_of(2, 70000, "fp32", 4), r, "fp32")
    same = {"bias_tokens": torch.full((1, 60000), 17, dtype=torch.int32, device="cuda"),
            "bias_values": torch.arange(60000, device="cuda").float()[None]}
    check(logits_of(1, 100, "fp32", 4), same, "fp32")


def test_a_token_many_times():
    import torch
    tokens = torch.full((2, 200000), 5, dtype=torch.int32, device="cuda")
    r = {"tokens": tokens, "frequency": torch.full((2,), 0.001, device="cuda"),
         "repetition": torch.full((2,), 1.5, device="cuda"),
         "prompts": torch.tensor([0, 199999], dtype=torch.int32, device="cuda")}
    check(logits_of(2, 64, "fp32", 5), r, "fp32")


def test_offsets_past_32_bits():
    import torch

    from wide_bf16_row_gb300 import topk
    rows, cols = 9000, 248320
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    allowed = torch.full((rows, cols // 32), -1, dtype=torch.int32, device="cuda")
    allowed[-1, -1] = 1
    tokens = torch.full((rows, 1), cols - 32, dtype=torch.int32, device="cuda")
    topk.penalize_logits(x, tokens=tokens, presence=torch.full((rows,), 2.0, device="cuda"), allowed=allowed, out=x)
    assert bool((x[:, -32] == -2).all()) and bool((x[:-1, -31:] == 0).all()) and bool((x[-1, -31:] == -float("inf")).all())
    assert int((x != 0).sum()) == rows + 31


def test_refusals():
    import torch

    from wide_bf16_row_gb300 import topk
    x = logits_of(4, 100, "bf16", 1)
    r = request(4, 100, 10, 3, True, seed=1)
    for change in ({"tokens": r["tokens"].long()}, {"tokens": r["tokens"][:3]}, {"lengths": r["lengths"][:2]},
                   {"repetition": r["repetition"].double()}, {"bias_values": r["bias_values"][:, :2]},
                   {"bias_values": None}, {"allowed": r["allowed"][:, :3]}, {"tokens": r["tokens"].cpu()},
                   {"out": torch.empty(4, 100, device="cuda")}, {"out": torch.empty(4, 99, dtype=x.dtype, device="cuda")}):
        with pytest.raises(ValueError):
            topk.penalize_logits(x, **{**r, **change})
    with pytest.raises(TypeError):
        topk.penalize_logits(x.int())
    wide = {"bias_tokens": torch.zeros(1, 65536, dtype=torch.int32, device="cuda"),
            "bias_values": torch.zeros(1, 65536, device="cuda")}
    with pytest.raises(topk.TopkError) as e:
        topk.penalize_logits(x[:1], **wide)
    assert e.value.status == topk.ERR_SHAPE
    assert topk.penalize_logits(x[:0], **{n: t[:0] for n, t in r.items()}).shape == (0, 100)


def test_captured_and_on_another_stream():
    import torch

    from wide_bf16_row_gb300 import topk
    x, r = logits_of(6, 5000, "bf16", 1), request(6, 5000, 100, 4, True, seed=2)
    ref = topk.penalize_logits(x, **r)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = topk.penalize_logits(x, **r, stream=side)
    side.synchronize()
    assert torch.equal(got, ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = topk.penalize_logits(x, **r)
    x.copy_(logits_of(6, 5000, "bf16", 9))
    r["lengths"].fill_(100)
    graph.replay()
    assert torch.equal(kept, topk.penalize_logits(x, **r)) and not torch.equal(kept, ref)
