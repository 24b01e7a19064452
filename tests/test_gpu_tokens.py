"""GPU parity of tokens sorted by expert and back, their gradients, and rows in
8 bits, against the oracle in 64 bits.

The order, gathered rows and rows in 8 bits are equal.  Tolerances of the rest,
from the kernels' fp32 arithmetic (u = 2^-24): a combined element is a chain of
k fused multiply-adds, each off by at most u times the sum of the terms'
magnitudes, then one rounding to its type (eps / 2, and half its smallest
step).  A row's gradient is one product (u) and that rounding.  A weight's
gradient is a chain of at most dim / 32 + 8 fused multiply-adds a lane, five
additions across lanes and up to eight across warps."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import tokens as oracle

pytestmark = pytest.mark.gpu

TYPES = ("bf16", "fp16", "fp32")
U = 2.0 ** -24
TINY = {"bf16": 1e-38, "fp16": 2.0 ** -25, "fp32": 1e-44}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from wide_bf16_row_gb300 import build
    build.build()


def _dtype(name):
    import torch
    return {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[name]


def _np(x):
    return x.double().cpu().numpy()


def _rand(shape, dtype, seed, stride=None, offset=0):
    """Values of `shape`, rows `stride` apart from an address `offset` elements in."""
    import torch
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(*shape, generator=g).to(_dtype(dtype))
    if stride is None and not offset:
        return x.cuda()
    stride = stride or shape[1]
    flat = torch.full((offset + shape[0] * stride + 8,), float("nan"), dtype=x.dtype, device="cuda")
    view = flat.as_strided(shape, (stride, 1), offset)
    view.copy_(x)
    return view


def _choices(tokens, k, experts, seed, lost=0.0):
    import torch
    g = torch.Generator().manual_seed(seed)
    idx = torch.randint(0, experts, (tokens, k), generator=g, dtype=torch.int32)  # an expert may come twice
    drop = torch.rand(tokens, k, generator=g) < lost
    bad = torch.tensor([-1, experts, -2**31, 2**31 - 1], dtype=torch.int32)[torch.randint(0, 4, (tokens, k), generator=g)]
    return torch.where(drop, bad, idx).cuda()


def near(got, ref, terms, size, dtype):
    import torch
    allow = torch.finfo(_dtype(dtype)).eps / 2 * np.abs(ref) + terms * U * 1.01 * size + TINY[dtype]
    off = np.abs(_np(got) - ref)
    assert (off <= allow).all(), f"off by {np.max(off - allow)} at {np.argwhere(off > allow)[0]}"


def sorted_as_the_oracle(idx, experts):
    from wide_bf16_row_gb300 import topk
    order = topk.sort_by_expert(idx, experts)
    slot, source, offsets = oracle.order(idx.cpu().numpy(), experts)
    assert np.array_equal(order.offsets.cpu().numpy(), offsets)
    assert np.array_equal(order.source.cpu().numpy(), source)
    assert np.array_equal(order.slot.cpu().numpy(), slot)
    return order, slot, source


@pytest.mark.parametrize("tokens,k,experts,lost", [
    (1, 1, 1, 0), (1, 8, 256, 0), (3, 5, 2, 0.5), (33, 1, 1024, 0), (1000, 8, 64, 0.1), (1024, 8, 128, 0),
    (1025, 8, 1024, 0.3), (257, 32, 60, 0), (5000, 3, 7, 1.0), (70000, 2, 256, 0.05), (40000, 32, 1000, 0),
    (8193, 1, 33, 0.2), (65536, 8, 256, 0), (300000, 4, 1, 0.5)])
def test_order(tokens, k, experts, lost):
    sorted_as_the_oracle(_choices(tokens, k, experts, tokens + k, lost), experts)


def test_order_of_one_expert_for_all_and_of_no_tokens():
    import torch

    from wide_bf16_row_gb300 import topk
    sorted_as_the_oracle(torch.full((20000, 4), 5, dtype=torch.int32, device="cuda"), 9)
    order = topk.sort_by_expert(torch.empty(0, 4, dtype=torch.int32, device="cuda"), 6)
    assert order.offsets.tolist() == [0] * 7 and order.slot.shape == (0, 4) and order.source.shape == (0,)
    x = torch.empty(0, 32, device="cuda")
    assert topk.gather_tokens(x, order).shape == (0, 32) and topk.combine_tokens(x, order).shape == (0, 32)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tokens,dim,k,experts,lost,stride,offset", [
    (1, 8, 1, 4, 0, None, 0), (1, 2048, 8, 256, 0, None, 0), (5, 1, 3, 6, 0.4, None, 0), (70, 1001, 5, 60, 0.2, None, 0),
    (300, 264, 8, 16, 0.1, 272, 0), (300, 264, 8, 16, 0.1, 273, 0), (41, 640, 32, 1024, 0.3, None, 1),
    (129, 514, 7, 3, 1.0, None, 0), (65, 4096, 9, 40, 0.05, 4100, 4), (2000, 96, 2, 128, 0.5, None, 0),
    (17, 8200, 4, 8, 0, None, 0)])
def test_there_and_back(dtype, tokens, dim, k, experts, lost, stride, offset):
    import torch

    from wide_bf16_row_gb300 import topk
    order, slot, source = sorted_as_the_oracle(_choices(tokens, k, experts, dim, lost), experts)
    x = _rand((tokens, dim), dtype, 1, stride, offset)
    rows = topk.gather_tokens(x, order)
    assert rows.dtype == x.dtype and np.array_equal(_np(rows), oracle.gather(_np(x), source, k))

    y = _rand((tokens * k, dim), dtype, 2, stride, offset)
    y[torch.from_numpy(source < 0).cuda()] = float("nan")  # rows that no choice has are not read
    weight = torch.randn(tokens, k, generator=torch.Generator().manual_seed(3)).cuda()
    weight[torch.from_numpy(slot < 0).cuda()] = float("nan")
    ref, size = oracle.combine(_np(y), slot, _np(weight))
    near(topk.combine_tokens(y, order, weight), ref, k, size, dtype)
    ref, size = oracle.combine(_np(y), slot)
    near(topk.gather_tokens_grad(y, order), ref, k, size, dtype)

    grad = _rand((tokens, dim), dtype, 4, stride, offset)
    d_rows, d_weight = topk.combine_tokens_grad(grad, y, order, weight)
    ref_rows, ref_weight, size = oracle.combine_grad(_np(grad), _np(y), slot, _np(weight))
    ref_rows[source < 0] = 0
    near(d_rows, ref_rows, 1, np.abs(ref_rows), dtype)
    near(d_weight, ref_weight, dim / 32 + 8 + 5 + 8, size, "fp32")
    if dim <= 600 and dim % 16 == 0:
        again = topk.combine_tokens_grad(grad, y, order, weight)
        assert torch.equal(again[0], d_rows) and torch.equal(again[1], d_weight)


def test_combine_gradient_is_the_slope():
    import torch

    from wide_bf16_row_gb300 import topk
    idx = _choices(9, 3, 4, 8, 0.2)
    order = topk.sort_by_expert(idx, 4)
    y, grad = _rand((27, 20), "fp32", 1), _rand((9, 20), "fp32", 2)
    weight = _rand((9, 3), "fp32", 3)
    d_rows, d_weight = topk.combine_tokens_grad(grad, y, order, weight)
    # the result is linear in either: a step of 1 gives the slope but for its roundings
    for x, d in ((y, d_rows), (weight, d_weight)):
        for at in ((0, 0), (4, 2), (8, 1)):
            up = x.clone()
            up[at] += 1
            ends = [topk.combine_tokens(up if x is y else y, order, up if x is weight else weight),
                    topk.combine_tokens(y, order, weight)]
            slope = ((ends[0].double() - ends[1].double()) * grad.double()).sum()
            assert abs(float(slope - d[at])) < 1e-4


def test_a_token_s_results_do_not_depend_on_the_others():
    import torch

    from wide_bf16_row_gb300 import topk
    idx = _choices(500, 4, 16, 1)
    y, grad, weight = _rand((2000, 1000), "bf16", 1), _rand((500, 1000), "bf16", 2), _rand((500, 4), "fp32", 3)
    order = topk.sort_by_expert(idx, 16)
    out, (_, d_weight) = topk.combine_tokens(y, order, weight), topk.combine_tokens_grad(grad, y, order, weight)
    one = topk.sort_by_expert(idx[7:8].contiguous(), 16)
    mine = torch.empty(4, 1000, dtype=y.dtype, device="cuda")
    mine[one.slot[0].long()] = y[order.slot[7].long()]
    assert torch.equal(topk.combine_tokens(mine, one, weight[7:8].contiguous()), out[7:8])
    assert torch.equal(topk.combine_tokens_grad(grad[7:8], mine, one, weight[7:8].contiguous())[1], d_weight[7:8])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tokens,dim,k,stride,offset", [(1, 16, 1, None, 0), (7, 128, 2, None, 0), (33, 1040, 3, None, 0),
                                                        (64, 2048, 8, 2052, 0), (9, 272, 4, 273, 1), (500, 144, 1, None, 0)])
def test_rows_in_8_bits(dtype, tokens, dim, k, stride, offset):
    import torch

    from wide_bf16_row_gb300 import topk
    x = _rand((tokens, dim), dtype, dim, stride, offset)
    x[0, :min(dim, 128)] = 0
    if tokens > 6:
        x[1] *= 1000
        x[2] *= 1e-4
        x[3, 5] = float("nan")
        x[4, dim - 1] = float("-inf")
        x[5, :16] = torch.tensor([448, 17, 19, 1, 2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -10, 0, -448, -17, -19, -1, 416, 432,
                                  440, 24]).to(x.dtype)
    q, scale = topk.quantize_tokens_fp8(x)
    ref_q, ref_scale = oracle.quantize(x.float().cpu().numpy())
    assert np.array_equal(scale.cpu().numpy(), ref_scale, equal_nan=True)
    assert np.array_equal(_np(q.float()), ref_q, equal_nan=True)
    order, _, source = sorted_as_the_oracle(_choices(tokens, k, 5, 2, 0.2), 5)
    q, scale = topk.quantize_tokens_fp8(x, order)
    assert np.array_equal(scale.cpu().numpy(), oracle.gather(ref_scale, source, k), equal_nan=True)
    assert np.array_equal(_np(q.float()), oracle.gather(ref_q, source, k), equal_nan=True)


def test_rows_in_8_bits_of_the_smallest_numbers():
    import torch

    from wide_bf16_row_gb300 import topk
    x = torch.zeros(3, 256, device="cuda")
    x[0, 3], x[1, 200], x[2, 7] = 2.0 ** -149, -2.0 ** -101, 3.4e38
    q, scale = topk.quantize_tokens_fp8(x)
    ref_q, ref_scale = oracle.quantize(x.cpu().numpy())
    assert np.array_equal(scale.cpu().numpy(), ref_scale) and np.array_equal(_np(q.float()), ref_q)


def test_offsets_past_32_bits():
    """Rows whose elements pass 2^31, forward and backward, against torch's indexing."""
    import torch

    from wide_bf16_row_gb300 import topk
    tokens, dim, k = 36000, 8192, 8
    order = topk.sort_by_expert(_choices(tokens, k, 64, 5), 64)
    x = torch.randn(tokens, dim, device="cuda", dtype=torch.bfloat16)
    rows = topk.gather_tokens(x, order)
    for lo in range(0, tokens * k, 32000):
        at = order.source[lo:lo + 32000].long()
        assert torch.equal(rows[lo:lo + 32000], x[at // k])
    ones = torch.ones(tokens, k, device="cuda")
    assert torch.equal(topk.combine_tokens(rows, order, ones / 8), x)  # eight eighths, exactly
    d_rows, d_weight = topk.combine_tokens_grad(x, rows, order, ones)
    assert torch.equal(d_rows, rows)
    square = (x.double() ** 2).sum(1)
    assert bool(((d_weight.double() - square[:, None]).abs() <= (dim / 32 + 21) * U * square[:, None]).all())
    assert topk.device_fault() == 0


def test_nothing_beside_the_outputs_is_written():
    import torch

    from wide_bf16_row_gb300 import topk
    tokens, dim, k, experts = 2100, 40, 4, 9

    def guarded(shape, dtype):
        n = int(np.prod(shape))
        raw = torch.zeros(n + 64, dtype=dtype, device="cuda")
        raw.view(torch.uint8).fill_(0x5A)
        return raw, raw[32:32 + n].view(shape)

    def intact(raw):
        b, side = raw.view(torch.uint8), 32 * raw.element_size()
        return bool((b[:side] == 0x5A).all()) and bool((b[-side:] == 0x5A).all())

    idx = _choices(tokens, k, experts, 1, 0.1)
    kept = [guarded((tokens, k), torch.int32), guarded((tokens * k,), torch.int32), guarded((experts + 1,), torch.int32)]
    need = topk.tf_topk_sort_experts_workspace(tokens, k, experts)
    assert need > 0
    space = guarded((need,), torch.uint8)
    order = topk.sort_by_expert(idx, experts, out=[v for _, v in kept], workspace=space[1])
    x = _rand((tokens, dim), "bf16", 1)
    weight = torch.rand(tokens, k, device="cuda")
    kept += [space] + [guarded(s, t) for s, t in (((tokens * k, dim), x.dtype), ((tokens, dim), x.dtype),
                                                  ((tokens * k, dim), x.dtype), ((tokens, k), torch.float32))]
    rows = topk.gather_tokens(x, order, out=kept[4][1])
    topk.combine_tokens(rows, order, weight, out=kept[5][1])
    topk.combine_tokens_grad(x, rows, order, weight, out=(kept[6][1], kept[7][1]))
    wide = _rand((tokens, 48), "bf16", 1)
    kept += [guarded((tokens * k, 48), torch.float8_e4m3fn), guarded((tokens * k, 1), torch.float32)]
    topk.quantize_tokens_fp8(wide, order, out=(kept[8][1], kept[9][1]))
    torch.cuda.synchronize()
    assert all(intact(raw) for raw, _ in kept)
    small = torch.empty(need - 4, dtype=torch.uint8, device="cuda")
    with pytest.raises(topk.TopkError) as e:
        topk.sort_by_expert(idx, experts, workspace=small)
    assert e.value.status == topk.ERR_SCRATCH


def test_refusals():
    import torch

    from wide_bf16_row_gb300 import topk
    idx = _choices(10, 2, 4, 1)
    order = topk.sort_by_expert(idx, 4)
    x = _rand((10, 32), "bf16", 1)
    rows = topk.gather_tokens(x, order)
    for call in (lambda: topk.gather_tokens(x[:9], order), lambda: topk.gather_tokens(x.t(), order),
                 lambda: topk.combine_tokens(x, order), lambda: topk.combine_tokens(rows, order, torch.ones(10, 2)),
                 lambda: topk.combine_tokens(rows, order, torch.ones(10, 3, device="cuda")),
                 lambda: topk.combine_tokens_grad(x.half(), rows, order, torch.ones(10, 2, device="cuda")),
                 lambda: topk.gather_tokens(x, order, out=rows[:, :16]), lambda: topk.sort_by_expert(idx.t(), 4),
                 lambda: topk.sort_by_expert(idx, 4, out=order[:2] + (order.offsets[:4],)),
                 lambda: topk.quantize_tokens_fp8(x, order, out=(rows, rows))):
        with pytest.raises(ValueError):
            call()
    for call, status in ((lambda: topk.sort_by_expert(idx, 0), topk.ERR_SHAPE),
                         (lambda: topk.sort_by_expert(idx, 1025), topk.ERR_SHAPE),
                         (lambda: topk.sort_by_expert(_choices(4, 33, 4, 1), 4), topk.ERR_K),
                         (lambda: topk.quantize_tokens_fp8(_rand((4, 24), "bf16", 1)), topk.ERR_SHAPE)):
        with pytest.raises(topk.TopkError) as e:
            call()
        assert e.value.status == status


def test_other_streams_and_a_captured_step():
    """A forward and backward pass on a side stream, then captured and replayed on new values."""
    import torch

    from wide_bf16_row_gb300 import topk
    tokens, dim, k, experts = 3000, 128, 4, 32
    idx, x = _choices(tokens, k, experts, 1, 0.1), _rand((tokens, dim), "bf16", 1)
    weight, grad = torch.rand(tokens, k, device="cuda"), _rand((tokens, dim), "bf16", 2)

    def step(stream=None):
        order = topk.sort_by_expert(idx, experts, stream=stream)
        rows = topk.gather_tokens(x, order, stream=stream)
        out = topk.combine_tokens(rows, order, weight, stream=stream)
        d_rows, d_weight = topk.combine_tokens_grad(grad, rows, order, weight, stream=stream)
        return (*order, rows, out, d_rows, d_weight, topk.gather_tokens_grad(d_rows, order, stream=stream))

    def same(a, b):
        return all(torch.equal(p, q) for p, q in zip(a, b))

    first = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(side)
    side.synchronize()
    assert same(got, first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = step()
    idx.copy_(_choices(tokens, k, experts, 9, 0.2))
    x.copy_(_rand((tokens, dim), "bf16", 9))
    graph.replay()
    torch.cuda.synchronize()
    assert same(kept, step()) and not torch.equal(kept[3], first[3])
