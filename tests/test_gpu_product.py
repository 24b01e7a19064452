"""GPU parity of the product in 8 bits against the oracle in 64 bits.

Tolerance (u = 2^-24): the products of e4m3 values are exact.  A block's sum is
four additions of 32 products to an accumulator; an addition cuts each of its 33
terms below the last of 24 places of the largest, so that each is off by less
than 2u of a term that is at most the block's sum of magnitudes: 4 * 33 * 2 = 264
u.  The scales' product and each block's FMA add u, of the magnitudes' sum so
far.  Then one rounding to the result's type."""
from __future__ import annotations

import time

import numpy as np
import pytest

from oracle import tokens as oracle
from tests.test_gpu_fault import FAULT_WAIT_TIMEOUT

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


def _np(x):
    return x.double().cpu().numpy()


def inputs(rows, dim, cols, groups=None, seed=0):
    import torch
    g = torch.Generator().manual_seed(seed)
    lead = () if groups is None else (groups,)
    blocks, col_blocks = -(-dim // 128), -(-cols // 128)

    def eight(*shape):
        return (60 * torch.randn(*shape, generator=g)).clamp(-448, 448).to(torch.float8_e4m3fn).cuda()

    def scales(*shape):
        return (torch.rand(*shape, generator=g) + 0.1).cuda() * 0.01

    return eight(rows, dim), scales(rows, blocks), eight(*lead, cols, dim), scales(*lead, col_blocks, blocks)


def check(args, dtype, offsets=None):
    import torch

    from wide_bf16_row_gb300 import topk
    q, scale, weight, weight_scale = args
    at = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device="cuda")
    y = topk.product_fp8(*args, offsets=at, dtype=_dtype(dtype))
    assert y.dtype == _dtype(dtype) and y.shape == (q.shape[0], weight.shape[-2])
    ref, size = oracle.product(_np(q.float()), _np(scale), _np(weight.float()), _np(weight_scale), offsets)
    allow = torch.finfo(y.dtype).eps / 2 * np.abs(ref) + (264 + 1 + scale.shape[1]) * U * 1.01 * size + TINY[dtype]
    off = np.abs(_np(y) - ref)
    assert (off <= allow).all(), f"off by {np.max(off - allow)} at {np.argwhere(off > allow)[0]}"
    assert topk.device_fault() == 0
    return y


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,dim,cols", [(1, 16, 1), (1, 128, 128), (15, 2048, 1000), (16, 144, 129), (17, 1040, 257),
                                           (127, 112, 640), (128, 256, 256), (129, 256, 255), (256, 896, 512),
                                           (257, 400, 384), (700, 272, 1111), (2, 8192, 70)])
def test_one_matrix(dtype, rows, dim, cols):
    check(inputs(rows, dim, cols, seed=rows + dim), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("dim,cols,counts,behind", [
    (256, 130, [0, 3, 0, 0, 1], 0), (144, 512, [16, 17, 128, 129, 256, 257], 5), (64, 96, [1] * 70, 3),
    (528, 300, [0, 0, 0], 9), (128, 640, [5000, 0, 300], 40), (272, 272, [40, 400, 4, 0, 77], 1000), (16, 24, [3], 0),
    (1024, 128, [100] * 12, 0)])
def test_groups(dtype, dim, cols, counts, behind):
    offsets = np.concatenate([[0], np.cumsum(counts)]).tolist()
    args = inputs(offsets[-1] + behind, dim, cols, len(counts), seed=dim)
    y = check(args, dtype, offsets)
    assert not y[offsets[-1]:].any()


def test_1024_groups():
    rng = np.random.default_rng(1)
    counts = rng.integers(0, 4, 1024)
    counts[-1] = 2
    offsets = np.concatenate([[0], np.cumsum(counts)]).tolist()
    check(inputs(offsets[-1] + 7, 128, 136, 1024, seed=3), "bf16", offsets)


def test_a_long_sum_of_one_sign_keeps_its_digits():
    """8192 positive terms: no drift beyond the tolerance's first term, 32 digits' worth measured separately."""
    import torch
    q, s, w, ws = inputs(40, 8192, 256, seed=2)
    q, w = q.float().abs().to(q.dtype), w.float().abs().to(w.dtype)
    y = check((q, s, w, ws), "fp32")
    ref, _ = oracle.product(_np(q.float()), _np(s), _np(w.float()), _np(ws))
    assert np.linalg.norm(_np(y) - ref) <= 2e-6 * np.linalg.norm(ref)
    assert torch.isfinite(y).all()


def test_rows_keep_to_themselves():
    """NaN and infinite scales reach their own row alone, and a row's bits do not depend on the rows beside it."""
    import torch

    from wide_bf16_row_gb300 import topk
    q, s, w, ws = inputs(300, 400, 200, seed=4)
    y = topk.product_fp8(q, s, w, ws, dtype=torch.float32)
    bad = q.clone()
    bad.view(torch.uint8)[5, 100] = 0x7F
    worse = s.clone()
    worse[7, 1], worse[290, 0] = float("nan"), float("inf")
    z = topk.product_fp8(bad, worse, w, ws, dtype=torch.float32)
    touched = torch.zeros(300, dtype=torch.bool)
    touched[[5, 7, 290]] = True
    assert z[5].isnan().all() and z[7].isnan().all() and not z[290].isfinite().any()
    assert torch.equal(z[~touched.cuda()], y[~touched.cuda()])
    for rows in (1, 16, 17, 130):
        assert torch.equal(topk.product_fp8(q[:rows], s[:rows], w, ws, dtype=torch.float32), y[:rows])


def test_offsets_that_do_not_fit_do_not_read_or_write_out_of_range():
    import torch

    from wide_bf16_row_gb300 import topk
    args = inputs(100, 128, 128, 4, seed=5)
    raw = torch.full((102 * 128,), 7.0, device="cuda")
    out = raw[128:-128].view(100, 128)
    for offsets in ([0, 50, 20, 200, 90], [5, -3, 2**31 - 1, -2**31, 100], [100, 0, 0, 0, 0], [-5, 3, 3, 3, 1000]):
        topk.product_fp8(*args, offsets=torch.tensor(offsets, dtype=torch.int32, device="cuda"), out=out)
        torch.cuda.synchronize()
        assert bool((raw[:128] == 7).all()) and bool((raw[-128:] == 7).all()) and topk.device_fault() == 0


@pytest.mark.parametrize("dtype,cols,lead", [("bf16", 256, 1), ("bf16", 250, 3), ("fp32", 136, 1), ("fp16", 77, 0)])
def test_nothing_beside_the_output_is_written(dtype, cols, lead):
    import torch

    from wide_bf16_row_gb300 import topk
    args = inputs(150, 256, cols, 3, seed=6)
    at = torch.tensor([0, 10, 10, 140], dtype=torch.int32, device="cuda")
    ref = topk.product_fp8(*args, offsets=at, dtype=_dtype(dtype))
    raw = torch.full((150 * cols + 64 + lead,), 5.0, dtype=_dtype(dtype), device="cuda")
    out = raw[32 + lead:32 + lead + 150 * cols].view(150, cols)
    topk.product_fp8(*args, offsets=at, out=out)
    assert torch.equal(out, ref)
    assert bool((raw[:32 + lead] == 5).all()) and bool((raw[32 + lead + 150 * cols:] == 5).all())


def test_a_result_past_32_bits():
    import torch

    from wide_bf16_row_gb300 import topk
    rows, cols = 40000, 60000
    q, s, w, ws = inputs(rows, 16, cols, seed=7)
    y = topk.product_fp8(q, s, w, ws)
    assert y.numel() > 2**31
    for r in (0, 12345, rows - 1):
        ref, size = oracle.product(_np(q[r:r + 1].float()), _np(s[r:r + 1]), _np(w.float()), _np(ws))
        assert (np.abs(_np(y[r:r + 1]) - ref) <= 2.0 ** -8 * np.abs(ref) + 266 * U * 1.01 * size).all()


def test_refusals():
    import torch

    from wide_bf16_row_gb300 import topk
    q, s, w, ws = inputs(8, 64, 40, seed=1)
    gw, gs = inputs(8, 64, 40, 3, seed=1)[2:]
    at = torch.zeros(4, dtype=torch.int32, device="cuda")
    for call in (lambda: topk.product_fp8(q, s, w[:, :32], ws), lambda: topk.product_fp8(q, s[:, :0], w, ws),
                 lambda: topk.product_fp8(q, s, gw, gs), lambda: topk.product_fp8(q, s, w, ws, offsets=at),
                 lambda: topk.product_fp8(q, s, gw, gs, offsets=at[:3]), lambda: topk.product_fp8(q, s.double(), w, ws),
                 lambda: topk.product_fp8(q, s, gw, gs[:2], offsets=at), lambda: topk.product_fp8(q, s.cpu(), w, ws),
                 lambda: topk.product_fp8(q, s, w, ws, out=torch.empty(8, 41, device="cuda")),
                 lambda: topk.product_fp8(q.t(), s, w, ws)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        topk.product_fp8(q, s, w, ws, dtype=torch.float64)
    with pytest.raises(TypeError):
        topk.product_fp8(q.view(torch.uint8), s, w, ws)
    q, s, w, ws = inputs(8, 24, 40, seed=1)
    with pytest.raises(topk.TopkError) as e:
        topk.product_fp8(q, s, w, ws)
    assert e.value.status == topk.ERR_SHAPE


def test_captured_and_on_another_stream():
    import torch

    from wide_bf16_row_gb300 import topk
    args = inputs(500, 512, 384, 8, seed=8)
    at = torch.tensor([0, 1, 60, 60, 200, 300, 400, 450, 490], dtype=torch.int32, device="cuda")
    ref = topk.product_fp8(*args, offsets=at)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = topk.product_fp8(*args, offsets=at, stream=side)
    side.synchronize()
    assert torch.equal(got, ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = topk.product_fp8(*args, offsets=at)
    at.copy_(torch.tensor([0, 100, 100, 110, 200, 300, 420, 450, 500], dtype=torch.int32))
    graph.replay()
    assert torch.equal(kept, topk.product_fp8(*args, offsets=at)) and not torch.equal(kept, ref)


@pytest.mark.parametrize("rows", [10, 64, 300])
def test_a_wait_that_runs_out_is_reported_and_the_next_calls_are_right(rows):
    """In the test build the warp that issues the products waits first for a barrier that nothing completes, 16 ms at
    most; the kernel winds down, the code is read on the host, and the product library's results are what they were."""
    import torch

    from wide_bf16_row_gb300 import build, topk
    args = inputs(rows, 2608, 700, seed=9)
    product = topk.library()
    ref = topk.product_fp8(*args)
    assert topk.device_fault() == 0
    try:
        topk.LIBRARY, kept = build.build_variant("wait_timeout", ("TF_TOPK_TEST_WAIT_TIMEOUT",)), topk.LIBRARY
        topk._lib = None
        assert topk.device_fault() == 0
        begun = time.monotonic()
        topk.product_fp8(*args)
        torch.cuda.synchronize()
        assert time.monotonic() - begun < 5
        assert topk.device_fault() == FAULT_WAIT_TIMEOUT
        assert topk.device_fault() == 0
    finally:
        topk.LIBRARY, topk._lib = kept, product
    assert torch.equal(topk.product_fp8(*args), ref) and topk.device_fault() == 0
