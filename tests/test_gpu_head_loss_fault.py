"""A bounded wait of the head's loss that runs out, on the GPU, without a fault.

The test build of the library (macro TF_TOPK_TEST_WAIT_TIMEOUT) makes the warp
that issues the products wait first for a barrier that nothing completes, 16 ms
at most.  The wait runs out, the code is recorded, the pair's other warps give
up, the copies in flight land, the tensor memory is freed and the kernel
returns.  The host reads the code through ``tf_topk_device_fault``; the context
and the stream stay usable, and the product library's results are what they
were.
"""
from __future__ import annotations

import time

import pytest

from tests.test_gpu_fault import FAULT_WAIT_TIMEOUT

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,dim,vocab", [(5, 1032, 3001), (100, 64, 700), (300, 520, 2049)])
def test_a_wait_that_runs_out_is_reported_and_the_next_calls_are_right(rows, dim, vocab):
    import torch

    from wide_bf16_row_gb300 import build, topk

    g = torch.Generator().manual_seed(rows)
    hidden = torch.randn(rows, dim, generator=g).bfloat16().cuda()
    weight = (torch.randn(vocab, dim, generator=g) / dim ** 0.5).bfloat16().cuda()
    target = torch.randint(0, vocab, (rows,), generator=g).cuda()
    grad = torch.rand(rows, generator=g).cuda()
    product = topk.library()
    loss, lse = topk.head_loss_bf16(hidden, weight, target)
    d_hidden, d_weight = topk.head_loss_grad_bf16(hidden, weight, target, lse, grad)
    assert topk.device_fault() == 0
    try:
        topk.LIBRARY, kept = build.build_variant("wait_timeout", ("TF_TOPK_TEST_WAIT_TIMEOUT",)), topk.LIBRARY
        topk._lib = None
        assert topk.device_fault() == 0
        for call in (lambda: topk.head_loss_bf16(hidden, weight, target),
                     lambda: topk.head_loss_grad_bf16(hidden, weight, target, lse, grad)):
            begun = time.monotonic()
            call()
            torch.cuda.synchronize()  # the kernels returned: no hang, no CUDA error
            assert time.monotonic() - begun < 5
            assert topk.device_fault() == FAULT_WAIT_TIMEOUT
            assert topk.device_fault() == 0  # reported once, then cleared
    finally:
        topk.LIBRARY, topk._lib = kept, product
    again = topk.head_loss_bf16(hidden, weight, target)
    assert torch.equal(again[0], loss) and torch.equal(again[1], lse)
    again = topk.head_loss_grad_bf16(hidden, weight, target, lse, grad)
    assert torch.equal(again[0], d_hidden) and torch.equal(again[1], d_weight)
    assert topk.device_fault() == 0
