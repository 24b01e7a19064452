"""Calls of the operators around an expert layer and before sampling that their
documentation allows and that meet other calls."""
from __future__ import annotations

import ctypes
import threading

import numpy as np
import pytest

from oracle import tokens as oracle
from tests import test_gpu_product as product
from tests import test_gpu_tokens as tokens

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from wide_bf16_row_gb300 import build
    build.build()


def test_orders_from_several_host_threads():
    """Calls that need different amounts of shared memory, each thread on a stream
    of its own; up to 8192 choices take one launch, more take two."""
    import torch

    from wide_bf16_row_gb300 import topk
    work = []
    for i, (n, k, experts) in enumerate(((1000, 8, 1024), (1000, 8, 400), (5000, 4, 1000), (5000, 4, 330))):
        idx, stream = tokens._choices(n, k, experts, i, 0.1), torch.cuda.Stream()
        out = topk.sort_by_expert(idx, experts)
        space = torch.empty(max(topk.tf_topk_sort_experts_workspace(n, k, experts), 4), dtype=torch.uint8, device="cuda")
        work.append((idx, experts, out, stream, space, (idx.data_ptr(), n, k, experts, space.data_ptr(), space.nbytes,
                                                        *(t.data_ptr() for t in out), stream.cuda_stream)))
    for t in (t for w in work for t in w[2]):
        t.fill_(-7)
    torch.cuda.synchronize()
    start, status = threading.Barrier(len(work)), [[] for _ in work]

    def calls(i):
        start.wait()
        for n in range(10000):
            status[i].append(topk.tf_topk_sort_experts(*work[i][5]))
            if n % 200 == 0:  # not so far ahead that the launches queue up
                work[i][3].synchronize()

    threads = [threading.Thread(target=calls, args=(i,)) for i in range(len(work))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert [sum(s != topk.OK for s in each) for each in status] == [0] * len(work)
    for idx, experts, out, *_ in work:
        for got, ref in zip(out, oracle.order(idx.cpu().numpy(), experts)):
            assert np.array_equal(got.cpu().numpy(), ref)


def test_sizes_past_32_bits_are_refused():
    """2^32 and a little more: what 32 bits hold of it would be a size that runs."""
    import torch

    from wide_bf16_row_gb300 import topk
    idx, logits = tokens._choices(4, 2, 8, 1), tokens._rand((1, 64), "bf16", 2)
    one = topk.sort_by_expert(idx[:1, :1].contiguous(), 8)
    raw = torch.zeros(2**32 + 16, dtype=torch.int32, device="cuda")
    wide = raw.view(torch.bfloat16)[:2**32 + 16].view(1, -1)
    eight = raw.view(torch.float8_e4m3fn)[:2**32 + 16].view(1, -1)
    scale, weight = torch.ones(1, 2**25 + 1, device="cuda"), torch.ones(1, 1, device="cuda")
    many = raw.view(1, -1)
    for call in (lambda: topk.sort_by_expert(idx, 2**32 + 8), lambda: topk.sort_by_expert(idx, 8 - 2**32),
                 lambda: topk.gather_tokens(wide, one, out=wide),
                 lambda: topk.quantize_tokens_fp8(wide, out=(eight, scale)),
                 lambda: topk.combine_tokens(wide, one, weight, out=wide),
                 lambda: topk.combine_tokens_grad(wide, wide, one, weight, out=(wide, weight)),
                 lambda: topk.product_fp8(eight, scale, eight, scale),
                 lambda: topk.penalize_logits(logits, tokens=many, frequency=weight[0]),
                 lambda: topk.penalize_logits(logits, bias_tokens=many, bias_values=many.view(torch.float32))):
        with pytest.raises(topk.TopkError) as e:
            call()
        assert e.value.status == topk.ERR_SHAPE


def test_a_failed_call_leaves_nothing_to_the_next():
    """A call on a stream whose capture has become invalid fails; the calls after it do not report its error."""
    import torch

    from wide_bf16_row_gb300 import topk
    x = tokens._rand((50, 32), "bf16", 1)
    order = topk.sort_by_expert(tokens._choices(50, 2, 8, 1), 8)
    rows = torch.zeros(100, 32, dtype=x.dtype, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    driver, stream, graph = ctypes.CDLL("libcuda.so.1"), ctypes.c_void_p(side.cuda_stream), ctypes.c_void_p()
    assert driver.cuStreamBeginCapture_v2(stream, 2) == 0  # relaxed: nothing else is held back
    assert driver.cuStreamSynchronize(stream) != 0  # not allowed in a capture, and the end of this one
    try:
        with pytest.raises(topk.TopkError) as e:
            topk.gather_tokens(x, order, out=rows, stream=side)
    finally:
        assert driver.cuStreamEndCapture(stream, ctypes.byref(graph)) != 0
    assert e.value.status == topk.ERR_CUDA and not rows.any()
    topk.gather_tokens(x, order, out=rows)
    assert np.array_equal(tokens._np(rows), oracle.gather(tokens._np(x), order.source.cpu().numpy(), 2))
    assert topk.device_fault() == 0


@pytest.mark.parametrize("rows,groups,dim,cols", [(100, 4, 272, 136), (400, 4, 128, 264), (3000, 1024, 32, 40),
                                                  (60000, 1024, 32, 136), (700, 7, 144, 77)])
def test_offsets_that_run_backwards_give_no_row_to_two_groups(rows, groups, dim, cols):
    """Each is held to the rows there are, and counts as the largest before it where it is lower."""
    import torch

    from wide_bf16_row_gb300 import topk
    args = product.inputs(rows, dim, cols, groups, seed=rows)
    rng = np.random.default_rng(rows)
    turns = np.where(np.arange(groups + 1) % 2, rows, 0)
    for offsets in (turns, turns[::-1], rng.integers(-9, rows + 9, groups + 1), np.sort(rng.integers(0, rows, groups + 1)),
                    np.full(groups + 1, -2**31), np.full(groups + 1, 2**31 - 1)):
        held = np.clip(offsets, 0, rows)
        held[0] = 0
        held = np.maximum.accumulate(held)
        y, ref = (topk.product_fp8(*args, offsets=torch.from_numpy(o.astype(np.int32)).cuda()) for o in (offsets, held))
        assert torch.equal(y, ref) and not y[held[-1]:].any()
    product.check(args, "bf16", held.tolist())
    assert topk.device_fault() == 0


@pytest.mark.parametrize("rows,hot,share", [(512, 8, 0.9), (4096, 1, 0.5), (6000, 3, 0.7), (8192, 1, 0.6)])
def test_routing_that_favours_few_experts(rows, hot, share):
    """Groups of many times the average, in tiles of either kernel."""
    rng = np.random.default_rng(rows)
    counts = rng.multinomial(rows - hot * int(rows * share / hot), np.ones(128) / 128)
    counts[rng.permutation(128)[:hot]] += int(rows * share / hot)
    product.check(product.inputs(rows + 5, 272, 392, 128, seed=rows), "bf16", np.concatenate([[0], np.cumsum(counts)]).tolist())


def test_a_layer_from_several_host_threads():
    """Each thread's calls on its own stream give the bits that they give alone."""
    import torch

    from tests import test_gpu_penalty as penalty
    from wide_bf16_row_gb300 import topk

    def of(seed):
        experts, stream = (16, 500, 1000, 64)[seed], torch.cuda.Stream()
        idx, x = tokens._choices(700 * (seed + 1), 4, experts, seed, 0.1), tokens._rand((700 * (seed + 1), 256), "bf16", seed)
        _, _, w, ws = product.inputs(1, 256, 136 + seed, experts, seed=seed)
        logits, r = penalty.logits_of(9, 20001, "bf16", seed), penalty.request(9, 20001, 300 * 10**(seed % 3), 5, True, seed)

        def run():
            order = topk.sort_by_expert(idx, experts, stream=stream)
            q, s = topk.quantize_tokens_fp8(x, order, stream=stream)
            y = topk.product_fp8(q, s, w, ws, offsets=order.offsets, stream=stream)
            out = topk.combine_tokens(y, order, stream=stream)
            grads = topk.combine_tokens_grad(out, y, order, share, stream=stream)
            return (*order, y, out, *grads, topk.gather_tokens_grad(grads[0], order, stream=stream),
                    topk.penalize_logits(logits, **r, stream=stream))

        share = torch.ones(idx.shape, device="cuda")
        return run, stream

    work = [of(seed) for seed in range(4)]
    torch.cuda.synchronize()
    alone = []
    for run, stream in work:
        alone.append(run())
        stream.synchronize()
    start, got = threading.Barrier(len(work)), [[] for _ in work]

    def calls(i):
        run, stream = work[i]
        start.wait()
        for _ in range(50):
            last = run()
        stream.synchronize()
        got[i].extend(last)

    threads = [threading.Thread(target=calls, args=(i,)) for i in range(len(work))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for a, b in zip(alone, got):
        assert len(a) == len(b) and all(torch.equal(p, q) for p, q in zip(a, b))
    assert topk.device_fault() == 0
