"""Calls of the operators around an expert layer and before sampling that their
documentation allows and that meet other calls."""
from __future__ import annotations

import threading

import numpy as np
import pytest

from oracle import tokens as oracle
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
