"""Seeded random shapes, strides, types and values of the operators around an
expert layer and before sampling, against their oracles, with the tolerances of
their own tests; several calls at once on several streams; sizes at which a
kernel or a table changes."""
from __future__ import annotations

import random

import numpy as np
import pytest

from oracle import tokens as oracle
from tests import test_gpu_penalty as penalty
from tests import test_gpu_product as product
from tests import test_gpu_tokens as tokens

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from wide_bf16_row_gb300 import build
    build.build()


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


@pytest.mark.parametrize("seed", range(24))
def test_tokens(seed):
    rng = random.Random(seed)
    dim = _log(rng, 1, 3000)
    stride = rng.choice((None, dim + rng.randint(0, 9)))
    tokens.test_there_and_back(rng.choice(tokens.TYPES), _log(rng, 1, 600), dim, rng.randint(1, 12), _log(rng, 1, 1024),
                               rng.choice((0, 0.1, 0.9)), stride, rng.choice((0, 0, 1, 2, 8)))


@pytest.mark.parametrize("seed", range(16))
def test_orders(seed):
    rng = random.Random(100 + seed)
    k, experts = rng.randint(1, 32), _log(rng, 1, 1024)
    tokens.sorted_as_the_oracle(tokens._choices(_log(rng, 1, 200000 // k), k, experts, seed, rng.choice((0, 0.3))), experts)


@pytest.mark.parametrize("seed", range(24))
def test_products(seed):
    rng = random.Random(200 + seed)
    dim, cols = 16 * _log(rng, 1, 130), _log(rng, 1, 1500)
    groups = rng.choice((None, _log(rng, 1, 40)))
    if groups is None:
        product.check(product.inputs(_log(rng, 1, 700), dim, cols, seed=seed), rng.choice(product.TYPES))
        return
    most = rng.choice((3, 40, 300))
    counts = [rng.choice((0, rng.randint(0, most))) for _ in range(groups)]
    offsets = np.concatenate([[0], np.cumsum(counts)]).tolist()
    product.check(product.inputs(offsets[-1] + rng.choice((0, 7)) + 1, dim, cols, groups, seed=seed),
                  rng.choice(product.TYPES), offsets)


@pytest.mark.parametrize("rows,dim,cols", [(16, 144, 40000), (5, 272, 50003), (64, 128, 39000), (64, 256, 300),
                                           (65, 256, 300), (48, 16, 20016), (300, 128, 136), (257, 128, 2056)])
def test_products_where_the_tiles_change(rows, dim, cols):
    """Narrow tiles that cross the weight's scale blocks, the last rows of the thin kernel, results of 16-byte rows."""
    product.check(product.inputs(rows, dim, cols, seed=rows), "bf16")


@pytest.mark.parametrize("seed", range(24))
def test_penalties(seed):
    rng = random.Random(300 + seed)
    dtype, cols, rows = rng.choice(penalty.TYPES), _log(rng, 1, 60000), _log(rng, 1, 30)
    width, biases = rng.choice((0, _log(rng, 1, 12000))), rng.choice((0, _log(rng, 1, 400)))
    x = penalty.logits_of(rows, cols, dtype, seed, rng.choice((None, cols + rng.randint(0, 9))), rng.choice((0, 0, 1, 8)))
    r = penalty.request(rows, cols, width, biases, rng.random() < 0.5, seed=seed,
                        token_stride=rng.choice((None, width + 1 + rng.randint(0, 3))) if width else None)
    penalty.check(x, r, dtype, **({"out": x} if rng.random() < 0.3 else {}))


@pytest.mark.parametrize("width,biases", [(8192, 0), (8193, 0), (8000, 192), (8000, 193), (127, 1), (128, 0), (129, 0)])
def test_penalties_where_the_table_changes(width, biases):
    """As many distinct tokens as the tables of either kind hold, at their fullest."""
    import torch
    cols = 100003
    r = penalty.request(3, cols, width, biases, True, seed=width)
    r["tokens"] = torch.stack([torch.randperm(cols, generator=torch.Generator().manual_seed(s))[:width].int()
                               for s in range(3)]).cuda()
    for name in ("lengths", "prompts"):
        r[name] = torch.tensor([width, width, width // 2], dtype=torch.int32, device="cuda")
    r["repetition"][:] = 1.5
    penalty.check(penalty.logits_of(3, cols, "fp32", 1), r, "fp32")


def test_calls_on_several_streams_at_once():
    """Each stream's calls keep to their own inputs, outputs and workspaces."""
    import torch

    from wide_bf16_row_gb300 import topk

    def step(seed, stream):
        idx = tokens._choices(6000, 4, 64, seed, 0.1)
        x = tokens._rand((6000, 256), "bf16", seed)
        q, s, w, ws = product.inputs(1, 256, 384, 64, seed=seed)
        logits = penalty.logits_of(50, 20001, "bf16", seed)
        r = penalty.request(50, 20001, 700, 9, True, seed=seed)
        torch.cuda.synchronize()

        def run():
            order = topk.sort_by_expert(idx, 64, stream=stream)
            q, s = topk.quantize_tokens_fp8(x, order, stream=stream)
            y = topk.product_fp8(q, s, w, ws, offsets=order.offsets, stream=stream)
            out = topk.combine_tokens(y, order, stream=stream)
            few = topk.product_fp8(q[:20], s[:20], w[0], ws[0], stream=stream)
            return order.slot, y, out, few, topk.penalize_logits(logits, **r, stream=stream)
        return run

    streams = [torch.cuda.Stream() for _ in range(4)]
    runs = [step(i, s) for i, s in enumerate(streams)]
    alone = []
    for run in runs:
        alone.append([t.clone() for t in run()])
        torch.cuda.synchronize()
    for _ in range(5):
        got = [run() for run in runs]
    torch.cuda.synchronize()
    for a, b in zip(alone, got):
        assert all(torch.equal(p, q) for p, q in zip(a, b))
    assert topk.device_fault() == 0
    assert np.array_equal(alone[0][0].cpu().numpy(), oracle.order(tokens._choices(6000, 4, 64, 0, 0.1).cpu().numpy(), 64)[0])
