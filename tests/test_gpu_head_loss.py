"""GPU parity of the head's loss and its gradient against the 64-bit oracle.

Tolerances (u = 2^-24).  The tensor cores add 16 products at a time to a
running fp32 sum and truncate, so a logit is off by at most (dim / 16 + 2) *
2^-23 * sum |h w| (`logit_error`); exp2, the sums of up to a few hundred terms
per thread and of a few thousand per row add below 1e-5 relative to the sum of
exponentials, so lse and loss are within twice the logit error + 1e-5 + 4 u of
their own size.  G's entries are off by that relative to p, then rounded to
bf16 (2^-8 at most), and the products' fp32 sums of K terms truncate by
(K / 16 + 2) * 2^-23 of the sum of magnitudes; the gradients are rounded once
more (2^-8).  The roundings of different terms are independent, so a second
check holds the 2-norm of the error against their sum in squares (with a
factor 2)."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import head_loss as oracle_loss

pytestmark = pytest.mark.gpu

HALF = 2.0 ** -8  # half a step of bf16, relative


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from wide_bf16_row_gb300 import build
    build.build()


def _inputs(rows, dim, vocab, seed, ignored=0.0, peak=6.0, hidden_pad=0, weight_pad=0, wide=True):
    import torch
    g = torch.Generator().manual_seed(seed)
    weight = (torch.randn(vocab, dim + weight_pad, generator=g) * dim ** -0.5 * 2).bfloat16()
    target = torch.randint(0, vocab, (rows,), generator=g)
    lean = peak * torch.rand(rows, 1, generator=g)
    hidden = torch.randn(rows, dim + hidden_pad, generator=g)
    hidden[:, :dim] += lean * weight[target, :dim].float() / 4
    hidden = hidden.bfloat16()
    target[torch.rand(rows, generator=g) < ignored] = -100
    return hidden.cuda()[:, :dim], weight.cuda()[:, :dim], (target if wide else target.int()).cuda()


def _np(t):
    return t.detach().double().cpu().numpy()


def logit_error(h, w):
    """Per row, the most any logit of it is off."""
    dim = h.shape[1]
    with np.errstate(invalid="ignore"):
        return (dim / 16 + 2) * 2.0 ** -23 * (np.abs(h) @ np.abs(w).T).max(1)


def check_loss(hidden, weight, target, loss, lse, ignore=-100):
    h, w, t = _np(hidden), _np(weight), target.cpu().numpy()
    ref_loss, ref_lse = oracle_loss.loss(h, w, t, ignore)
    allow = 2 * logit_error(h, w) + 1e-5
    for got, ref, name in ((_np(loss), ref_loss, "loss"), (_np(lse), ref_lse, "lse")):
        assert np.array_equal(np.isnan(got), np.isnan(ref)), name
        ok = ~np.isnan(ref)
        off = np.abs(got - ref)[ok]
        assert (off <= (allow + 4 * 2.0 ** -24 * np.abs(ref))[ok]).all(), (name, off.max())
    assert (_np(loss)[t == ignore] == 0).all() and (_np(lse)[t == ignore] == 0).all()


def check_grad(hidden, weight, target, g, d_hidden, d_weight, ignore=-100):
    h, w, t = _np(hidden), _np(weight), target.cpu().numpy()
    ref_h, ref_w, G = oracle_loss.grad(np.nan_to_num(h), w, t, _np(g), ignore)
    counts = (t != ignore) & (t >= 0) & (t < len(w))
    h = np.where(counts[:, None], np.nan_to_num(h), 0.0)
    hot = np.zeros_like(G)
    hot[np.flatnonzero(counts), t[counts]] = 1
    # an entry of G = g (p - hot): p's relative error, and the rounding to bf16; exp2 and the entry relative to the
    # largest |g| are flushed to 0 below the normal range, so either is off by up to 2^-126 times the largest |g|
    entry = 2.0 ** -125 * np.abs(_np(g)).max() + HALF * np.abs(G) + (2 * logit_error(h, w) + 1e-5)[:, None] * np.abs(G + hot * _np(g)[:, None])
    for got, ref, terms, name in ((d_hidden, ref_h, lambda e: e @ np.abs(w), "d_hidden"),
                                  (d_weight, ref_w, lambda e: e.T @ np.abs(h), "d_weight")):
        if got is None:
            continue
        got = _np(got)
        k = len(w) if name == "d_hidden" else len(h)
        trunc = (k / 16 + 34) * 2.0 ** -23
        allow = terms(entry) + trunc * terms(np.abs(G)) + HALF * np.abs(ref) + 1e-37
        off = np.abs(got - ref)
        assert (off <= allow).all(), (name, np.argwhere(off > allow)[0], (off - allow).max())
        squares = (entry ** 2) @ (w ** 2) if name == "d_hidden" else (entry ** 2).T @ (h ** 2)
        norm = 2 * np.sqrt(squares.sum() + (HALF ** 2 * ref ** 2).sum()) + np.linalg.norm(trunc * terms(np.abs(G)))
        assert np.linalg.norm(off) <= norm + 1e-37, (name, np.linalg.norm(off), norm)


def run(hidden, weight, target, g=None, ignore=-100, least=False, seed=0, **want):
    import torch

    from wide_bf16_row_gb300 import topk
    rows, dim = hidden.shape
    loss, lse = topk.head_loss_bf16(hidden, weight, target, ignore_index=ignore)
    check_loss(hidden, weight, target, loss, lse, ignore)
    if g is None:
        g = torch.randn(rows, generator=torch.Generator().manual_seed(seed)).cuda()
    space = None
    if least:
        space = torch.empty(topk.tf_topk_head_loss_grad_bf16_workspace(rows, dim, len(weight), True),
                            dtype=torch.uint8, device="cuda")
    dh, dw = topk.head_loss_grad_bf16(hidden, weight, target, lse, g, ignore_index=ignore, workspace=space, **want)
    check_grad(hidden, weight, target, g, dh, dw, ignore)
    assert topk.device_fault() == 0
    return loss, lse, dh, dw


@pytest.mark.parametrize("rows,dim,vocab", [(1, 8, 1), (1, 64, 7), (3, 8, 100), (1, 2048, 4096), (15, 256, 3001),
                                            (16, 264, 2048), (127, 72, 999), (128, 128, 1024), (129, 512, 513),
                                            (256, 520, 255), (257, 320, 2049), (300, 1032, 777), (513, 200, 4100),
                                            (700, 64, 1500)])
def test_sizes(rows, dim, vocab):
    run(*_inputs(rows, dim, vocab, seed=rows + dim + vocab, wide=rows % 2 == 0))


def test_rows_beyond_one_block():
    """More rows than the loss takes at a time, a ragged last block; the workspace it asks for is enough and one byte
    less than it needs is refused."""
    import torch

    from wide_bf16_row_gb300 import topk
    rows = 16384 + 77
    hidden, weight, target = _inputs(rows, 64, 300, seed=4, ignored=0.1)
    loss, lse, dh, dw = run(hidden, weight, target)
    again = topk.head_loss_bf16(hidden[16384:], weight, target[16384:])
    assert torch.equal(loss[16384:], again[0]) and torch.equal(lse[16384:], again[1])
    small = torch.empty(1024, dtype=torch.uint8, device="cuda")
    for call in (lambda: topk.head_loss_bf16(hidden, weight, target, workspace=small),
                 lambda: topk.head_loss_grad_bf16(hidden, weight, target, lse, loss, workspace=small)):
        with pytest.raises(topk.TopkError) as e:
            call()
        assert e.value.status == topk.ERR_SCRATCH


@pytest.mark.parametrize("rows,ignored", [(40, 0.5), (300, 0.3), (600, 0.9), (1000, 0.999)])
def test_ignored_rows(rows, ignored):
    run(*_inputs(rows, 136, 1111, seed=rows, ignored=ignored))


@pytest.mark.parametrize("rows", [1, 20, 300])
def test_every_row_ignored(rows):
    import torch
    hidden, weight, target = _inputs(rows, 64, 500, seed=1)
    target.fill_(-100)
    loss, lse, dh, dw = run(hidden, weight, target)
    for t in (loss, lse, dh, dw):
        assert not torch.any(t != 0)


def test_pieces_of_the_vocabulary():
    """The smallest workspace: one tile of the vocabulary at a time; sizes in between; the same gradient."""
    import torch

    from wide_bf16_row_gb300 import topk
    hidden, weight, target = _inputs(300, 128, 3000, seed=3, ignored=0.2)
    *_, dh, dw = run(hidden, weight, target, least=True)
    _, lse = topk.head_loss_bf16(hidden, weight, target)
    g = torch.randn(300, generator=torch.Generator().manual_seed(0)).cuda()
    size = topk.tf_topk_head_loss_grad_bf16_workspace(300, 128, 3000, True)
    space = torch.empty(size + 512 * 2 * 512 + 100, dtype=torch.uint8, device="cuda")
    dh2, dw2 = topk.head_loss_grad_bf16(hidden, weight, target, lse, g, workspace=space)
    check_grad(hidden, weight, target, g, dh2, dw2)
    assert torch.equal(dw, dw2)  # a column's gradient does not depend on the pieces


@pytest.mark.parametrize("want", [dict(hidden_grad=False), dict(weight_grad=False)])
def test_one_gradient(want):
    import torch
    args = _inputs(70, 256, 1300, seed=8)
    both, one = run(*args)[2:], run(*args, **want)[2:]
    for a, b, name in zip(both, one, ("hidden_grad", "weight_grad")):
        assert b is None if name in want else torch.equal(a, b)


def test_row_strides():
    run(*_inputs(45, 64, 700, seed=5, hidden_pad=24, weight_pad=8))
    run(*_inputs(290, 64, 700, seed=6, hidden_pad=8, weight_pad=16))


@pytest.mark.parametrize("rows", [20, 300])
def test_garbage_in_rows_that_do_not_count(rows):
    """Hidden states of NaN and infinity in ignored rows, targets out of range."""
    import torch

    from wide_bf16_row_gb300 import topk
    hidden, weight, target = _inputs(rows, 128, 900, seed=9)
    hidden = hidden.clone()
    target[::3] = -100
    target[1] = 900
    target[4] = -1
    target[7] = 1 << 40
    hidden[::3] = float("nan")
    hidden[3] = float("inf")
    loss, lse = topk.head_loss_bf16(hidden, weight, target)
    check_loss(torch.where(target[:, None] == -100, 0, hidden), weight, target, loss, lse)
    g = torch.rand(rows, device="cuda")
    g[::3] = float("inf")
    dh, dw = topk.head_loss_grad_bf16(hidden, weight, target, lse, g)
    check_grad(hidden, weight, target, g.nan_to_num(), dh, dw)
    counts = (target >= 0) & (target < 900)
    assert not torch.any(dh[~counts] != 0)


def test_other_ignore_index():
    hidden, weight, target = _inputs(30, 64, 300, seed=2)
    target[::2] = 7
    run(hidden, weight, target, ignore=7)


def test_infinite_logits():
    """A column of -inf logits has no share; one of +inf has all of it."""
    import torch

    from wide_bf16_row_gb300 import topk
    inf = float("inf")
    hidden = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    hidden[:, 0] = 1
    weight = torch.zeros(600, 64, dtype=torch.bfloat16, device="cuda")
    weight[5, 0] = -inf
    target = torch.tensor([0, 5, 599, 300], device="cuda")
    # inf * 0 is NaN: the other dims are cut away
    loss, lse = topk.head_loss_bf16(hidden[:, :8].contiguous(), weight[:, :8].contiguous(), target)
    assert torch.isnan(lse).all() or torch.allclose(lse, torch.tensor(599.0).log().cuda().expand(4))
    weight[5, 0] = float("nan")
    loss, lse = topk.head_loss_bf16(hidden, weight, target)
    assert torch.isnan(loss).all() and torch.isnan(lse).all()


def test_a_loss_near_zero_keeps_its_digits():
    """Targets that win by far: loss = exp(-gap) (V - 1), with the sums exact in fp32."""
    import torch

    from wide_bf16_row_gb300 import topk
    vocab = 1000
    weight = torch.zeros(vocab, 64, dtype=torch.bfloat16, device="cuda")
    weight[:16] = torch.eye(16, 64, device="cuda").bfloat16()
    hidden = (torch.arange(16, device="cuda")[:, None] * torch.eye(16, 64, device="cuda") * 2).bfloat16()
    target = torch.arange(16, device="cuda")
    loss, lse = topk.head_loss_bf16(hidden, weight, target)
    gap = 2.0 * np.arange(16)
    ref = np.log1p((vocab - 1) * np.exp(-gap))
    # log2 and its rounding around log2(999) = 10: 12 * 2^-23 of an exponent, expf and log1pf 4 ulp
    np.testing.assert_allclose(_np(loss), ref, rtol=(2 * 12 + 8) * 2.0 ** -23)


def test_large_logits():
    """Logits of some hundreds: no overflow, the exact winner."""
    import torch
    hidden, weight, target = _inputs(64, 64, 900, seed=4)
    run((hidden.float() * 64).bfloat16(), weight, target)


@pytest.mark.parametrize("g", ["mean", "one", "tiny", "huge", "mixed", "zero"])
def test_scales_of_the_gradient(g):
    import torch
    rows = 90
    hidden, weight, target = _inputs(rows, 128, 800, seed=6)
    grad = {"mean": torch.full((rows,), 1 / 90), "one": torch.ones(rows), "tiny": torch.full((rows,), 1e-30),
            "huge": torch.full((rows,), 1e30), "mixed": 10.0 ** (-torch.arange(rows) / 10),
            "zero": torch.zeros(rows)}[g].cuda()
    run(hidden, weight, target, g=grad)


def test_against_differences():
    """The gradient of one hidden coordinate against central differences of the
    loss (64-bit oracle at rounded inputs is not needed: the step is exact in bf16)."""
    import torch

    from wide_bf16_row_gb300 import topk
    hidden, weight, target = _inputs(8, 64, 400, seed=12)
    hidden = hidden.clone()
    hidden[:, 3] = 1.0
    _, lse = topk.head_loss_bf16(hidden, weight, target)
    dh, _ = topk.head_loss_grad_bf16(hidden, weight, target, lse, torch.ones(8, device="cuda"))
    step = 2.0 ** -4
    sides = []
    for s in (step, -step):
        moved = hidden.clone()
        moved[:, 3] = 1.0 + s
        sides.append(topk.head_loss_bf16(moved, weight, target)[0].double())
    slope = (sides[0] - sides[1]) / (2 * step)
    # |third derivative| <= 2 max|w|^3, a sixth of it times the step squared; losses within 1e-5 + logit errors;
    # the gradient's own roundings: 2^-8 of sum |G w| <= 2 max|w|, twice
    top = float(weight[:, 3].abs().max())
    allow = 2 * top ** 3 * step ** 2 / 6 + (1e-5 + 2 * float(logit_error(_np(hidden), _np(weight)).max())) / step \
        + 2 * HALF * 2 * top
    assert float((slope - dh[:, 3].double()).abs().max()) <= allow


def test_repeats_bit_for_bit():
    import torch
    args = _inputs(400, 136, 2000, seed=20, ignored=0.3)
    first, second = run(*args), run(*args)
    assert all(torch.equal(a, b) for a, b in zip(first, second))


def test_streams_and_graphs():
    """A side stream; both calls captured with a caller's workspaces and replayed on new inputs."""
    import torch

    from wide_bf16_row_gb300 import topk
    hidden, weight, target = _inputs(300, 128, 1500, seed=30, ignored=0.2)
    hidden, weight = hidden.clone(), weight.clone()
    g = torch.rand(300, device="cuda")
    loss, lse = topk.head_loss_bf16(hidden, weight, target)
    dh, dw = topk.head_loss_grad_bf16(hidden, weight, target, lse, g)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    loss2, lse2 = topk.head_loss_bf16(hidden, weight, target, stream=side)
    dh2, dw2 = topk.head_loss_grad_bf16(hidden, weight, target, lse2, g, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in ((loss, loss2), (lse, lse2), (dh, dh2), (dw, dw2)))
    space = torch.empty(topk.tf_topk_head_loss_grad_bf16_workspace(300, 128, 1500), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss3, lse3 = topk.head_loss_bf16(hidden, weight, target)
        dh3, dw3 = topk.head_loss_grad_bf16(hidden, weight, target, lse3, g, workspace=space)
    new = _inputs(300, 128, 1500, seed=31, ignored=0.6)
    for a, b in zip((hidden, weight, target), new):
        a.copy_(b)
    graph.replay()
    graph.replay()
    check_loss(hidden, weight, target, loss3, lse3)
    check_grad(hidden, weight, target, g, dh3, dw3)


def test_no_rows():
    import torch

    from wide_bf16_row_gb300 import topk
    hidden = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    weight = torch.ones(100, 64, dtype=torch.bfloat16, device="cuda")
    target = torch.empty(0, dtype=torch.int64, device="cuda")
    loss, lse = topk.head_loss_bf16(hidden, weight, target)
    assert loss.shape == lse.shape == (0,)
    dh, dw = topk.head_loss_grad_bf16(hidden, weight, target, lse, loss)
    assert dh.shape == (0, 64) and not torch.any(dw != 0)


@pytest.mark.parametrize("rows", [4096, 4097])
def test_many_rows_packed(rows):
    """Up to 4096 rows are found and packed in one launch, more in two."""
    run(*_inputs(rows, 72, 300, seed=rows, ignored=0.3, hidden_pad=8))


def _inside(shape, dtype, before=8, after=512):
    """A tensor in the middle of bytes of 0xA5, and a check that those still stand."""
    import torch
    size = int(np.prod(shape)) * dtype.itemsize
    block = torch.full((before * 16 + size + after,), 0xA5, dtype=torch.uint8, device="cuda")
    part = block[before * 16:before * 16 + size].view(dtype).view(shape)
    return part, lambda: bool((block[:before * 16] == 0xA5).all()) and bool((block[before * 16 + size:] == 0xA5).all())


@pytest.mark.parametrize("rows,dim,vocab", [(1, 8, 1), (5, 72, 130), (130, 64, 257), (300, 136, 515), (4097, 72, 300)])
@pytest.mark.parametrize("least", [False, True])
def test_nothing_beside_the_outputs_is_written(rows, dim, vocab, least):
    """Outputs and workspaces of exactly their sizes inside larger buffers; bf16 bits as int16; int32 targets."""
    import torch

    from wide_bf16_row_gb300 import topk
    hidden, weight, target = _inputs(rows, dim, vocab, seed=11, ignored=0.2, wide=False)
    bits = hidden.contiguous().view(torch.int16), weight.contiguous().view(torch.int16)
    g = torch.rand(rows, device="cuda")
    loss, lse = topk.head_loss_bf16(hidden, weight, target)
    need = topk.tf_topk_head_loss_bf16_workspace(rows, dim, vocab)
    grad_need = topk.tf_topk_head_loss_grad_bf16_workspace(rows, dim, vocab, least)
    parts = [_inside((rows,), torch.float32), _inside((rows,), torch.float32), _inside((need,), torch.uint8, 1),
             _inside((rows, dim), torch.bfloat16), _inside((vocab, dim), torch.bfloat16), _inside((grad_need,), torch.uint8, 1)]
    outs = [p for p, _ in parts]
    topk.head_loss_bf16(*bits, target, out=outs[:2], workspace=outs[2])
    topk.head_loss_grad_bf16(*bits, target, outs[1], g, out=outs[3:5], workspace=outs[5])
    assert all(ok() for _, ok in parts)
    assert torch.equal(outs[0], loss) and torch.equal(outs[1], lse)
    check_grad(hidden, weight, target, g, *outs[3:5])
    assert topk.device_fault() == 0
