"""GPU: the digits of the head's loss and of its gradient, where sums are exact
or known well enough to hold the kernels to a few units in the last place."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import head_loss as oracle_loss

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from wide_bf16_row_gb300 import build
    build.build()


def _np(t):
    return t.detach().double().cpu().numpy()


@pytest.mark.parametrize("rows", [5, 200, 300])
@pytest.mark.parametrize("tied", [2, 7])
def test_exact_sums_of_large_logits(rows, tied):
    """One-hot hidden states at 4096 dims, `tied` columns with a logit of 32 and the target among them: nothing is
    rounded in a sum, so lse = 32 + log(tied) and loss = log(tied), but for the exponents: 32 log2 e = 46 is rounded
    when taken as a reference and when log2 of the sum is added to it, and their product with ln 2 once more
    (2^-19 ln 2, twice, and 2^-20); the constants are 2 u off, relatively, and the rest some u of numbers up to 3."""
    import torch

    from wide_bf16_row_gb300 import topk
    dim, vocab = 4096, 700
    hidden = torch.zeros(rows, dim, dtype=torch.bfloat16, device="cuda")
    at = (torch.arange(rows) * 37 % dim).cuda()
    hidden[torch.arange(rows), at] = 1
    weight = torch.zeros(vocab, dim, dtype=torch.bfloat16, device="cuda")
    weight[100:100 + 90 * tied:90] = 32
    target = torch.full((rows,), 100 + 90 * (tied - 1), device="cuda")
    loss, lse = topk.head_loss_bf16(hidden, weight, target)
    allow = 2 * 2.0 ** -19 * 0.7 + 2.0 ** -20 + 2 * U * 32 + 16 * U
    rest = (vocab - tied) * np.exp(-32.0)
    assert np.abs(_np(lse) - 32 - np.log(tied + rest)).max() <= allow
    assert np.abs(_np(loss) - np.log(tied + rest)).max() <= allow


@pytest.mark.parametrize("rows", [3, 140, 300])
@pytest.mark.parametrize("dim", [512, 2048, 4096, 16384])
@pytest.mark.parametrize("lead", [0, 300])
def test_a_leading_dim(rows, dim, lead):
    """Logits of about 32 of which one dim holds all but a few parts in a hundred, as hidden states with a massive
    activation have them: beyond the dims of a part the error does not grow.  The tensor cores add 16 products and the
    sum so far at a time, each aligned to the largest of them and cut off below 2^-23 of it at the latest: 17 units
    lost at most.  They sum 512 dims at most, 32 additions, with more than 128 rows 4096; the parts are then added
    rounding to nearest (u of the sum each).  The exponents' roundings are those of the test above.  (Over all of 16384
    dims in one sum such a logit lost 9.7e-3.)"""
    import torch

    from wide_bf16_row_gb300 import topk
    g = torch.Generator().manual_seed(dim + rows)
    vocab = 300
    hidden = (0.01 * torch.rand(rows, dim, generator=g)).bfloat16()
    weight = torch.rand(vocab, dim, generator=g).bfloat16()
    hidden[:, lead] = 8
    weight[:, lead] = 4
    target = torch.randint(0, vocab, (rows,), generator=g)
    loss, lse = topk.head_loss_bf16(hidden.cuda(), weight.cuda(), target.cuda())
    h, w = _np(hidden), _np(weight)
    ref_loss, ref_lse = oracle_loss.loss(h, w, target.numpy())
    most = 512 if rows <= 128 else 4096
    parts = [(np.abs(h[:, i:i + most]) @ np.abs(w[:, i:i + most]).T).max(1) for i in range(0, dim, most)]
    size = sum(parts)
    allow = most / 16 * 17 * 2.0 ** -23 * size + (len(parts) + 1) * U * size + 4 * 2.0 ** -19 * 0.7 + 2.0 ** -19 + 1e-6
    assert (np.abs(_np(lse) - ref_lse) <= allow).all(), (np.abs(_np(lse) - ref_lse).max(), allow.min())
    # the target's logit: 32 lanes' sums by FMA and their butterfly
    allow += (dim / 32 + 5) * U * size
    assert (np.abs(_np(loss) - ref_loss) <= allow).all(), (np.abs(_np(loss) - ref_loss).max(), allow.min())


@pytest.mark.parametrize("rows", [1, 300, 5000])
@pytest.mark.parametrize("gap", [8.0, 11.0, 14.0])
def test_gradient_of_a_sure_row(rows, gap):
    """The target's entry of G = g (p - 1) where p is nearly 1: 64 columns at a logit of 0 and the target's, a sum of
    4096 positive products, at `gap`.  p - 1 = expm1(x_t - lse), with lse rounded (half of its unit, 2^-21) and from
    the same x_t; x_t by FMA, 133 roundings at most of u of itself, moves 1 - p by as much of it; the 64 exponentials
    and their sum by 1e-5 of it; G and the gradient are each rounded to bf16 (2^-8).  One row alone has a gradient,
    so that d_weight[target] = G h and d_hidden = G weight[target]."""
    import torch

    from wide_bf16_row_gb300 import topk
    dim, vocab = 4096, 65
    g = torch.Generator().manual_seed(int(gap))
    hidden = (torch.rand(rows, dim, generator=g) + 0.5).bfloat16()
    weight = torch.zeros(vocab, dim)
    at = rows // 2
    shape = torch.rand(dim, generator=g) + 0.5
    weight[7] = shape * gap / (shape @ hidden[at].float())
    weight = weight.bfloat16()
    target = torch.full((rows,), 7)
    grad = torch.zeros(rows)
    grad[at] = 0.25
    args = hidden.cuda(), weight.cuda(), target.cuda()
    loss, lse = topk.head_loss_bf16(*args)
    dh, dw = topk.head_loss_grad_bf16(*args, lse, grad.cuda())
    x = float(_np(hidden)[at] @ _np(weight)[7])
    others = 64 * np.exp(-x)
    entry = -0.25 * others / (1 + others)  # p - 1
    allow = 0.25 * 2.0 ** -21 + abs(entry) * (133 * U * x + 1e-5)
    for got, by in ((_np(dw)[7], _np(hidden)[at]), (_np(dh)[at], _np(weight)[7])):
        off = np.abs(got - entry * by)
        assert (off <= (allow + 2 * 2.0 ** -8 * (abs(entry) + allow)) * np.abs(by)).all(), (off / np.abs(by)).max() / abs(entry)


@pytest.mark.parametrize("rows", [4, 150, 300])
@pytest.mark.parametrize("dim", [64, 4608])
@pytest.mark.parametrize("level", [0.0, 100.0, -100.0])
def test_infinite_columns(rows, dim, level):
    """A column of -inf logits has no share and an infinite loss of its own; one of +inf has all of it, however large
    the other logits.  Sums are exact; the exponents' roundings as above."""
    import torch

    from wide_bf16_row_gb300 import topk
    inf = float("inf")
    vocab = 600
    hidden = torch.zeros(rows, dim, dtype=torch.bfloat16, device="cuda")
    hidden[:, 0] = 1
    target = torch.arange(rows, device="cuda") * 5 % vocab
    own = target == 5
    for column in (-inf, inf):
        weight = torch.zeros(vocab, dim, dtype=torch.bfloat16, device="cuda")
        weight[:, 0] = level
        weight[5, 0] = column
        loss, lse = topk.head_loss_bf16(hidden, weight, target)
        assert own.any()
        if column == inf:
            assert (lse == inf).all() and (loss[own] == 0).all() and (loss[~own] == inf).all()
        else:
            allow = 4 * 2.0 ** -17 * 0.7 + 2.0 ** -17 + 16 * U
            assert (lse - level - np.log(599)).abs().max() <= allow
            assert (loss[own] == inf).all() and (loss[~own] - np.log(599)).abs().max() <= allow


@pytest.mark.parametrize("rows", [4, 150, 300])
@pytest.mark.parametrize("dim", [64, 4608])
def test_no_column_has_a_share(rows, dim):
    """All logits -inf: lse = log 0 = -inf, and the loss -inf + inf has no value."""
    import torch

    from wide_bf16_row_gb300 import topk
    inf = float("inf")
    hidden = torch.zeros(rows, dim, dtype=torch.bfloat16, device="cuda")
    hidden[:, 0] = 1
    weight = torch.zeros(600, dim, dtype=torch.bfloat16, device="cuda")
    weight[:, 0] = -inf
    loss, lse = topk.head_loss_bf16(hidden, weight, torch.arange(rows, device="cuda"))
    assert (lse == -inf).all() and torch.isnan(loss).all()


def test_the_smallest_workspace_is_taken_and_one_byte_less_refused():
    """At each place of a workspace the least size that a call takes, found by halving, is within the queried one;
    a byte less is refused before anything is launched, and the call at that size is right and writes nothing past it."""
    import torch

    from wide_bf16_row_gb300 import topk
    g = torch.Generator().manual_seed(1)
    rows, dim, vocab = 300, 72, 500
    hidden, weight = torch.randn(rows, dim, generator=g).bfloat16().cuda(), torch.randn(vocab, dim, generator=g).bfloat16().cuda()
    target = torch.randint(0, vocab, (rows,), generator=g).cuda()
    grad = torch.ones(rows, device="cuda")
    want = topk.head_loss_bf16(hidden, weight, target)
    want_grad = topk.head_loss_grad_bf16(hidden, weight, target, want[1], grad)
    for start in (0, 16, 240):
        for loss in (True, False):
            need = topk.tf_topk_head_loss_bf16_workspace(rows, dim, vocab) if loss else \
                topk.tf_topk_head_loss_grad_bf16_workspace(rows, dim, vocab, True)
            block = torch.full((start + need + 512,), 0xA5, dtype=torch.uint8, device="cuda")

            def call(size):
                space = block[start:start + size]
                if loss:
                    return topk.head_loss_bf16(hidden, weight, target, workspace=space)
                return topk.head_loss_grad_bf16(hidden, weight, target, want[1], grad, workspace=space)

            lo, hi = 8, need
            call(hi)
            while lo + 1 < hi:
                mid = (lo + hi) // 2
                try:
                    call(mid)
                    hi = mid
                except topk.TopkError as e:
                    assert e.status == topk.ERR_SCRATCH
                    lo = mid
            with pytest.raises(topk.TopkError):
                call(hi - 1)
            block.fill_(0xA5)
            got = call(hi)
            assert bool((block[start + hi:] == 0xA5).all()) and bool((block[:start] == 0xA5).all())
            if loss:
                assert all(torch.equal(a, b) for a, b in zip(got, want))
            else:
                assert torch.equal(got[1], want_grad[1])
                torch.testing.assert_close(got[0], want_grad[0], rtol=2.0 ** -7, atol=2.0 ** -7)


@pytest.mark.parametrize("rows", [3, 300])
@pytest.mark.parametrize("level", [9.5, 13.0, 17.25, 25.0, 40.5, 61.0, -33.0])
@pytest.mark.parametrize("tied", [2, 3, 90])
def test_a_loss_has_the_digits_of_its_own_size(rows, level, tied):
    """All columns at one logit or `tied` at it and the others far below: loss = log of their number, whatever the
    logit.  An exponent is a multiple of log2 e less its rounded reference, which a fused product takes exactly; the
    reference's logarithm less the target's logit cancels to a few u of 1; log2 of the sum, its product with ln 2, the
    exponential and log1p are 2 u each of numbers up to log 700 = 6.6, their sums u."""
    import torch

    from wide_bf16_row_gb300 import topk
    vocab = 700
    hidden = torch.zeros(rows, 64, dtype=torch.bfloat16, device="cuda")
    hidden[:, 5] = 1
    weight = torch.zeros(vocab, 64, dtype=torch.bfloat16, device="cuda")
    weight[:, 5] = level - 64
    weight[50:50 + tied, 5] = level
    target = torch.full((rows,), 51, device="cuda")
    for columns, others in ((tied, np.exp(-64.0) * (vocab - tied)), (vocab, 0.0)):
        if columns == vocab:
            weight[:, 5] = level
        loss, lse = topk.head_loss_bf16(hidden, weight, target)
        ref = np.log(columns + others)
        assert np.abs(_np(loss) - ref).max() <= (8 * ref + 8) * U, (np.abs(_np(loss) - ref).max() / U, ref)
        assert np.abs(_np(lse) - level - ref).max() <= (8 * ref + 8 + 2 * abs(level + ref)) * U


@pytest.mark.parametrize("rows", [3, 300])
def test_the_target_s_logit_keeps_its_last_digits(rows):
    """The target's products are 32 and thirty-one quarters of a unit of it, one to a lane of its sum; the two other
    columns' logits are 32.  Added up in fp32 three of the quarters would be lost, 2.9e-6 of the logit and two thirds
    of that of the loss; the allowance is that of the test above."""
    import torch

    from wide_bf16_row_gb300 import topk
    hidden = torch.zeros(rows, 256, dtype=torch.bfloat16, device="cuda")
    hidden[:, ::8] = 1
    weight = torch.zeros(3, 256, dtype=torch.bfloat16, device="cuda")
    weight[:, 0] = 32
    weight[1, 8::8] = 2.0 ** -20
    loss, _ = topk.head_loss_bf16(hidden, weight, torch.ones(rows, dtype=torch.int64, device="cuda"))
    ref = np.log(1 + 2 * np.exp(-31 * 2.0 ** -20))
    assert np.abs(_np(loss) - ref).max() <= (8 * ref + 8) * U, np.abs(_np(loss) - ref).max() / U
