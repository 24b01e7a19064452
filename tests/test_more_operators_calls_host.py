"""Calls of the operators around an expert layer and before sampling that are
refused, without a GPU (nothing is launched)."""
from __future__ import annotations

import pytest

from tests.test_abi_host import FAKE
from tests.test_more_operators_host import call_penalize


@pytest.fixture(scope="module")
def lib():
    from wide_bf16_row_gb300 import build
    build.build()
    from wide_bf16_row_gb300 import topk
    return topk.library()


@pytest.mark.parametrize("kwargs", [dict(os=104), dict(stride=104), dict(os=108, stride=104, rows=2),
                                    dict(os=104, allowed=FAKE, als=4), dict(os=104, width=0, tokens=None)])
def test_penalties_in_place_at_another_stride(lib, kwargs):
    """The logits' own address with other rows: a row's result would lie on another row's logits."""
    assert call_penalize(lib, **kwargs) == 2
