"""Refusals of the linear layer's backward pass come before any HIP call: on a
machine without a GPU (or with one that is never asked) a refused call returns
its reason, not a launch error."""
from __future__ import annotations

import pytest

from tests.test_abi_linear_moe import INVALID, UNSUPPORTED, P, backward, lib  # noqa: F401  (lib: the fixture)

FAR = (1 << 20) + 8


@pytest.mark.parametrize("kw", [dict(ldda=FAR), dict(lddb=FAR), dict(ldda=FAR, db=None), dict(lddb=FAR, da=None),
                                dict(ldda=FAR, lddb=FAR, dbias=None, act=0)])
def test_backward_gradient_rows_too_far_apart(lib, kw):  # noqa: F811
    assert backward(lib, **kw) == UNSUPPORTED


@pytest.mark.parametrize("kw", [dict(dbias=P + 2, da=None, db=None), dict(dc=P + 1), dict(pre=P + 1),
                                dict(k=(1 << 22) + 8, lda=(1 << 22) + 8, ldb=(1 << 22) + 8, ldda=1 << 23, lddb=1 << 23)])
def test_backward_unsupported(lib, kw):  # noqa: F811
    assert backward(lib, **kw) == UNSUPPORTED


def test_gradients_not_asked_for_are_not_checked(lib):  # noqa: F811
    """(the first fault that is left: rows of db closer than its columns)"""
    assert backward(lib, da=None, ldda=FAR, b=None, ldb=0, lddb=8) == INVALID
