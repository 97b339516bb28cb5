"""Refusals of linear_ce_bwd_ex, on the host before anything is launched (CPU)."""
import pytest

import cross_entropy_loss_ce_gb300 as gbce
from cross_entropy_loss_ce_gb300 import build as gbuild
from test_linear_abi import FAKE, bwd

NULL, SIZE, DTYPE, ALIGN = 1, 2, 3, 4


@pytest.fixture(scope="module")
def lib():
    gbuild.build()
    return gbce.load_library()


def ex(row_loss=FAKE, **kw):
    a = bwd(**kw)
    return a[:6] + [row_loss] + a[6:]


@pytest.mark.parametrize("kw,code", [(dict(row_loss=FAKE + 2), ALIGN), (dict(lse=None), NULL), (dict(t=None), NULL),
                                     (dict(dtype=0), DTYPE), (dict(dhs=63), SIZE), (dict(row_loss=None, h=None), NULL)])
def test_linear_ce_bwd_ex_refuses(lib, kw, code):
    assert lib.linear_ce_bwd_ex(*ex(**kw)) == code


def test_nothing_to_do_needs_no_device(lib):
    assert lib.linear_ce_bwd_ex(*ex(M=0, dw=None)) == gbce.OK
