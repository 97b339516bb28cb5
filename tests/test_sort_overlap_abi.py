"""moe_sort refuses arrays that share memory: it keeps intermediate values in position (CPU; each call is refused
before anything is launched)."""
import itertools

import pytest

import cross_entropy_loss_ce_gb300 as gbce
from cross_entropy_loss_ce_gb300 import build as gbuild

T, K, E, ALIGN, STRIDE = 5000, 4, 60, 16, 6
ROWS = -(-(T * K + E * (ALIGN - 1)) // ALIGN) * ALIGN
SIZES = {"experts": ((T - 1) * STRIDE + K) * 8, "position": T * K * 4, "source": ROWS * 4, "offsets": (E + 1) * 4,
         "counts": E * 4}


@pytest.fixture(scope="module")
def lib():
    gbuild.build()
    return gbce.load_library()


@pytest.mark.parametrize("first,second", list(itertools.permutations(SIZES, 2)))
@pytest.mark.parametrize("side", ["start", "end"])
def test_arrays_that_share_memory(lib, first, second, side):
    at = {name: 2 ** 30 * (i + 1) for i, name in enumerate(SIZES)}  # never dereferenced
    # `second` starts within the last value of `first`, or on its first one
    at[second] = at[first] + (SIZES[first] - 8 if side == "end" else 0)
    assert lib.moe_plan_rows(T, E, K, ALIGN) == ROWS
    # experts within the last value of a 4-byte array may also start off 8 bytes, which is looked at first
    want = gbce.ERR_ALIGN if at["experts"] % 8 else gbce.ERR_OVERLAP
    assert lib.moe_sort(at["experts"], STRIDE, at["position"], at["source"], at["offsets"], at["counts"], T, E, K, ALIGN,
                        None) == want


def test_strides_past_any_address(lib):
    # the span of the choices is the widest that can be: everything behind their start lies in it
    assert lib.moe_sort(2 ** 20, 2 ** 46, 2 ** 30, 2 ** 31, 2 ** 32, 2 ** 33, 2 ** 27 - 1, E, K, 1, None) == gbce.ERR_OVERLAP
