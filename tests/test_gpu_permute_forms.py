"""Every form of the expert permutation's kernels in every type (tolerances in permute_ref): the combine takes
other kernels from 16 warps an SM on, by units of a row and slots of a token (GPU)."""
import pytest
import torch

from test_gpu_permute import DT, check_all

pytestmark = pytest.mark.gpu

WARPS = 16  # of an SM: with fewer a lane takes one unit


def tokens(pieces):
    """A little more than the fewest tokens of `pieces` warps each that give every SM its warps."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return -(-WARPS * sms // pieces) + 3


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("k", [1, 2, 3])
def test_whole_units(dtype, k):
    v = 4 if dtype == "f32" else 8
    # up to 32 units, up to 64, and more: two pieces of 64 units each, then three
    for units in (31, 33, 64, 65, 129):
        check_all(tokens(-(-units // 64)), k, 9, units * v, DT[dtype], align=4)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("k", [1, 2, 3, 5])
def test_single_values(dtype, k):
    for H in (33, 511, 1025):
        check_all(tokens(-(-H // 512)), k, 9, H, DT[dtype], align=4)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("k", [1, 2, 3])
def test_pairs(dtype, k):
    for H in (66, 1022, 1030):
        check_all(tokens(-(-(H // 2) // 512)), k, 9, H, DT[dtype], align=4)


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("k", [2, 4, 8])
def test_gradients_by_one_warp_of_a_token_and_by_several(dtype, k):
    v = 4 if dtype == "f32" else 8
    for T in (40, 700):
        for H in (32 * v, 40 * v, 260 * v, 260 * v + 2, 260 * v + 1, 700 * v, 2051):
            check_all(T, k, 9, H, DT[dtype], align=4)
