"""The rows of a plan that are no slot's, at the largest sizes the library accepts: the row arithmetic of the
kernels, compiled for the host (CPU)."""
import subprocess

import pytest

from cross_entropy_loss_ce_gb300 import build as gbuild

PROGRAM = r"""
#include <climits>
#include <cstdio>
#include <cstdlib>
#include "permute_kernels.cuh"

struct Print {
    int *left;
    __host__ __device__ void operator()(int row) const
    {
        printf("%d ", row);
        if (--*left < 0)
            exit(3);  // rows without end
    }
};

int main(int argc, char **argv)
{
    int left = 2000;
    for (int lane = 0; lane < 32; ++lane)
        gbce::sort_pad_rows(atoi(argv[1]), atoi(argv[2]), atoi(argv[3]), lane, Print{&left});
    return 0;
}
"""


@pytest.fixture(scope="module")
def pad_rows(tmp_path_factory):
    d = tmp_path_factory.mktemp("pad_rows")
    (d / "rows.cu").write_text(PROGRAM)
    subprocess.run([gbuild.nvcc(), "-gencode", "arch=compute_103a,code=sm_103a", "-std=c++17", "-I", gbuild.CSRC,
                    str(d / "rows.cu"), "-o", str(d / "rows")], check=True, capture_output=True)

    def run(off, total, following):
        r = subprocess.run([str(d / "rows"), str(off), str(total), str(following)], capture_output=True, text=True)
        assert r.returncode == 0, r.stdout[:200]
        return sorted(map(int, r.stdout.split()))
    return run


LAST = 2 ** 31 - 1


@pytest.mark.parametrize("off,total,following", [
    (0, 0, 0), (0, 5, 5), (0, 5, 8), (128, 1, 256), (7, 0, 7), (1000, 1, 2024),
    # 2^31 - 16 slots of two experts, align 2: the last ends within 32 rows of 2^31
    (2 ** 31 - 16, 1, 2 ** 31 - 14), (LAST - 64, 1, LAST), (LAST - 2, 1, LAST), (LAST - 1, 1, LAST), (LAST, 0, LAST),
    (LAST - 1023, 1, LAST), (0, LAST - 40, LAST - 3), (5, LAST - 10, LAST)])
def test_rows_behind_an_experts_slots(pad_rows, off, total, following):
    assert pad_rows(off, total, following) == list(range(off + total, following))
