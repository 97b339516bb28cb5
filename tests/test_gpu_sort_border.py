"""A plan whose rows reach the end of the 32-bit range (34 GB on the device)."""
import pytest
import torch

import cross_entropy_loss_ce_gb300 as gbce

pytestmark = pytest.mark.gpu


def test_rows_up_to_the_last_one():
    # 2^31 - 16 slots, experts padded to 2 rows: the last expert's only slot is followed by a row that is none's,
    # 15 rows below 2^31
    T, k = 2 ** 27 - 1, 16
    n = T * k
    free, _ = torch.cuda.mem_get_info()
    if free < 48e9:
        pytest.skip("needs 48 GB of device memory")
    experts = torch.zeros(T, k, device="cuda", dtype=torch.int64)
    experts[T - 1, k - 1] = 1
    plan = gbce.moe_sort(experts, 2, 2)
    assert gbce.last_error() == gbce.OK
    assert plan.rows == n + 2 == gbce.load_library().moe_plan_rows(T, 2, k, 2)
    del experts
    assert plan.counts.tolist() == [n - 1, 1] and plan.offsets.tolist() == [0, n, n + 2]
    position, source = plan.position.view(-1), plan.source
    assert position[n - 1].item() == n and source[n - 1:].tolist() == [-1, n - 1, -1]
    step = 2 ** 28
    for a in range(0, n - 1, step):  # expert 0: slots and rows are the same
        b = min(a + step, n - 1)
        want = torch.arange(a, b, device="cuda", dtype=torch.int32)
        assert torch.equal(position[a:b], want) and torch.equal(source[a:b], want)
