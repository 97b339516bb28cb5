"""Router rows at the ends of their type's range (GPU), against the 64-bit plain form of head_ref."""
import pytest
import torch

import cross_entropy_loss_ce_gb300 as gbce
from head_ref import MoeRef, near

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T", [40, 600])
def test_rows_of_the_types_lowest_value(T, dtype):
    # a mask of the lowest value that leaves a counted token nothing: all its experts are equally likely
    x = torch.randn(T, 12, device="cuda", generator=torch.Generator("cuda").manual_seed(T)).to(dtype)
    ex = x.float().topk(2, 1).indices.contiguous()
    low = torch.finfo(dtype).min
    x[3] = low
    x[5, 1:] = low
    x[6] = -low
    x[7, :5] = low
    x[8, 5] = -low
    ref = MoeRef(x, ex, 0.5, 0.0)
    loss, counts, grad = gbce.moe_balance(x, ex, 0.5, 0.0)
    assert torch.equal(counts, ref.counts)
    near(loss, ref.loss, ref.loss_tol, "loss")
    near(grad, ref.grad, ref.grad_tol, "grad")


@pytest.mark.parametrize("T", [40, 600])
@pytest.mark.parametrize("size", [1e5, 2e6, 1e10, 1e22, 1e37])
def test_logits_of_any_size(T, size):
    # differences of a few units at 1e5, of thousands of steps of the type above
    g = torch.Generator("cuda").manual_seed(T)
    x = size * torch.randn(T, 12, device="cuda", generator=g)
    x[::2] = torch.sign(x[::2]) * size + torch.randn(T // 2, 12, device="cuda", generator=g)
    ex = x.topk(2, 1).indices.contiguous()
    ref = MoeRef(x, ex, 0.5, 0.0)
    loss, counts, grad = gbce.moe_balance(x, ex, 0.5, 0.0)
    assert torch.equal(counts, ref.counts)
    near(loss, ref.loss, ref.loss_tol, "loss")
    near(grad, ref.grad, ref.grad_tol, "grad")


@pytest.mark.parametrize("T", [40, 600])
def test_a_row_loss_past_the_range_of_fp32(T):
    # a logit of 1e22: z_coef lse^2 is 1e41, past fp32, and over 40 tokens the loss is too: infinite, not NaN.
    # Over 600 it is 1.7e38, which fp32 holds.  Every gradient is finite.
    x = torch.randn(T, 8, device="cuda", generator=torch.Generator("cuda").manual_seed(T))
    ex = x.topk(2, 1).indices.contiguous()
    x[T // 2, 3] = 1e22
    ref = MoeRef(x, ex, 0.01, 0.001)
    loss, counts, grad = gbce.moe_balance(x, ex, 0.01, 0.001)
    if T == 40:
        assert float(ref.loss.float()) == float("inf") and float(loss) == float("inf")
    else:
        near(loss, ref.loss, ref.loss_tol, "loss")
    assert torch.equal(counts, ref.counts)
    near(grad, ref.grad, ref.grad_tol, "grad")
