"""What the autograd forms of the expert permutation keep between forward and backward (GPU)."""
import pytest
import torch
from torch.utils.checkpoint import checkpoint

import cross_entropy_loss_ce_gb300 as gbce
from permute_ref import PlanRef, combine_bwd_ref, combine_ref, near

pytestmark = pytest.mark.gpu
T, k, E, H = 50, 2, 6, 40


def operands(dtype=torch.float32):
    g = torch.Generator("cuda").manual_seed(5)
    experts = torch.randint(-1, E, (T, k), device="cuda", generator=g)
    plan, ref = gbce.moe_sort(experts, E, 4), PlanRef(experts, E, 4)
    x = torch.randn(T, H, device="cuda", generator=g).to(dtype)
    y = torch.randn(ref.rows, H, device="cuda", generator=g).to(dtype)
    w = torch.rand(T, k, device="cuda", generator=g)
    return plan, ref, x, y, w


def test_recomputed_forward():
    # a plan whose parts are looked at between the forward and its recomputation
    plan, ref, x, y, w = operands()
    y, w = y.requires_grad_(), w.requires_grad_()
    out = checkpoint(lambda a, b: gbce.combine_tokens(a, plan, b), y, w, use_reentrant=False)
    assert plan.position.shape == (T, k)
    d_y, d_w = torch.autograd.grad(out, (y, w), x)
    want = combine_bwd_ref(x, y.detach(), ref.position, w.detach())
    near(d_y, *want[0], "d_y")
    near(d_w, *want[1], "d_weights")
