"""What the autograd forms of the expert permutation keep between forward and backward (GPU)."""
import gc

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


def of_parts(plan):
    return gbce.MoePlan(plan.position.clone(), plan.source.clone(), plan.offsets.clone(), plan.counts.clone(),
                        plan.align)


@pytest.mark.parametrize("own", [True, False])  # a plan of moe_sort, and one of the caller's tensors
@pytest.mark.parametrize("part", ["position", "source"])
def test_a_plan_that_changed_before_the_backward_is_refused(own, part):
    plan, _, x, y, w = operands()
    if not own:
        plan = of_parts(plan)
    x, y, w = x.requires_grad_(), y.requires_grad_(), w.requires_grad_()
    outs = [gbce.dispatch_tokens(x, plan), gbce.combine_tokens(y, plan, w), gbce.combine_tokens(y, plan)]
    torch.autograd.grad(outs[0].sum(), x, retain_graph=True)
    getattr(plan, part).fill_(0)
    for out, leaf in zip(outs, (x, y, y)):
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            torch.autograd.grad(out.sum(), leaf)


@pytest.mark.parametrize("own", [True, False])
def test_backward_from_what_hooks_kept(own):
    # hooks that move saved tensors away: the plan may then change, the gradients are of the one that was saved
    plan, ref, x, y, w = operands()
    if not own:
        plan = of_parts(plan)
    x, y, w = x.requires_grad_(), y.requires_grad_(), w.requires_grad_()
    with torch.autograd.graph.save_on_cpu():
        rows, out, bare = gbce.dispatch_tokens(x, plan), gbce.combine_tokens(y, plan, w), gbce.combine_tokens(y, plan)
    plan.position.fill_(-1)
    plan.source.fill_(-1)
    near(torch.autograd.grad(rows, x, y.detach())[0], *combine_ref(y.detach(), ref.position, None), "d_x")
    d_y, d_w = torch.autograd.grad(out, (y, w), x.detach())
    want = combine_bwd_ref(x.detach(), y.detach(), ref.position, w.detach())
    near(d_y, *want[0], "d_y")
    near(d_w, *want[1], "d_weights")
    (d_bare,) = torch.autograd.grad(bare, y, x.detach())
    token = ref.source.long().clamp_min(0) // k
    assert torch.equal(d_bare, torch.where((ref.source >= 0)[:, None], x.detach()[token], 0.0))


@pytest.mark.parametrize("weighted", [True, False])
def test_rows_are_kept_for_the_weights_gradient_only(weighted):
    plan, ref, x, y, w = operands(torch.bfloat16)
    gc.collect()
    leaf = y.requires_grad_()
    rows = leaf * 1  # an activation that nothing else keeps
    size = rows.untyped_storage().nbytes()
    out = gbce.combine_tokens(rows, plan, w if weighted else None)
    after = torch.cuda.memory_allocated()
    del rows
    gc.collect()
    assert torch.cuda.memory_allocated() <= after - size
    (d_y,) = torch.autograd.grad(out, leaf, x)
    (want, tol), _ = combine_bwd_ref(x, y.detach(), ref.position, w if weighted else torch.ones_like(w))
    near(d_y, want, tol, "d_y")


def test_rows_may_change_where_no_gradient_needs_them():
    plan, ref, x, y, w = operands()
    leaf = y.requires_grad_()
    rows = leaf * 1
    out = gbce.combine_tokens(rows, plan, w)
    rows.detach().zero_()
    (d_y,) = torch.autograd.grad(out, leaf, x)
    near(d_y, *combine_bwd_ref(x, y.detach(), ref.position, w)[0], "d_y")


def test_gradient_of_the_rows_without_the_rows():
    plan, ref, x, y, w = operands(torch.float16)
    d_y, d_w = gbce.moe_combine_bwd(x, None, plan, w, want_weights=False)
    assert d_w is None and torch.equal(d_y, gbce.moe_combine_bwd(x, y, plan, w)[0])
    with pytest.raises(ValueError, match="y is needed"):
        gbce.moe_combine_bwd(x, None, plan, w)
    with pytest.raises(ValueError, match="y is needed"):
        gbce.moe_combine_bwd(x, None, plan, w, want_y=False)
    buf = torch.zeros(plan.rows, H, device="cuda")
    with pytest.raises(ValueError, match="shares memory with d_out"):
        gbce.moe_combine_bwd(buf[:T], None, plan, w, want_weights=False, d_y=buf)


def test_recomputed_plan():
    # a whole block under checkpointing: its plan is made again, in other memory
    _, ref, x, y, w = operands()
    experts = torch.randint(-1, E, (T, k), device="cuda", generator=torch.Generator("cuda").manual_seed(5))
    x, w = x.requires_grad_(), w.requires_grad_()

    def block(a, b):
        plan = gbce.moe_sort(experts, E, 4)
        return gbce.combine_tokens(gbce.dispatch_tokens(a, plan), plan, b)
    d_out = x.detach().flip(0)
    want = torch.autograd.grad(block(x, w), (x, w), d_out)
    out = checkpoint(block, x, w, use_reentrant=False)
    filler = [torch.full((ref.rows * 4,), 7, device="cuda", dtype=torch.int32) for _ in range(8)]
    got = torch.autograd.grad(out, (x, w), d_out)
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and len(filler) == 8
    # each token's own row comes back, times the sum of its weights in use
    used = torch.where(ref.position >= 0, w.detach(), 0.0).double().sum(1, keepdim=True)
    near(out, used * x.detach().double(), 2.0 ** -21 * used * x.detach().double().abs() + 2.0 ** -120, "out")
