"""The router, the expert permutation, the output layer's losses and the gradient norm together, as a
mixture-of-experts training step and a decoding step use them.  Each call's result is checked against the
64-bit plain form of what it was given (tolerances in head_ref and permute_ref), so no tolerance spans
several calls."""
import pytest
import torch

import cross_entropy_loss_ce_gb300 as gbce
from head_ref import HeadRef, MoeRef, make_head, near
from permute_ref import PlanRef, clip_ref, combine_bwd_ref, combine_ref, norm_ref

pytestmark = pytest.mark.gpu


def experts_of(rows, plan, weights):
    """Each expert's product on its segment of the rows (segments are padded: their sizes are no matter)."""
    at = plan.offsets.tolist()
    return torch.cat([rows[a:b] @ w for a, b, w in zip(at, at[1:], weights)] + [rows[at[-1]:, :weights.shape[2]]])


@pytest.mark.parametrize("T,H,E,k,align", [(300, 64, 6, 2, 16), (2000, 128, 16, 4, 128)])
def test_training_step(T, H, E, k, align):
    V, bf16 = 1000, torch.bfloat16
    hidden, head, targets = make_head(T, H, V, bf16, ignored=0.1)
    g = torch.Generator("cuda").manual_seed(T)
    router = (torch.randn(H, E, device="cuda", generator=g) / H ** 0.5).to(bf16).requires_grad_()
    up = (torch.randn(E, H, H, device="cuda", generator=g) / H ** 0.5).to(bf16).requires_grad_()
    x, head = hidden.contiguous().requires_grad_(), head.contiguous().requires_grad_()
    logits = (x @ router).float()
    logits.retain_grad()
    top = logits.topk(k, 1)
    experts = torch.where((targets == -100)[:, None], -1, top.indices)  # tokens that do not count go nowhere
    weights = torch.softmax(top.values, 1)
    weights.retain_grad()
    plan = gbce.moe_sort(experts, E, align)
    rows = gbce.dispatch_tokens(x, plan)
    y = experts_of(rows, plan, up)
    y.retain_grad()
    rows.retain_grad()
    mixed = gbce.combine_tokens(y, plan, weights)
    mixed.retain_grad()
    loss = gbce.linear_cross_entropy(mixed, head, targets)
    balance, counts = gbce.moe_balance_loss(logits, experts, 1e-2, 1e-3)
    (loss + balance).backward()
    assert gbce.last_error() == gbce.OK

    ref = PlanRef(experts, E, align)
    ref.check(plan)
    assert torch.equal(counts, plan.counts.long())  # the same choices, counted by both
    token = ref.source.long().clamp_min(0) // k
    assert torch.equal(rows, torch.where((ref.source >= 0)[:, None], x[token], 0.0))
    near(mixed, *combine_ref(y.detach(), ref.position, weights.detach()), "mixed")
    head_ref = HeadRef(mixed.detach(), head.detach(), targets)
    near(loss, head_ref.loss, head_ref.loss_tol, "loss")
    near(mixed.grad, head_ref.d_hidden, head_ref.dh_tol, "d_mixed")
    near(head.grad, head_ref.d_weight, head_ref.dw_tol, "d_head")
    moe_ref = MoeRef(logits.detach(), experts, 1e-2, 1e-3)
    near(balance, moe_ref.loss, moe_ref.loss_tol, "balance")
    (d_y, y_tol), (d_w, w_tol) = combine_bwd_ref(mixed.grad, y.detach(), ref.position, weights.detach())
    near(y.grad, d_y, y_tol, "d_y")
    near(weights.grad, d_w, w_tol, "d_weights")
    # the hidden states' gradient comes by two ways, the dispatch and the router, each rounded to bf16 and added
    through, tol = combine_ref(rows.grad, ref.position, None)
    by_router = logits.grad.to(bf16) @ router.detach().t()
    total = through + by_router.double()
    near(x.grad, total, tol + 2.0 ** -8 * total.abs() + 2.0 ** -126, "d_hidden")

    grads = [p.grad for p in (router, up, head, x)]
    before = [t.clone() for t in grads]
    norm, rel = norm_ref(before, 2.0)
    limit = float(norm) / 3
    got = gbce.clip_grad_norm(grads, limit)
    near(got, norm.cuda(), (rel + 2.0 ** -24) * float(norm), "norm")
    for now, was in zip(grads, before):
        near(now, *clip_ref(was, norm, rel, limit, 1e-6), "clipped")


@pytest.mark.parametrize("T", [1, 9])
def test_decoding_step_captured(T):
    H, E, k, V, f16 = 128, 16, 4, 2000, torch.float16
    hidden, head, _ = make_head(T, H, V, f16)
    x = hidden.contiguous()
    g = torch.Generator("cuda").manual_seed(T)
    experts = torch.empty(T, k, device="cuda", dtype=torch.int64)
    weights = torch.empty(T, k, device="cuda")

    def route():
        top = torch.randn(T, E, device="cuda", generator=g).topk(k, 1)
        experts.copy_(top.indices)
        weights.copy_(torch.softmax(top.values, 1))

    def step():
        plan = gbce.moe_sort(experts, E)
        rows = gbce.moe_dispatch(x, plan)
        out = gbce.moe_combine(rows * 2, plan, weights)  # experts that double
        return plan, rows, out, gbce.linear_greedy(out, head)
    route()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan, rows, out, (token, logprob) = step()
    for _ in range(3):
        route()
        x.mul_(-0.75)
        graph.replay()
        torch.cuda.synchronize()
        ref = PlanRef(experts, E)
        ref.check(plan)
        assert torch.equal(rows, x[ref.source.long() // k])
        near(out, *combine_ref(rows * 2, ref.position, weights), "out")
        head_ref = HeadRef(out, head)
        best = head_ref.x.gather(1, token[:, None]).squeeze(1)
        assert bool((best >= head_ref.x.amax(1) - 2 * head_ref.D).all())
        near(logprob, best - head_ref.lse, 2 * head_ref.D + 2.0 ** -19 * (1 + head_ref.lse.abs()), "logprob")
