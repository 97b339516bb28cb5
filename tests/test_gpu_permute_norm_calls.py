"""The expert permutation's and the norms' calls as programs make them: on side streams beside a busy current
one, from several host threads, back to back, on operands that broadcast, on another device (GPU)."""
import threading

import pytest
import torch

import cross_entropy_loss_ce_gb300 as gbce
from permute_ref import PlanRef, combine_bwd_ref, combine_ref, near, norm_ref

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
BUSY = 200_000_000  # cycles: about a tenth of a second


def routed(T, seed=0, device="cuda", H=136, E=24, k=4):
    g = torch.Generator().manual_seed(100 * seed + T)
    ex = torch.randint(-1, E, (T, k), generator=g).to(device)
    x = torch.randn(T, H, generator=g).to(BF).to(device)
    w = torch.rand(T, k, generator=g).to(device)
    grads = [torch.randn(n, generator=g).to(t).to(device) for n, t in ((T * 40 + 3, BF), (77, torch.float32), (T, torch.float16))]
    return ex, x, w, grads


def step(ex, x, w, grads, stream=None, E=24):
    """Everything once: plan, rows out and back, gradients, norm and clipped copies."""
    plan = gbce.moe_sort(ex, E, 8, stream=stream)
    rows = gbce.moe_dispatch(x, plan, stream=stream)
    out = gbce.moe_combine(rows, plan, w, stream=stream)
    d_y, d_w = gbce.moe_combine_bwd(x, rows, plan, w, stream=stream)
    if stream is None:
        outs = [torch.empty_like(t) for t in grads]
    else:
        with torch.cuda.stream(stream):
            outs = [torch.empty_like(t) for t in grads]
    norm = gbce.clip_grad_norm(grads, 2.0, outs=outs, stream=stream)
    return (plan.position, plan.source, plan.offsets, plan.counts, rows, out, d_y, d_w, norm, *outs)


def same(got, want):
    return all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("T", [60, 4000])
def test_results_do_not_depend_on_the_current_stream(T):
    case = routed(T)
    want = step(*case)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    # blocks of the results' sizes, freed while the current stream has yet to overwrite them
    old = [torch.empty_like(t) for t in want] + [torch.empty(T * 8 + 4000, device="cuda", dtype=torch.int32)]
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    for t in old:
        t.fill_(7)
    del old, t
    got = step(*case, stream=side)
    torch.cuda.synchronize()
    assert same(got, want)


def test_operands_made_on_another_stream():
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
        case = routed(3000, 1)
        got = step(*case)
    s.synchronize()
    assert same(got, step(*case))
    PlanRef(case[0], 24, 8).check(gbce.moe_sort(case[0], 24, 8))


def test_host_threads_at_once():
    cases = [routed(T, 7 + i) for i, T in enumerate((1, 33, 700, 3000, 9000, 64))]
    want = [step(*c) for c in cases]
    torch.cuda.synchronize()
    got, errors = [None] * len(cases), []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(10):
                    got[i] = step(*cases[i])
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # pragma: no cover
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(cases))]
    [th.start() for th in threads]
    [th.join() for th in threads]
    assert not errors
    assert all(same(a, b) for a, b in zip(got, want))


def test_calls_back_to_back_reuse_their_scratch_in_order():
    cases = [routed(T, 20 + i) for i, T in enumerate((5000, 64, 12000, 1, 2600))]
    outs = [[step(*c) for c in cases] for _ in range(4)]
    torch.cuda.synchronize()
    for round_ in outs[1:]:
        assert all(same(a, b) for a, b in zip(round_, outs[0]))


def test_one_plan_on_two_streams():
    ex, x, w, _ = routed(3000, 3)
    plan = gbce.moe_sort(ex, 24)
    other = x.neg()
    want = [gbce.moe_dispatch(t, plan) for t in (x, other)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [gbce.moe_dispatch(t, plan, stream=s) for _ in range(5) for s, t in zip(streams, (x, other))]
    torch.cuda.synchronize()
    assert all(torch.equal(g, want[i % 2]) for i, g in enumerate(got))


def test_broadcast_operands_and_their_gradients():
    ex, x, w, _ = routed(90, 4)
    plan, ref = gbce.moe_sort(ex, 24, 8), PlanRef(ex, 24, 8)
    one = x[:1].clone().requires_grad_()
    g = torch.randn(ref.rows, 136, device="cuda", generator=torch.Generator("cuda").manual_seed(1)).to(BF)
    rows = gbce.dispatch_tokens(one.expand(90, 136), plan)
    assert torch.equal(rows, torch.where((ref.source >= 0)[:, None], one.detach(), 0.0))
    rows.backward(g)
    each, tol = combine_ref(g, ref.position, None)
    # the library's row for each token (rounded to bf16), added by autograd in bf16 or wider and rounded once
    near(one.grad[0], each.sum(0), (tol + 2.0 ** -8 * each.abs()).sum(0) + 2.0 ** -8 * each.sum(0).abs(), "one row")
    y = g.clone().requires_grad_()
    per_token = w[:, :1].clone().requires_grad_()
    d_out = x[:, :].clone()
    gbce.combine_tokens(y, plan, per_token.expand(90, 4)).backward(d_out)
    full = per_token.detach().expand(90, 4)
    (d_y, y_tol), (d_w, w_tol) = combine_bwd_ref(d_out, y.detach(), ref.position, full)
    near(y.grad, d_y, y_tol, "d_y")
    near(per_token.grad[:, 0], d_w.sum(1), w_tol.sum(1) + 2.0 ** -22 * d_w.abs().sum(1), "one weight a token")


def test_norm_of_many_calls_in_flight():
    cases = [routed(T, 40 + i)[3] for i, T in enumerate((3, 900, 40000))]
    norms = [gbce.grad_norm(c) for _ in range(20) for c in cases]
    torch.cuda.synchronize()
    for i, n in enumerate(norms):
        want, rel = norm_ref(cases[i % 3], 2.0)
        near(n, want, (rel + 2.0 ** -24) * float(want), "norm")


@pytest.mark.skipif("torch.cuda.device_count() < 2")
def test_tensors_on_another_device_than_the_current_one():
    case = routed(700, device="cuda:1")
    got = step(*case)
    torch.cuda.synchronize(1)
    PlanRef(case[0], 24, 8).check(gbce.moe_sort(case[0], 24, 8))
    assert all(t.device.index == 1 for t in got)
