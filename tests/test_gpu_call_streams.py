"""Calls with ``stream=`` of a side stream while torch's current stream is busy: what a call allocates or
fills for itself belongs to its stream, so neither a number given as a factor nor a block that work of the
current stream still uses can reach its results (GPU)."""
import pytest
import torch

import cross_entropy_loss_ce_gb300 as gbce
from head_ref import make_head

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
BUSY = 200_000_000  # cycles: about a tenth of a second


def on_side_stream(call, like):
    """call(stream) while the current stream sleeps, holding just freed blocks of the sizes of ``like`` (which
    it overwrites after) and of one float (of NaN)."""
    side = torch.cuda.Stream()
    old = [torch.empty_like(t) for t in like] + [torch.full((1,), float("nan"), device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    for t in old:
        t.fill_(7)
    del old, t
    out = call(side)
    torch.cuda.synchronize()
    return out


def same(got, want):
    got, want = (x if isinstance(x, tuple) else (x,) for x in (got, want))
    return all(a is b is None or torch.equal(a, b) for a, b in zip(got, want))


def head():
    h, w, t = make_head(300, 136, 1500, BF, ignored=0.2)
    return h, w, t, gbce.linear_ce_fwd(h, w, t)[2]


def router():
    x = torch.randn(700, 48, device="cuda", generator=torch.Generator("cuda").manual_seed(2))
    return x, x.topk(4, 1).indices.contiguous()


def calls():
    h, w, t, lse = head()
    x, ex = router()
    logits = torch.randn(300, 700, device="cuda")
    y, dy = torch.softmax(logits, 1), torch.randn(300, 700, device="cuda")
    return {
        "linear_ce_fwd": lambda s: gbce.linear_ce_fwd(h, w, t, stream=s),
        "linear_ce_bwd": lambda s: gbce.linear_ce_bwd(h, w, t, lse, 2.0, stream=s),
        "linear_ce_bwd_none": lambda s: gbce.linear_ce_bwd(h, w, t, lse, 2.0, reduction="none", stream=s),
        "linear_greedy": lambda s: gbce.linear_greedy(h, w, stream=s),
        "moe_balance": lambda s: gbce.moe_balance(x, ex, 0.01, 0.001, grad_scale=2.0, stream=s),
        "softmax_fwd": lambda s: gbce.softmax_fwd(logits, stream=s),
        "softmax_bwd": lambda s: gbce.softmax_bwd(y, dy, stream=s),
    }


@pytest.mark.parametrize("name", ["linear_ce_fwd", "linear_ce_bwd", "linear_ce_bwd_none", "linear_greedy",
                                  "moe_balance", "softmax_fwd", "softmax_bwd"])
def test_results_do_not_depend_on_the_current_stream(name):
    call = calls()[name]
    want = call(None)
    torch.cuda.synchronize()
    like = [t for t in (want if isinstance(want, tuple) else (want,)) if t is not None]
    assert same(on_side_stream(call, like), want)


@pytest.mark.parametrize("name", ["ce_fwd_bwd", "ce_fwd_bwd_noalloc", "ce_fwd_bwd_ex"])
def test_losses_do_not_depend_on_the_current_stream(name):
    # these overwrite their logits: a copy of them, made beforehand, for each call
    logits, ids = torch.randn(300, 700, device="cuda"), torch.arange(300, device="cuda")
    mine = logits.clone()

    def call(x, s):
        if name == "ce_fwd_bwd_ex":
            return gbce.ce_fwd_bwd_ex(x, ids, grad_scale=2.0, want_row_loss=True, stream=s)
        return (getattr(gbce, name)(x, ids, stream=s),)

    want = call(logits, None)
    torch.cuda.synchronize()
    assert same(on_side_stream(lambda s: call(mine, s), want), want)
    assert torch.equal(mine, logits)


def test_scale_rows_by_a_number():
    x = torch.randn(300, 700, device="cuda")
    mine, want = x.clone(), gbce.scale_rows(x, 3.0)
    torch.cuda.synchronize()
    assert same(on_side_stream(lambda s: gbce.scale_rows(mine, 3.0, stream=s), []), want)


def test_host_logits_into_a_gradient_of_the_call():
    x, ids = torch.randn(300, 700).pin_memory(), torch.arange(300).pin_memory()
    want, loss = gbce.ce_fwd_bwd_host(x, ids)
    torch.cuda.synchronize()
    got, mine = on_side_stream(lambda s: gbce.ce_fwd_bwd_host(x, ids, stream=s), [want])
    assert torch.equal(got, want) and torch.equal(mine, loss)


def test_an_output_dropped_while_the_current_stream_reads_it():
    x, other = torch.randn(300, 700, device="cuda"), torch.zeros(300, 700, device="cuda")
    want, side = torch.softmax(x, 1), torch.cuda.Stream()
    torch.cuda.synchronize()
    y = gbce.softmax_fwd(x, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(BUSY)
    read = y * 1.0
    del y
    again = gbce.softmax_fwd(other, stream=side)
    torch.cuda.synchronize()
    assert torch.allclose(read, want, rtol=1e-5) and torch.allclose(again, torch.full_like(x, 1 / 700), rtol=1e-5)


def test_a_side_stream_that_captures():
    h, w, t, lse = head()
    want = gbce.linear_ce_bwd(h, w, t, lse, 2.0)
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        out = gbce.linear_ce_bwd(h, w, t, lse, 2.0, stream=side)
        main.wait_stream(side)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert same(out, want)
