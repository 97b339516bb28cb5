"""Calls of the output-layer and router operators as programs make them: refusals on the GPU, captured
graphs, several streams and threads, another current device, a wait that runs out (GPU)."""
import ctypes
import os
import subprocess
import sys
import threading

import pytest
import torch

import cross_entropy_loss_ce_gb300 as gbce
from head_ref import HeadRef, MoeRef, make_head, near

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def step(h, w, t):
    loss, row, lse = gbce.linear_ce_fwd(h, w, t)
    return (loss, row, lse, *gbce.linear_ce_bwd(h, w, t, lse), *gbce.linear_greedy(h, w))


def check_step(out, h, w, t):
    ref = HeadRef(h, w, t)
    near(out[0], ref.loss, ref.loss_tol, "loss")
    near(out[1], ref.row_loss, ref.row_tol, "row loss")
    near(out[3], ref.d_hidden, ref.dh_tol, "d_hidden")
    near(out[4], ref.d_weight, ref.dw_tol, "d_weight")
    near(out[6], ref.logprob, 2 * ref.D + 2.0 ** -19 * (1 + ref.lse.abs()), "logprob")


def test_refusals_on_the_device():
    h, w, t = make_head(8, 64, 100, BF)
    with pytest.raises(ValueError, match="overlapping"):
        gbce.linear_ce_fwd(h[:1].expand(8, 64), w, t)
    with pytest.raises(ValueError, match="columns"):
        gbce.linear_ce_fwd(h, w[:, :32], t)
    with pytest.raises(TypeError, match="float16"):
        gbce.linear_ce_fwd(h, w.half(), t)
    with pytest.raises(gbce.GbceError) as e:
        gbce.linear_ce_fwd(h.float(), w.float(), t)
    assert e.value.code == gbce.ERR_DTYPE
    with pytest.raises(ValueError, match="targets"):
        gbce.linear_ce_fwd(h, w, t.int())
    with pytest.raises(ValueError, match="targets"):
        gbce.linear_ce_fwd(h, w, t.cpu())
    with pytest.raises(ValueError, match="unit column"):
        gbce.linear_greedy(h.T, w[:, :8])
    _, _, lse = gbce.linear_ce_fwd(h, w, t)
    with pytest.raises(ValueError, match="lse"):
        gbce.linear_ce_bwd(h, w, t, lse[:4])
    with pytest.raises(ValueError, match="grad_scale"):
        gbce.linear_ce_bwd(h, w, t, lse, torch.ones(8, device="cuda"))
    with pytest.raises(ValueError, match="shares memory"):
        gbce.linear_ce_bwd(h, w, t, lse, d_hidden=h)
    with pytest.raises(ValueError, match="shares memory"):
        gbce.linear_ce_bwd(h, w, t, lse, d_weight=w)
    x, ex = torch.zeros(8, 16, device="cuda"), torch.zeros(8, 2, device="cuda", dtype=torch.int64)
    with pytest.raises(ValueError, match="experts"):
        gbce.moe_balance(x, ex[:4], 0.1)
    with pytest.raises(ValueError, match="experts"):
        gbce.moe_balance(x, ex.int(), 0.1)
    with pytest.raises(ValueError, match="grad"):
        gbce.moe_balance(x, ex, 0.1, grad=torch.zeros(8, 16, device="cuda", dtype=BF))
    with pytest.raises(gbce.GbceError) as e:
        gbce.moe_balance(torch.zeros(4, 1025, device="cuda"), ex[:4], 0.1)
    assert e.value.code == gbce.ERR_SIZE


def test_two_graphs_replayed_at_once():
    # each graph allocates its own scratch: replays on two streams do not meet
    cases = [make_head(M, 136, 1500, BF, seed=s, ignored=0.2) for s, M in enumerate((300, 300, 40))]
    step(*cases[0])
    torch.cuda.synchronize()
    graphs = []
    for c in cases:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step(*c)
        graphs.append((g, out))
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(5):
        for s, (g, _) in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for c, (_, out) in zip(cases, graphs):
        check_step(out, *c)


def test_autograd_step_captured_and_raw_gradients_beside_an_eager_graph():
    h, w, t = make_head(100, 64, 300, BF)
    hl, wl = h.clone().requires_grad_(), w.clone().requires_grad_()
    x = torch.randn(300, 16, device="cuda", requires_grad=True)
    ex = x.detach().topk(2, 1).indices.contiguous()

    def total():
        return gbce.linear_cross_entropy(hl, wl, t).float() + gbce.moe_balance_loss(x, ex, 0.1, 0.01)[0]

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):  # the leaves' first use, as torch asks of a step to be captured
        want = torch.autograd.grad(total(), (hl, wl, x))
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        grads = torch.autograd.grad(total(), (hl, wl, x))
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(grads, want))
    # the raw calls keep nothing of the leaves: an eager graph of them may live on
    eager = total()
    g2 = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g2):
        _, _, lse = gbce.linear_ce_fwd(hl.detach(), wl.detach(), t)
        raw = gbce.linear_ce_bwd(hl.detach(), wl.detach(), t, lse)
        raw_x = gbce.moe_balance(x.detach(), ex, 0.1, 0.01)[2]
    g2.replay()
    got = torch.autograd.grad(eager, (hl, wl, x))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((*raw, raw_x), want))
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_host_threads_at_once():
    cases = [make_head(M, 136, 1500, BF, seed=7 + i, ignored=0.1) for i, M in enumerate((5, 33, 70, 300, 1100, 64))]
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
    for a, b in zip(got, want):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_calls_back_to_back_reuse_their_scratch_in_order():
    # the pool hands one call's scratch to the next: results of many calls in flight
    cases = [make_head(M, 72, 700, BF, seed=20 + i, ignored=0.3) for i, M in enumerate((300, 64, 1030, 1, 600))]
    outs = [[step(*c) for c in cases] for _ in range(4)]
    torch.cuda.synchronize()
    for round_ in outs:
        for c, out in zip(cases, round_):
            check_step(out, *c)
        assert all(torch.equal(a, b) for o, p in zip(round_, outs[0]) for a, b in zip(o, p))


def test_operands_made_on_another_stream():
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
        h, w, t = make_head(200, 64, 500, BF)
        out = step(h, w, t)
    s.synchronize()
    check_step(out, h, w, t)


def test_losses_of_a_mixture_of_experts_step():
    # a training step that uses all of them: hidden states -> router loss and output-layer loss
    T, K, E, V, k = 512, 128, 16, 1000, 2
    g = torch.Generator(device="cuda").manual_seed(1)
    hidden = torch.randn(T, K, device="cuda", generator=g).to(BF).requires_grad_()
    head = (torch.randn(V, K, device="cuda", generator=g) / K ** 0.5).to(BF).requires_grad_()
    router = torch.randn(E, K, device="cuda", generator=g).to(BF).requires_grad_()
    t = torch.randint(0, V, (T,), device="cuda", generator=g)
    t[::7] = -100
    logits = (hidden @ router.T).float()
    experts = logits.detach().topk(k, 1).indices.contiguous()
    experts[t == -100] = -1
    balance, counts = gbce.moe_balance_loss(logits, experts, 0.01, 0.001)
    loss = gbce.linear_cross_entropy(hidden, head, t) + balance
    loss.backward()
    assert int(counts.sum()) == k * int((t != -100).sum())
    ref, mref = HeadRef(hidden.detach(), head.detach(), t), MoeRef(logits.detach(), experts, 0.01, 0.001)
    near(loss.detach(), ref.loss + mref.loss, ref.loss_tol + mref.loss_tol + 1e-6, "loss")
    near(head.grad, ref.d_weight, ref.dw_tol, "head gradient")
    dr = mref.grad.T @ hidden.detach().double()  # autograd rounds the logits' gradient to bf16 on its way
    tol = 2.0 ** -7 * (mref.grad.abs().T @ hidden.detach().double().abs()) + 1e-6
    near(router.grad, dr, tol, "router gradient")
    tokens, logprob = gbce.linear_greedy(hidden.detach(), head.detach())
    near(logprob, ref.logprob, 2 * ref.D + 2.0 ** -19 * (1 + ref.lse.abs()), "logprob")


@pytest.mark.skipif("torch.cuda.device_count() < 2")
def test_tensors_on_another_device_than_the_current_one():
    h, w, t = make_head(70, 64, 300, BF, device="cuda:1")
    out = step(h, w, t)
    torch.cuda.synchronize(1)
    check_step(out, h, w, t)


@pytest.mark.parametrize("M,drop", [(20, 0), (300, 0), (300, 3)])
def test_a_wait_that_runs_out_ends_the_call(M, drop):
    # one operand copy is left out on purpose: its waits give up after 2 s, the call
    # reports it, and the next one is whole
    h, w, t = make_head(M, 320, 1500, BF)
    fn = gbce.load_library().gbce_test_failure_path
    fn.argtypes, fn.restype = [ctypes.c_int64], ctypes.c_int
    want = step(h, w, t)
    assert gbce.last_error() == gbce.OK
    try:
        assert fn(drop) == gbce.OK
        loss, _, _ = gbce.linear_ce_fwd(h, w, t)
        assert gbce.last_error() == gbce.ERR_TIMEOUT
        assert bool(torch.isnan(loss))
        tok, _ = gbce.linear_greedy(h, w)
        assert gbce.last_error() == gbce.ERR_TIMEOUT
        assert bool(((tok >= 0) & (tok < 1500)).all())
        gbce.linear_ce_bwd(h, w, t, want[2])
        assert gbce.last_error() == gbce.ERR_TIMEOUT
    finally:
        torch.cuda.synchronize()
        fn(-1)
    got = step(h, w, t)
    assert gbce.last_error() == gbce.OK
    assert all(torch.equal(a, b) for a, b in zip(got, want))


FIRST_CALLS = r"""
import os, sys
sys.path[:0] = [os.getcwd(), os.path.join(os.getcwd(), "tests")]
import torch
import cross_entropy_loss_ce_gb300 as gbce
from head_ref import HeadRef, MoeRef, make_head, near
torch.zeros(1, device="cuda")
cases = [make_head(M, 72, 900, torch.bfloat16, ignored=0.2) for M in (20, 300, 1300)]
x = torch.randn(3000, 48, device="cuda")
ex = x.topk(4, 1).indices.contiguous()
graph, outs = torch.cuda.CUDAGraph(), []
with torch.cuda.graph(graph):
    for h, w, t in cases:
        loss, row, lse = gbce.linear_ce_fwd(h, w, t)
        outs.append((loss, row, *gbce.linear_ce_bwd(h, w, t, lse), *gbce.linear_greedy(h, w)))
    moe = gbce.moe_balance(x, ex, 0.01, 0.001)
graph.replay()
torch.cuda.synchronize()
for (h, w, t), (loss, row, dh, dw, tok, lp) in zip(cases, outs):
    ref = HeadRef(h, w, t)
    near(loss, ref.loss, ref.loss_tol, "loss")
    near(dh, ref.d_hidden, ref.dh_tol, "d_hidden")
    near(dw, ref.d_weight, ref.dw_tol, "d_weight")
    near(lp, ref.logprob, 2 * ref.D + 2.0 ** -19 * (1 + ref.lse.abs()), "logprob")
ref = MoeRef(x, ex, 0.01, 0.001)
assert torch.equal(moe[1], ref.counts)
near(moe[0], ref.loss, ref.loss_tol, "balance loss")
near(moe[2], ref.grad, ref.grad_tol, "balance gradient")
print("captured first calls: ok")
"""


def test_a_process_whose_first_calls_are_captured():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured first calls: ok" in r.stdout, r.stdout + r.stderr


def test_weights_past_32_bit_offsets():
    # 1.1 million classes of 2048: 2.25e9 values, the last rows beyond 2^31
    V, K, M = 1_100_000, 2048, 5
    g = torch.Generator(device="cuda").manual_seed(3)
    w = torch.empty(V, K, device="cuda", dtype=BF)
    for i in range(0, V, 100_000):
        w[i:i + 100_000] = torch.randn(100_000, K, device="cuda", generator=g).to(BF) / 64
    t = torch.tensor([V - 1, 3, V - 40_000, -100, 600_000], device="cuda")
    h = (w[t.clamp_min(0)].float() * 40).to(BF)
    h[3] = (w[V - 7].float() * 40).to(BF)
    tokens, logprob = gbce.linear_greedy(h, w)
    assert tokens.tolist() == [V - 1, 3, V - 40_000, V - 7, 600_000]
    loss, row, lse = gbce.linear_ce_fwd(h, w, t, reduction="sum")
    x = torch.cat([h.double() @ w[i:i + 100_000].double().T for i in range(0, V, 100_000)], 1)
    want = torch.logsumexp(x, 1)
    D = (K / 16 + 8) * 2.0 ** -23 * max(float((h[i].abs().double() @ w[:1000].abs().double().T).amax()) for i in range(M)) * 4
    keep = t >= 0
    near(lse[keep], want[keep], D + 2.0 ** -20 * (1 + want[keep].abs()), "lse")
    near(logprob, x.amax(1) - want, 2 * D + 2.0 ** -19 * (1 + want.abs()), "logprob")
    dh, dw = gbce.linear_ce_bwd(h, w, t, lse, reduction="sum")
    p = torch.exp(x - want[:, None]) * keep[:, None]
    p[keep, t[keep]] -= 1
    for rows in (slice(0, 8), slice(600_000, 600_004), slice(V - 40_000, V - 39_996), slice(V - 8, V)):
        A = (p[:, rows].abs() + 1e-6).T @ h.double().abs()
        near(dw[rows], p[:, rows].T @ h.double(), (2.0 ** -8 + 2 * D + 2.0 ** -18) * A * 2, "d_weight")
    A = torch.zeros(M, K, device="cuda", dtype=torch.float64)
    want_dh = torch.zeros_like(A)
    for i in range(0, V, 100_000):
        block = w[i:i + 100_000].double()
        want_dh += p[:, i:i + 100_000] @ block
        A += p[:, i:i + 100_000].abs() @ block.abs()
    near(dh, want_dh, (2.0 ** -7 + 2 * D) * A + 2.0 ** -8 * want_dh.abs() + 2.0 ** -18 * w[t.clamp_min(0)].double().abs(), "d_hidden")


def test_router_logits_past_32_bit_offsets():
    # 2.1 million tokens of 1024 experts: 2.15e9 values
    T, E, k = 2_100_000, 1024, 2
    x = torch.empty(T, E, device="cuda", dtype=BF)
    g = torch.Generator(device="cuda").manual_seed(4)
    for i in range(0, T, 300_000):
        x[i:i + 300_000] = torch.randn(300_000, E, device="cuda", generator=g).to(BF)
    ex = torch.randint(0, E, (T, k), device="cuda", generator=g)
    ex[:, 0] = ex[:, 0] // 2  # the lower half is chosen more
    ex[-1] = -1
    loss, counts, grad = gbce.moe_balance(x, ex, 1.0, 0.0, grad_scale=1e6)
    assert torch.equal(counts, torch.bincount(ex[:-1].reshape(-1), minlength=E))
    n, f = T - 1, counts.double()
    total = sum(float((torch.softmax(x[i:i + 100_000].double(), 1)[:min(100_000, n - i)] @ f).sum()) for i in range(0, T, 100_000))
    assert abs(float(loss) - E / (k * n * n) * total) <= 2.0 ** -19
    last = x[-50:].double()
    p, c = torch.softmax(last, 1), f - f.mean()
    want = 1e6 * E / (k * n * n) * p * (c - (p @ c)[:, None])
    want[-1] = 0
    size = 1e6 * E / (k * n * n) * p * (c.abs() + (p @ c.abs())[:, None])
    near(grad[-50:], want, 2.0 ** -19 * size + 2.0 ** -8 * want.abs() + 2.0 ** -126, "grad")
