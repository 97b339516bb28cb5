"""The router's balance loss on the GPU against its 64-bit plain form (tolerances in head_ref)."""
import pytest
import torch

import cross_entropy_loss_ce_gb300 as gbce
from head_ref import MoeRef, near

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
A, B = 1e-2, 1e-3


def make(T, E, k, dtype, padded=0.0, seed=0, pad=0):
    g = torch.Generator().manual_seed(100 * seed + T + 3 * E + 11 * k)
    buf = torch.full((T, E + pad), 9.0).to(dtype)
    buf[:, :E] = (torch.randn(T, E, generator=g) + 0.7 * torch.randn(E, generator=g)).to(dtype)
    ex = buf[:, :E].float().topk(min(k, E), dim=1).indices
    if k > E:  # more slots than experts: some experts twice
        ex = torch.randint(0, E, (T, k), generator=g)
    ex[torch.rand(T, generator=g) < padded] = -1
    return buf.cuda()[:, :E], ex.cuda()


def check(x, ex, a=A, b=B, scale=None):
    ref = MoeRef(x, ex, a, b, 1.0 if scale is None else scale)
    loss, counts, grad = gbce.moe_balance(x, ex, a, b, grad_scale=scale)
    assert torch.equal(counts, ref.counts)
    near(loss, ref.loss, ref.loss_tol, "loss")
    near(grad, ref.grad, ref.grad_tol, "grad")
    return loss, counts, grad


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (5, 8, 2), (64, 8, 2), (256, 128, 8), (257, 128, 8),
                                   (300, 60, 4), (1000, 3, 1), (700, 17, 2), (500, 256, 8), (400, 512, 8),
                                   (300, 1024, 6), (33, 1000, 3), (400, 333, 2), (300, 130, 64)])
def test_shapes(T, E, k, dtype):
    x, ex = make(T, E, k, DT[dtype], padded=0.1 if T > 5 else 0.0)
    check(x, ex)
    assert gbce.last_error() == gbce.OK


@pytest.mark.parametrize("T", [40, 600])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_strides(T, dtype):
    x, ex = make(T, 24, 3, DT[dtype], pad=5)
    wide = torch.full((T, 7), 5, device="cuda", dtype=torch.int64)
    wide[:, :3] = ex
    out = torch.full((T, 31), 2.0, device="cuda", dtype=DT[dtype])
    ref = MoeRef(x, ex, A, B)
    _, counts, grad = gbce.moe_balance(x, wide[:, :3], A, B, grad=out[:, 2:26])
    assert torch.equal(counts, ref.counts)
    near(out[:, 2:26], ref.grad, ref.grad_tol, "grad")
    assert bool((out[:, :2] == 2).all() and (out[:, 26:] == 2).all())


@pytest.mark.parametrize("T", [40, 600])
def test_in_place(T):
    x, ex = make(T, 64, 4, torch.float32, padded=0.2)
    want = gbce.moe_balance(x, ex, A, B)
    y = x.clone()
    got = gbce.moe_balance(y, ex, A, B, grad=y)
    assert torch.equal(got[2], want[2]) and got[2].data_ptr() == y.data_ptr()
    assert torch.equal(got[0], want[0])


@pytest.mark.parametrize("T", [40, 600])
def test_no_token_counts(T):
    x, ex = make(T, 16, 2, torch.float32)
    ex.fill_(-1)
    loss, counts, grad = gbce.moe_balance(x, ex, A, B)
    assert bool(torch.isnan(loss)) and not bool(counts.any()) and not bool(grad.any())


def test_no_tokens():
    x, ex = torch.empty(0, 16, device="cuda"), torch.empty(0, 2, device="cuda", dtype=torch.int64)
    loss, counts, grad = gbce.moe_balance(x, ex, A, B)
    assert bool(torch.isnan(loss)) and not bool(counts.any()) and grad.shape == (0, 16)


@pytest.mark.parametrize("T", [40, 600])
def test_empty_slots_and_doubled_experts(T):
    x, ex = make(T, 16, 4, torch.bfloat16, padded=0.1)
    ex[::3, 2:] = -1
    ex[1::3, 1] = ex[1::3, 0]
    check(x, ex)


@pytest.mark.parametrize("T", [40, 600])
def test_bad_slots(T):
    x, ex = make(T, 16, 2, torch.float32)
    ex[3, 1], ex[7, 0] = 16, -2
    gbce.last_error()
    loss, counts, grad = check(x, ex)
    assert gbce.last_error() == gbce.ERR_BAD_TARGET
    assert bool(torch.isnan(loss)) and not bool(grad[3].any()) and not bool(grad[7].any())


@pytest.mark.parametrize("T", [40, 600])
def test_masked_experts_and_padded_rows_of_anything(T):
    x, ex = make(T, 16, 2, torch.float32, padded=0.3)
    top = ex[:, :1].clamp_min(0)
    off = torch.zeros_like(x, dtype=torch.bool).scatter_(1, (top + 5) % 16, True)
    x[off] = float("-inf")        # an expert a token may not use
    x[(ex < 0).all(1)] = float("nan")  # padding may hold anything
    ref = MoeRef(torch.where((ex < 0).all(1, keepdim=True), 0.0, x), ex, A, B)
    loss, counts, grad = gbce.moe_balance(x, ex, A, B)
    near(loss, ref.loss, ref.loss_tol, "loss")
    near(grad, ref.grad, ref.grad_tol, "grad")


def test_scale_and_coefficients():
    x, ex = make(500, 32, 2, torch.float32)
    check(x, ex, 1.0, 0.0, scale=-2.5)
    check(x, ex, 0.0, 1.0, scale=1024.0)
    loss, counts, grad = gbce.moe_balance(x, ex, A, B, want_loss=False)
    assert loss is None and torch.equal(grad, gbce.moe_balance(x, ex, A, B)[2])
    assert gbce.moe_balance(x, ex, A, B, want_grad=False)[2] is None


def test_evenly_spread_tokens_cost_the_coefficient():
    E, k = 16, 2
    x = torch.zeros(800, E, device="cuda")
    ex = torch.arange(1600, device="cuda").reshape(800, 2) % E
    loss, counts, grad = gbce.moe_balance(x, ex, 1.0)
    assert bool((counts == 100).all()) and not bool(grad.any())
    assert abs(float(loss) - 1.0) <= 2.0 ** -20


@pytest.mark.parametrize("T", [50, 700])
def test_gradient_against_differences(T):
    x, ex = make(T, 24, 3, torch.float32, padded=0.1)
    grad = gbce.moe_balance(x, ex, 1.0, 0.1)[2].double()
    v = torch.randn(x.shape, device="cuda", dtype=torch.float64, generator=torch.Generator("cuda").manual_seed(3))
    x64, e = x.double(), 1e-4
    diff = (MoeRef(x64.double() + e * v, ex, 1.0, 0.1).loss - MoeRef(x64 - e * v, ex, 1.0, 0.1).loss) / (2 * e)
    tol = (MoeRef(x, ex, 1.0, 0.1).grad_tol * v.abs()).sum() + 1e-7
    assert abs(float((grad * v).sum() - diff)) <= float(tol)


def test_autograd_form():
    x, ex = make(600, 64, 4, torch.bfloat16, padded=0.1)
    leaf = x.reshape(20, 30, 64).clone().requires_grad_()
    loss, counts = gbce.moe_balance_loss(leaf, ex.reshape(20, 30, 4), A, B)
    (2.0 * loss).backward(retain_graph=True)
    ref = MoeRef(x, ex, A, B, 2.0)
    near(leaf.grad.reshape(600, 64), ref.grad, ref.grad_tol, "grad")
    assert torch.equal(counts, ref.counts)
    first, leaf.grad = leaf.grad.clone(), None
    (2.0 * loss).backward()
    assert torch.equal(first, leaf.grad)


def test_same_bits_on_two_streams_and_captured():
    cases = [make(T, 60, 4, torch.float32, padded=0.1) for T in (200, 3000)]
    want = [gbce.moe_balance(x, ex, A, B) for x, ex in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [gbce.moe_balance(x, ex, A, B, stream=s) for _ in range(3) for s, (x, ex) in zip(streams, cases)]
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert all(torch.equal(p, q) for p, q in zip(g, want[i % 2]))
    graphs = []
    for x, ex in cases:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = gbce.moe_balance(x, ex, A, B)
        graphs.append((graph, out))
    for (x, ex), (graph, out) in zip(cases, graphs):
        x.neg_()
        graph.replay()
        torch.cuda.synchronize()
        ref = MoeRef(x, ex, A, B)
        near(out[0], ref.loss, ref.loss_tol, "loss")
        near(out[2], ref.grad, ref.grad_tol, "grad")


@pytest.mark.parametrize("T,k", [(2048, 4), (2049, 4), (8192, 1), (8193, 1), (1025, 8)])
def test_the_ways_of_counting(T, k):
    # up to 8192 slots one CTA counts, above several do
    x, ex = make(T, 48, k, torch.bfloat16, padded=0.2)
    check(x, ex)
