"""The norm of many tensors and its limit on the GPU, against plain forms (tolerances in permute_ref)."""
import math

import pytest
import torch

import cross_entropy_loss_ce_gb300 as gbce
from permute_ref import clip_ref, near, norm_ref

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
KINDS = [2.0, 1.0, math.inf]


def make(shapes, dtypes, size=1.0, seed=0):
    g = torch.Generator("cuda").manual_seed(seed)
    return [(torch.randn(*s, device="cuda", generator=g) * size).to(dtypes[i % len(dtypes)])
            for i, s in enumerate(shapes)]


def check(tensors, kind, max_norm, eps=1e-6, places=None):
    """The norm, the clipped copies, and the same in place."""
    want, rel = norm_ref(tensors, kind)
    norm = gbce.grad_norm(tensors, kind)
    assert norm.dtype == torch.float32 and norm.dim() == 0
    near(norm, want.cuda(), (rel + 2.0 ** -24) * float(want) + 2.0 ** -126, "norm")
    refs = [clip_ref(t, want, rel, max_norm, eps) for t in tensors]
    outs = places or [torch.full_like(t, 3.0) for t in tensors]
    assert torch.equal(gbce.clip_grad_norm(tensors, max_norm, kind, eps, outs=outs), norm)
    for o, (r, tol) in zip(outs, refs):
        near(o, r, tol, "clipped")
    if places is None:
        mine = [t.clone() for t in tensors]
        assert torch.equal(gbce.clip_grad_norm(mine, max_norm, kind, eps), norm)
        assert all(torch.equal(a, b) for a, b in zip(mine, outs))
    return norm


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("shapes", [[(1,)], [(7,), (0,), (3, 5)], [(64, 96), (96,), (1000, 3)], [(16385,), (2048, 8)],
                                    [(3, 40001), (5,), (70001,)], [(2, 3, 4, 5)] * 40])
def test_shapes(shapes, dtype, kind):
    tensors = make(shapes, [DT[dtype]])
    check(tensors, kind, 0.5)
    check(tensors, kind, 1e9)  # keeps the limit: bits are copied


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n", [63, 64, 65, 1023, 1025, 2600])
def test_many_tensors(n, kind):
    tensors = make([((i * 37) % 211,) for i in range(n)], [torch.float32, torch.bfloat16, torch.float16])
    check(tensors, kind, 2.0)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_places_that_do_not_start_on_16_bytes(dtype):
    # every start of a tensor against every start of its result, whole tiles and short ones
    dt = DT[dtype]
    step = 16 // torch.empty(0, dtype=dt).element_size()
    for n in (5, 100, 40000):
        src = make([(step * step * (n + 2 * step),)], [dt])[0]
        dst = torch.full_like(src, 9.0)
        tensors, outs = [], []
        for i in range(step * step):
            at = i * (n + 2 * step) // step * step
            tensors.append(src[at + i % step:at + i % step + n])
            outs.append(dst[at + i // step:at + i // step + n])
        check(tensors, 2.0, 1.0, places=outs)
        left = torch.ones_like(dst, dtype=torch.bool)
        for o in outs:
            left[o.storage_offset():o.storage_offset() + n] = False
        assert bool((dst[left] == 9.0).all())


@pytest.mark.parametrize("dtype,size", [("f32", 1e-20), ("f32", 1e-36), ("f32", 1e18), ("f32", 1e32), ("bf16", 1e-25),
                                        ("bf16", 1e30), ("f16", 1e-6), ("f16", 3000.0), ("f32", 3e-15),
                                        ("bf16", 1e-14), ("f32", 1e15)])
@pytest.mark.parametrize("kind", KINDS)
def test_sizes_whose_squares_leave_fp32(dtype, size, kind):
    tensors = make([(3000,), (40, 41), (9,)], [DT[dtype]], size)
    want = float(norm_ref(tensors, kind)[0])
    check(tensors, kind, want / 8, eps=0.0)
    # beside others: tiny and huge tensors of one call
    check(tensors + make([(5000,)], [torch.float32], 1.0, 1), kind, 0.25 * max(want, 1.0), eps=0.0)


@pytest.mark.parametrize("kind", [2.0, 1.0])
def test_a_norm_past_fp32(kind):
    tensors = [torch.full((50000,), 3e38, device="cuda"), torch.ones(5, device="cuda")]
    norm = gbce.grad_norm(tensors, kind)
    assert bool(torch.isinf(norm))
    want = float(norm_ref(tensors, kind)[0])
    outs = [torch.empty_like(t) for t in tensors]
    gbce.clip_grad_norm(tensors, 1e30, kind, 0.0, outs=outs)  # the factor is formed in fp64
    for o, t in zip(outs, tensors):
        near(o, *clip_ref(t, want, 70 * 2.0 ** -24, 1e30, 0.0), "clipped")


def test_a_factor_below_fp32s_normal_numbers():
    t = torch.full((5000,), 1e38, device="cuda")
    out = torch.empty_like(t)
    norm = norm_ref([t], 2.0)[0]
    gbce.clip_grad_norm([t], 7.0, 2.0, 0.0, outs=[out])      # 1e-39
    near(out, *clip_ref(t, norm, 36 * 2.0 ** -24, 7.0, 0.0), "clipped")
    gbce.clip_grad_norm([t], 0.0, outs=[out])
    assert not bool(out.any())


@pytest.mark.parametrize("kind", KINDS)
def test_infinities_and_nan(kind):
    tensors = make([(5000,), (300,)], [torch.float32, torch.bfloat16])
    tensors[0][4321] = -math.inf
    assert float(gbce.grad_norm(tensors, kind)) == math.inf
    mine = [t.clone() for t in tensors]
    gbce.clip_grad_norm(mine, 1.0, kind)  # f = 0
    assert bool(torch.isnan(mine[0][4321])) and int((mine[0] != 0).sum()) == 1 and not bool(mine[1].any())
    tensors[1][7] = math.nan
    assert bool(torch.isnan(gbce.grad_norm(tensors, kind)))
    gbce.clip_grad_norm(tensors, 1.0, kind)
    assert all(bool(torch.isnan(t).all()) for t in tensors)


def test_zeros_and_nothing():
    for kind in KINDS:
        assert float(gbce.grad_norm([], kind)) == 0.0
        assert float(gbce.clip_grad_norm([None, torch.empty(0, device="cuda")], 1.0, kind)) == 0.0
        z = torch.zeros(70000, device="cuda", dtype=torch.bfloat16)
        z[1] = -0.0
        assert float(gbce.clip_grad_norm([z, None], 1.0, kind)) == 0.0 and not bool(z.any())
    t = torch.tensor([3.0, 4.0], device="cuda")
    assert float(gbce.grad_norm(t)) == 5.0 and float(gbce.grad_norm([t, None, t])) == pytest.approx(50 ** 0.5, rel=1e-6)


def test_other_orders_of_axes():
    t = make([(40, 30, 8)], [torch.float32])[0].permute(2, 0, 1)
    w = make([(64, 32)], [torch.bfloat16], 1.0, 1)[0].t()
    check([t, w], 2.0, 0.5)
    check([t[:, :5]], 2.0, 0.5)  # the first 5 of the outermost axis in memory: one stretch
    with pytest.raises(ValueError, match="one stretch"):
        gbce.grad_norm([t[:, :, :5]])
    with pytest.raises(ValueError, match="one stretch"):
        gbce.grad_norm([t[:1].expand(4, -1, -1)])
    with pytest.raises(ValueError, match="outs must match"):
        gbce.clip_grad_norm([t], 1.0, outs=[torch.empty(t.shape, device="cuda")])


def test_a_tensor_past_32_bit_offsets():
    n = 2 ** 32 + 70001
    t = torch.zeros(n, device="cuda", dtype=torch.bfloat16)
    at = torch.tensor([0, 2 ** 31, 2 ** 32 - 1, 2 ** 32, n - 1], device="cuda")
    t[at] = torch.tensor([1.0, 2.0, 2.0, 4.0, 24.0], device="cuda", dtype=torch.bfloat16)
    assert float(gbce.grad_norm([t], 1.0)) == 33.0 and float(gbce.grad_norm([t], math.inf)) == 24.0
    want = 601 ** 0.5
    assert abs(float(gbce.clip_grad_norm([t], want / 4, 2.0, 0.0)) - want) <= 1e-5 * want
    near(t[at], torch.tensor([0.25, 0.5, 0.5, 1.0, 6.0]).cuda().double(), 6 * 2.0 ** -8, "clipped")
    assert int(torch.count_nonzero(t)) == 5


def test_same_bits_on_two_streams_and_captured():
    sets = [make([(300, 70), (9,)] * 3, [torch.float32, torch.bfloat16]),
            make([(3000, 700), (90,)] * 40, [torch.float16, torch.bfloat16])]
    outs = [[torch.empty_like(t) for t in s] for s in sets]
    want = [gbce.clip_grad_norm(s, 1.0, outs=o) for s, o in zip(sets, outs)]
    kept = [[t.clone() for t in o] for o in outs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [gbce.clip_grad_norm(s, 1.0, outs=o, stream=st) for _ in range(3) for st, s, o in zip(streams, sets, outs)]
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert torch.equal(g, want[i % 2])
    graphs = []
    for s, o in zip(sets, outs):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            graphs.append((graph, gbce.clip_grad_norm(s, 1.0, outs=o)))
    for s, o, k, (graph, norm), w in zip(sets, outs, kept, graphs, want):
        [t.neg_() for t in s]
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(norm, w) and all(torch.equal(a, -b) for a, b in zip(o, k))


def test_refusals_on_the_device():
    a, b = torch.ones(64, device="cuda"), torch.ones(64, device="cuda")
    for call, what in ((lambda: gbce.grad_norm([a], 3.0), "norm_type"),
                       (lambda: gbce.grad_norm([a, b.cpu()]), "CUDA"),
                       (lambda: gbce.clip_grad_norm([a, b], 1.0, outs=[a]), "1 outs for 2"),
                       (lambda: gbce.clip_grad_norm([a], 1.0, outs=[a[:32]]), "outs must match"),
                       (lambda: gbce.clip_grad_norm([a], 1.0, outs=[a.bfloat16()]), "outs must match"),
                       (lambda: gbce.grad_norm([a], norm=torch.empty(2, device="cuda")), "one-element")):
        with pytest.raises(ValueError, match=what):
            call()
    with pytest.raises(TypeError, match="float64"):
        gbce.grad_norm([a.double()])
    for tensors, outs in (([a, a], None), ([a, b], [b, a]), ([a, b], [a, a]), ([a[:32], a[16:48]], None),
                          ([a[:32]], [a[16:48]])):
        with pytest.raises(gbce.GbceError) as e:
            gbce.clip_grad_norm(tensors, 1.0, outs=outs)
        assert e.value.code == gbce.ERR_OVERLAP
    with pytest.raises(gbce.GbceError):
        gbce.clip_grad_norm([a], 1.0, norm=a[3:4])
    for limit, eps in ((-1.0, 0.0), (math.nan, 0.0), (1.0, -1e-9), (1.0, math.nan)):
        with pytest.raises(gbce.GbceError):
            gbce.clip_grad_norm([a], limit, eps=eps)
    assert bool((a == 1).all() and (b == 1).all())
