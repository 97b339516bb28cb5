"""Tokens sorted by expert and back on the GPU, against plain forms (tolerances in permute_ref)."""
import pytest
import torch

import cross_entropy_loss_ce_gb300 as gbce
from permute_ref import PlanRef, combine_bwd_ref, combine_ref, near

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def choose(T, k, E, empty=0.0, seed=0, uneven=False):
    g = torch.Generator().manual_seed(seed + 7 * T + 3 * k + E)
    x = torch.rand(T, k, generator=g)
    ex = ((x * x if uneven else x) * E).long().clamp_max(E - 1)
    ex[torch.rand(T, k, generator=g) < empty / 2] = -1
    ex[torch.rand(T, generator=g) < empty / 2] = -1
    return ex.cuda()


def rows(n, H, dtype, seed, pad=0, shift=0):
    g = torch.Generator("cuda").manual_seed(seed)
    buf = torch.full((n, H + pad + shift), 7.0, device="cuda", dtype=dtype)
    buf[:, shift:shift + H] = torch.randn(n, H, device="cuda", generator=g).to(dtype)
    return buf[:, shift:shift + H]


def check_all(T, k, E, H, dtype, align=1, empty=0.2, wtype=torch.float32, pad=0, shift=0, seed=0):
    ex = choose(T, k, E, empty, seed)
    plan, ref = gbce.moe_sort(ex, E, align), PlanRef(ex, E, align)
    ref.check(plan)
    x = rows(T, H, dtype, 1, pad, shift)
    out = gbce.moe_dispatch(x, plan)
    want = torch.where((ref.source >= 0)[:, None], x[ref.source.long().clamp_min(0) // k], 0.0)
    assert torch.equal(out, want)
    y = rows(ref.rows, H, dtype, 2, pad, shift)
    y[ref.source < 0] = float("nan")  # a product may leave anything there
    w = torch.rand(T, k, device="cuda", generator=torch.Generator("cuda").manual_seed(3)).to(wtype)
    w[ref.position < 0] = float("nan")  # an empty slot's weight may be anything
    near(gbce.moe_combine(y, plan, w), *combine_ref(y, ref.position, w), "out")
    near(gbce.moe_combine(y, plan), *combine_ref(y, ref.position, None), "sum")
    g = rows(T, H, dtype, 4, pad, shift)
    (d_y, y_tol), (d_w, w_tol) = combine_bwd_ref(g, y, ref.position, w)
    got_y, got_w = gbce.moe_combine_bwd(g, y, plan, w)
    assert got_w.dtype == wtype
    near(got_y, d_y, y_tol, "d_y")
    near(got_w, d_w, w_tol, "d_weights")
    assert gbce.last_error() == gbce.OK


@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 8, 128), (3, 2, 5), (33, 4, 64), (256, 8, 8), (257, 8, 60),
                                   (1024, 8, 17), (1025, 8, 256), (8193, 1, 1), (4097, 2, 1024), (3000, 64, 9),
                                   (40000, 2, 512), (20000, 6, 1023), (4000, 2, 1024), (8192, 1, 1000)])
@pytest.mark.parametrize("align", [1, 128])
def test_plans(T, k, E, align):
    for empty in (0.0, 0.4):
        ex = choose(T, k, E, empty, uneven=True)
        PlanRef(ex, E, align).check(gbce.moe_sort(ex, E, align))
    assert gbce.last_error() == gbce.OK


def test_more_slots_than_the_sms_rank_at_once():
    # a CTA takes several rounds of 8192 slots from 8192 a SM on
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    for T, k, E in ((8192 * sms + 1, 1, 300), (8192 * sms // 2 + 5000, 4, 3)):
        ex = choose(T, k, E, 0.1, uneven=True)
        PlanRef(ex, E, 16).check(gbce.moe_sort(ex, E, 16))


@pytest.mark.parametrize("T,k", [(0, 2), (5, 2), (3000, 4)])
def test_no_slot_in_use(T, k):
    ex = torch.full((T, k), -1, device="cuda", dtype=torch.int64)
    plan, ref = gbce.moe_sort(ex, 6, 4), PlanRef(ex, 6, 4)
    ref.check(plan)
    x = rows(T, 24, torch.bfloat16, 1)
    assert not bool(gbce.moe_dispatch(x, plan).any())
    y = torch.full((ref.rows, 24), float("nan"), device="cuda", dtype=torch.bfloat16)
    w = torch.rand(T, k, device="cuda")
    out = gbce.moe_combine(y, plan, w)
    assert out.shape == (T, 24) and not bool(out.any())
    d_y, d_w = gbce.moe_combine_bwd(x, y, plan, w)
    assert d_y.shape == y.shape and not bool(d_y.any()) and d_w.shape == (T, k) and not bool(d_w.any())


@pytest.mark.parametrize("T,k", [(40, 3), (5000, 3)])
def test_bad_slots_count_as_empty(T, k):
    ex = choose(T, k, 12)
    ex[3, 1], ex[7, 0], ex[T - 1, 2] = 12, -2, 2 ** 40
    gbce.last_error()
    plan = gbce.moe_sort(ex, 12)
    assert gbce.last_error() == gbce.ERR_BAD_TARGET
    PlanRef(ex, 12).check(plan)


@pytest.mark.parametrize("T", [40, 5000])
def test_strided_choices(T):
    wide = torch.full((T, 9), 3, device="cuda", dtype=torch.int64)
    ex = choose(T, 4, 10, 0.2)
    wide[:, 2:6] = ex
    PlanRef(ex, 10).check(gbce.moe_sort(wide[:, 2:6], 10))
    one = torch.zeros(T, 3, device="cuda", dtype=torch.int64)[:, 1:2]
    PlanRef(one, 2).check(gbce.moe_sort(one, 2))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,k,E,H", [(1, 8, 32, 2048), (2, 1, 2, 1), (5, 2, 3, 7), (33, 4, 16, 4096), (300, 2, 8, 1001),
                                     (64, 3, 5, 250), (100, 5, 9, 8), (257, 8, 64, 136), (20, 11, 12, 520),
                                     (9, 64, 100, 72)])
def test_shapes(T, k, E, H, dtype):
    check_all(T, k, E, H, DT[dtype])


@pytest.mark.parametrize("T,k,H", [(2600, 2, 512), (2600, 4, 264), (2600, 8, 100), (2600, 7, 1003), (2433, 1, 33),
                                   (1300, 3, 2056), (1300, 2, 1030), (1300, 5, 1030), (1300, 1, 1001), (1300, 6, 2061)])
def test_many_tokens(T, k, H):
    # from 16 warps a SM on a lane takes several units
    check_all(T, k, 40, H, torch.bfloat16, align=16)


@pytest.mark.parametrize("T,k,H", [(401, 8, 2056), (401, 4, 2048), (403, 2, 4104), (309, 8, 8200), (307, 1, 8192),
                                   (150, 2, 1024), (151, 4, 2050), (149, 3, 3001), (7, 8, 16384)])
def test_tokens_that_several_warps_share(T, k, H):
    # 2, 4 and 8 warps a token, the last CTA not full; k 8 at H 2056 is one unit more than whole trips
    check_all(T, k, 12, H, torch.bfloat16, align=4)


@pytest.mark.parametrize("wtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [50, 2600])
def test_weights_of_the_rows_type(T, wtype):
    check_all(T, 3, 7, 96, torch.bfloat16, wtype=DT[wtype])


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("pad,shift", [(8, 0), (3, 0), (0, 1), (6, 2), (4, 4), (8, 8)])
def test_strides_and_alignment(dtype, pad, shift):
    check_all(70, 4, 6, 200, DT[dtype], align=8, pad=pad, shift=shift)


@pytest.mark.parametrize("H", [128, 77])
def test_given_outputs_and_their_neighbours(H):
    T, k, E = 60, 3, 7
    ex = choose(T, k, E, 0.3)
    plan, ref = gbce.moe_sort(ex, E, 4), PlanRef(ex, E, 4)
    x, y, w = rows(T, H, torch.float32, 1), rows(ref.rows, H, torch.float32, 2), torch.rand(T, k, device="cuda")
    for n, call in ((ref.rows, lambda o: gbce.moe_dispatch(x, plan, out=o)),
                    (T, lambda o: gbce.moe_combine(y, plan, w, out=o)),
                    (ref.rows, lambda o: gbce.moe_combine_bwd(x, y, plan, w, want_weights=False, d_y=o)[0])):
        buf = torch.full((n + 2, H + 9), 5.0, device="cuda")
        out = call(buf[1:n + 1, 4:4 + H])
        assert out.data_ptr() == buf[1:, 4:].data_ptr()
        assert torch.equal(out, call(torch.empty(n, H, device="cuda")))
        out.fill_(5.0)
        assert bool((buf == 5.0).all())
    d_w = torch.full((T, k + 2), 5.0, device="cuda")
    got = gbce.moe_combine_bwd(x, y, plan, w, want_y=False, d_weights=d_w[:, 1:k + 1])
    assert got[0] is None and torch.equal(got[1], gbce.moe_combine_bwd(x, y, plan, w)[1])
    assert bool((d_w[:, 0] == 5).all() and (d_w[:, -1] == 5).all())
    assert gbce.moe_combine_bwd(x, y, plan, w, want_y=False, want_weights=False) == (None, None)


def test_infinities_and_nan_stay_in_their_slots():
    T, k, E, H = 40, 2, 4, 64
    ex = choose(T, k, E)
    ex[5, 1] = -1
    plan = gbce.moe_sort(ex, E)
    p = plan.position.long()
    y, w, g = rows(T * k, H, torch.bfloat16, 1), torch.rand(T, k, device="cuda"), rows(T, H, torch.bfloat16, 2)
    y[p[3, 0], 7], w[9, 1], g[5, 0] = float("inf"), float("nan"), float("inf")
    out = gbce.moe_combine(y, plan, w)
    assert bool(torch.isinf(out[3, 7])) and bool(torch.isnan(out[9]).all())
    rest = torch.ones_like(out, dtype=torch.bool)
    rest[3, 7] = rest[9] = False
    assert bool(torch.isfinite(out[rest]).all())
    d_y, d_w = gbce.moe_combine_bwd(g, y, plan, w)
    assert bool(torch.isnan(d_y[p[9, 1]]).all()) and float(d_w[5, 1]) == 0.0
    assert bool(torch.isinf(d_w[5, 0])) and bool(torch.isfinite(d_y[p[9, 0]]).all())


def test_positions_of_another_hand_are_not_followed_outside():
    T, k, H = 6, 2, 32
    position = torch.tensor([[0, 11], [12, 1], [-5, 2], [3, 2 ** 31 - 1], [4, 5], [6, 7]], device="cuda",
                            dtype=torch.int32)
    source = torch.full((12,), -1, device="cuda", dtype=torch.int32)
    good = (position >= 0) & (position < 12)
    slots = torch.arange(12, device="cuda", dtype=torch.int32).view(T, k)
    source[position[good].long()] = slots[good]
    plan = gbce.MoePlan(position, source, torch.tensor([0, 12], device="cuda", dtype=torch.int32),
                        torch.tensor([9], device="cuda", dtype=torch.int32))
    x = rows(T, H, torch.float32, 1)
    want = torch.where((source >= 0)[:, None], x[source.long().clamp_min(0) // k], 0.0)
    assert torch.equal(gbce.moe_dispatch(x, plan), want)
    y, w = rows(12, H, torch.float32, 2), torch.rand(T, k, device="cuda")
    inside = torch.where(good, position, -1)
    near(gbce.moe_combine(y, plan, w), *combine_ref(y, inside, w), "out")
    (d_y, y_tol), (d_w, w_tol) = combine_bwd_ref(x, y, inside, w)
    got = gbce.moe_combine_bwd(x, y, plan, w)
    near(got[0], d_y, y_tol, "d_y")
    near(got[1], d_w, w_tol, "d_weights")


def test_rows_past_32_bit_offsets():
    # 66000 x 2 rows of 32768 values: 4.3e9 values
    T, k, E, H = 66000, 2, 3, 32768
    ex = choose(T, k, E)
    plan = gbce.moe_sort(ex, E)
    x = torch.empty(T, H, device="cuda", dtype=torch.bfloat16)
    x[:] = torch.arange(T, device="cuda")[:, None] % 251
    x += torch.arange(H, device="cuda") % 3  # below 256: exact
    out = gbce.moe_dispatch(x, plan)
    probe = torch.tensor([0, 1, 65535, 65536, 131071, 131072, T * k - 1], device="cuda")
    assert torch.equal(out[probe], x[plan.source[probe].long() // k])
    w = torch.full((T, k), 0.5, device="cuda")
    assert torch.equal(gbce.moe_combine(out, plan, w), x)
    d_y, d_w = gbce.moe_combine_bwd(x, out, plan, w)
    assert torch.equal(d_y[probe], 0.5 * out[probe])
    t = torch.tensor([0, 65999], device="cuda")
    dot = x[t].double().square().sum(1)
    near(d_w[t], dot[:, None].expand(2, k), (H / 32 + 17) * 2.0 ** -24 * dot[:, None].expand(2, k), "d_weights")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_autograd_forms(dtype):
    T, k, E, H = 300, 3, 8, 80
    ex = choose(T, k, E, 0.2)
    plan, ref = gbce.moe_sort(ex, E, 8), PlanRef(ex, E, 8)
    x = rows(T, H, DT[dtype], 1).reshape(10, 30, H).requires_grad_()
    g = rows(ref.rows, H, DT[dtype], 2)
    out = gbce.dispatch_tokens(x, plan)
    out.backward(g, retain_graph=True)
    near(x.grad.reshape(T, H), *combine_ref(g, ref.position, None), "d_x")
    first, x.grad = x.grad.clone(), None
    out.backward(g)
    assert torch.equal(first, x.grad)
    y = rows(ref.rows, H, DT[dtype], 3).requires_grad_()
    w = torch.rand(T, k, device="cuda").requires_grad_()
    (gbce.combine_tokens(y, plan, w).float().sum() * 2.0).backward()
    two = torch.full((T, H), 2.0, device="cuda", dtype=DT[dtype])
    (d_y, y_tol), (d_w, w_tol) = combine_bwd_ref(two, y.detach(), ref.position, w.detach())
    near(y.grad, d_y, y_tol, "d_y")
    near(w.grad, d_w, w_tol, "d_weights")
    y.grad = None
    gbce.combine_tokens(y, plan).sum().backward()  # an expanded incoming gradient
    assert torch.equal(y.grad, (ref.source >= 0)[:, None].to(y.dtype).expand(-1, H))
    y.grad = w.grad = None
    gbce.combine_tokens(y.detach(), plan, w).sum().backward()
    assert y.grad is None and w.grad is not None


def test_gradients_against_differences():
    # out is linear in y and in w: a difference of any size is exact but for roundings
    T, k, E, H = 90, 2, 5, 40
    ex = choose(T, k, E, 0.2)
    plan, ref = gbce.moe_sort(ex, E), PlanRef(ex, E)
    y, w, g = rows(T * k, H, torch.float32, 1), torch.rand(T, k, device="cuda"), rows(T, H, torch.float32, 2)
    vy, vw = rows(T * k, H, torch.float32, 3), torch.randn(T, k, device="cuda")
    vy[ref.source < 0] = 0.0
    d_y, d_w = (t.double() for t in gbce.moe_combine_bwd(g, y, plan, w))
    (_, y_tol), (_, w_tol) = combine_bwd_ref(g, y, ref.position, w)

    def loss(a, b):
        return (combine_ref(a, ref.position, b)[0] * g.double()).sum()
    tol = 1e-9 * float(g.double().abs().sum())
    assert abs(float((d_y * vy.double()).sum() - (loss(y.double() + vy.double(), w) - loss(y.double(), w)))) <= \
        float((y_tol * vy.abs()).sum()) + tol
    assert abs(float((d_w * vw.double()).sum() - (loss(y.double(), w.double() + vw.double()) - loss(y.double(), w)))) <= \
        float((w_tol * vw.abs()).sum()) + tol


def test_same_bits_on_two_streams_and_captured():
    cases = [(choose(T, 4, 30, 0.1), rows(T, 256, torch.bfloat16, T), torch.rand(T, 4, device="cuda"))
             for T in (50, 5000)]

    def run(ex, x, w, stream=None):
        plan = gbce.moe_sort(ex, 30, 16, stream=stream)
        xs = gbce.moe_dispatch(x, plan, stream=stream)
        out = gbce.moe_combine(xs, plan, w, stream=stream)
        return (plan.position, plan.source, xs, out) + gbce.moe_combine_bwd(x, xs, plan, w, stream=stream)
    want = [run(*c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [run(*c, stream=s) for _ in range(3) for s, c in zip(streams, cases)]
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(g, want[i % 2]))
    graphs = []
    for c in cases:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = run(*c)
        graphs.append((graph, out))
    for (ex, x, w), (graph, out) in zip(cases, graphs):
        ex.copy_(ex.flip(0).clone())
        x.neg_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, run(ex, x, w)))


def test_refusals_on_the_device():
    ex = choose(20, 2, 4)
    plan = gbce.moe_sort(ex, 4)
    x, y, w = rows(20, 16, torch.float32, 1), rows(40, 16, torch.float32, 2), torch.rand(20, 2, device="cuda")
    for call, what in ((lambda: gbce.moe_dispatch(x[:19], plan), "x has 19 rows"),
                       (lambda: gbce.moe_combine(y[:39], plan), "y has 39 rows"),
                       (lambda: gbce.moe_combine(y, plan, w[:, :1]), "columns"),
                       (lambda: gbce.moe_dispatch(x, plan, out=torch.empty(40, 15, device="cuda")), "16 columns"),
                       (lambda: gbce.moe_dispatch(y[:20], plan, out=y), "shares memory with x"),
                       (lambda: gbce.moe_combine(y, plan, w, out=y[:20]), "shares memory with y"),
                       (lambda: gbce.moe_combine_bwd(x, y, plan, w, d_y=y), "shares memory with y"),
                       (lambda: gbce.moe_combine_bwd(x, y, plan, w, d_weights=w), "shares memory with weights"),
                       (lambda: gbce.moe_combine_bwd(x[:, :8], y, plan, w), "as y"),
                       (lambda: gbce.moe_dispatch(x.t(), plan), "column stride"),
                       (lambda: gbce.moe_dispatch(x[:1].expand(20, 16), plan), "overlapping rows"),
                       (lambda: gbce.moe_sort(ex.t(), 4), "unit column stride"),
                       (lambda: gbce.moe_sort(ex.int(), 4), "int64"),
                       (lambda: gbce.MoePlan(plan.position.long(), plan.source, plan.offsets, plan.counts), "int32"),
                       (lambda: gbce.MoePlan(plan.position, plan.source, plan.counts, plan.counts), "one value more")):
        with pytest.raises(ValueError, match=what):
            call()
    with pytest.raises(TypeError, match="float32 or"):
        gbce.moe_combine(y, plan, w.half())
    with pytest.raises(TypeError):
        gbce.moe_dispatch(x.double(), plan)
    for E, align in ((0, 1), (1025, 1), (4, 0), (4, 1025)):
        with pytest.raises(gbce.GbceError):
            gbce.moe_sort(ex, E, align)
    torch.cuda.synchronize()


@pytest.mark.parametrize("T,k,E,align", [(1, 8, 128, 1), (700, 3, 5, 16), (9000, 1, 1000, 1), (20000, 8, 61, 128)])
def test_a_plan_in_memory_of_the_caller_and_its_neighbours(T, k, E, align):
    ex = choose(T, k, E, 0.2)
    ref = PlanRef(ex, E, align)
    sizes, gap = [T * k, ref.rows, E + 1, E], 9
    buf = torch.full((sum(sizes) + gap * 5,), 77, device="cuda", dtype=torch.int32)
    at, parts = gap, []
    for n in sizes:
        parts.append(buf[at:at + n])
        at += n + gap
    rc = gbce.load_library().moe_sort(ex.data_ptr(), k, *[p.data_ptr() for p in parts], T, E, k, align,
                                      torch.cuda.current_stream().cuda_stream)
    assert rc == gbce.OK
    ref.check(gbce.MoePlan(parts[0].view(T, k), *parts[1:], align))
    for p in parts:
        p.fill_(77)
    assert bool((buf == 77).all())
