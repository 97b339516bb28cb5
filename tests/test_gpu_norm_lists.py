"""Lists that clip_grad_norm takes and refuses, and what long ones cost (GPU)."""
import ctypes

import pytest
import torch

import cross_entropy_loss_ce_gb300 as gbce
from permute_ref import clip_ref, near, norm_ref

pytestmark = pytest.mark.gpu


def test_parameters_are_refused_where_their_gradients_are_meant():
    layer = torch.nn.Linear(64, 32, device="cuda")
    layer(torch.ones(4, 64, device="cuda")).sum().backward()
    before = [p.detach().clone() for p in layer.parameters()]
    for call in (lambda: gbce.clip_grad_norm(layer.parameters(), 1e-3),
                 lambda: gbce.clip_grad_norm(list(layer.parameters()), 1e-3),
                 lambda: gbce.clip_grad_norm(layer.weight, 1e-3),
                 lambda: gbce.clip_grad_norm([layer.weight.grad], 1e-3, outs=[layer.weight]),
                 lambda: gbce.clip_grad_norm([layer.weight.grad, layer.bias], 1e-3,
                                             outs=[layer.weight.grad, layer.bias])):
        with pytest.raises(ValueError, match="require gradients"):
            call()
    with torch.no_grad(), pytest.raises(ValueError, match="require gradients"):
        gbce.clip_grad_norm(layer.parameters(), 1e-3)
    assert all(torch.equal(p, b) for p, b in zip(layer.parameters(), before))
    # what is only read may be a parameter, and what a caller has detached is its own affair
    near(gbce.grad_norm(layer.parameters()), norm_ref(before, 2.0)[0].cuda(), 1e-5, "norm")
    gbce.clip_grad_norm(layer.parameters(), 1e-3, outs=[torch.empty_like(p) for p in layer.parameters()])
    assert all(torch.equal(p, b) for p, b in zip(layer.parameters(), before))
    gbce.clip_grad_norm([p.grad for p in layer.parameters()], 1e-3)
    near(gbce.grad_norm([p.grad for p in layer.parameters()]), torch.tensor(1e-3, dtype=torch.float64).cuda(), 1e-6, "norm")
    gbce.clip_grad_norm([p.detach() for p in layer.parameters()], 1e-3)
    assert not torch.equal(layer.weight, before[0])


def test_each_out_is_compared_with_its_own_tensor():
    g = torch.Generator("cuda").manual_seed(3)
    w = torch.randn(64, 32, device="cuda", generator=g).t()  # not contiguous
    v = torch.randn(6, 10, device="cuda", generator=g)
    one = torch.randn(1, 8, 5, device="cuda", generator=g).transpose(1, 2)
    outs = [torch.empty(64, 32, device="cuda").t(), torch.empty(60, device="cuda"),
            torch.empty(8, 5, device="cuda").t()[None]]  # the same order, another stride of the axis of one
    assert one.stride() != outs[2].stride()
    want, rel = norm_ref([w, v, one], 2.0)
    gbce.clip_grad_norm([w, v, one], 1.0, outs=outs)
    for t, o in zip((w, v, one), outs):
        ref, tol = clip_ref(t.reshape(-1), want, rel, 1.0, 1e-6)
        near(o.reshape(-1), ref, tol, "clipped")
    for bad in (torch.empty(32, 64, device="cuda"), torch.empty(2048, device="cuda"), torch.empty(64, 32, device="cuda")):
        with pytest.raises(ValueError, match="outs must match"):
            gbce.clip_grad_norm([w, v], 1.0, outs=[bad, outs[1]])


def test_long_lists_cost_what_their_tables_cost():
    # 2^18 tensors of a few values: 256 launches of each kernel.  Clipping launches twice what the norm does, and each
    # of its launches may add up what that one launch's kernels left, not what all did.
    n, lib = 2 ** 18, gbce.load_library()
    src = torch.randn(n, 4, device="cuda", generator=torch.Generator("cuda").manual_seed(7))
    dst, norm = torch.zeros_like(src), torch.zeros((), device="cuda")
    ins = (ctypes.c_uint64 * n)(*range(src.data_ptr(), src.data_ptr() + 16 * n, 16))
    outs = (ctypes.c_uint64 * n)(*range(dst.data_ptr(), dst.data_ptr() + 16 * n, 16))
    sizes, types = (ctypes.c_int64 * n)(*[4] * n), (ctypes.c_int * n)()
    s = torch.cuda.current_stream().cuda_stream

    def read():
        assert lib.grad_norm(ins, sizes, types, n, 0, norm.data_ptr(), s) == gbce.OK

    def clip():
        assert lib.clip_grad_norm(ins, outs, sizes, types, n, 0, 1.0, 1e-6, norm.data_ptr(), s) == gbce.OK

    def ms(call):
        times = []
        for _ in range(4):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            torch.cuda.synchronize()
            torch.cuda._sleep(100_000_000)  # the host is ahead: its time is not counted
            a.record()
            call()
            b.record()
            b.synchronize()
            times.append(a.elapsed_time(b))
        return min(times)
    of_read, of_clip = ms(read), ms(clip)
    want, rel = norm_ref([src], 2.0)
    near(norm, want.cuda(), (rel + 2.0 ** -24) * float(want), "norm")
    near(dst, *clip_ref(src, want, rel, 1.0, 1e-6), "clipped")
    assert of_clip < 6 * of_read, (of_read, of_clip)
