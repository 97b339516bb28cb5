"""Refusals of the expert permutation and of the norm of many tensors, on the host before anything is
launched (CPU)."""
import ctypes

import pytest
import torch

import cross_entropy_loss_ce_gb300 as gbce
from cross_entropy_loss_ce_gb300 import build as gbuild

FAKE = 0x10000  # never dereferenced
NULL, SIZE, DTYPE, ALIGN, REDUCTION, OVERLAP = 1, 2, 3, 4, 9, 11


@pytest.fixture(scope="module")
def lib():
    gbuild.build()
    return gbce.load_library()


def sort(**kw):
    a = dict(e=FAKE, es=2, p=FAKE, s=FAKE, o=FAKE, c=FAKE, T=4, E=8, k=2, align=1)
    a.update(kw)
    return [a[n] for n in ("e", "es", "p", "s", "o", "c", "T", "E", "k", "align")] + [None]


def dispatch(**kw):
    a = dict(x=FAKE, xs=64, p=FAKE, s=FAKE, out=FAKE, os=64, T=4, H=64, k=2, rows=8, dtype=1)
    a.update(kw)
    return [a[n] for n in ("x", "xs", "p", "s", "out", "os", "T", "H", "k", "rows", "dtype")] + [None]


def combine(**kw):
    a = dict(y=FAKE, ys=64, p=FAKE, w=FAKE, ws=2, wt=0, out=FAKE, os=64, T=4, H=64, k=2, rows=8, dtype=1)
    a.update(kw)
    return [a[n] for n in ("y", "ys", "p", "w", "ws", "wt", "out", "os", "T", "H", "k", "rows", "dtype")] + [None]


def combine_bwd(**kw):
    a = dict(g=FAKE, gs=64, y=FAKE, ys=64, p=FAKE, s=FAKE, w=FAKE, ws=2, wt=0, dy=FAKE, dys=64, dw=FAKE, dws=2,
             T=4, H=64, k=2, rows=8, dtype=1)
    a.update(kw)
    return [a[n] for n in ("g", "gs", "y", "ys", "p", "s", "w", "ws", "wt", "dy", "dys", "dw", "dws", "T", "H", "k",
                           "rows", "dtype")] + [None]


@pytest.mark.parametrize("kw,code", [
    (dict(e=None), NULL), (dict(p=None), NULL), (dict(s=None), NULL), (dict(o=None), NULL), (dict(c=None), NULL),
    (dict(es=1), SIZE), (dict(es=2 ** 46 + 1), SIZE), (dict(T=-1), SIZE), (dict(T=2 ** 27), SIZE), (dict(E=0), SIZE),
    (dict(E=1025), SIZE), (dict(k=0), SIZE), (dict(k=65, es=65), SIZE), (dict(align=0), SIZE), (dict(align=1025), SIZE),
    (dict(T=2 ** 26, k=32, es=32), SIZE), (dict(T=2 ** 27 - 1, k=16, es=16, E=1024, align=1024), SIZE),
    (dict(e=FAKE + 4), ALIGN), (dict(p=FAKE + 2), ALIGN), (dict(s=FAKE + 2), ALIGN), (dict(o=FAKE + 2), ALIGN),
    (dict(c=FAKE + 2), ALIGN)])
def test_moe_sort_refuses(lib, kw, code):
    assert lib.moe_sort(*sort(**kw)) == code


def test_plan_rows(lib):
    for T, E, k, align in ((0, 1, 1, 1), (0, 5, 2, 128), (1, 128, 8, 1), (1, 128, 8, 128), (100, 7, 3, 16), (7, 1024, 64, 1024),
                           (2 ** 27 - 1, 3, 15, 1)):
        n = T * k
        assert lib.moe_plan_rows(T, E, k, align) == -(-(n + min(E, n) * (align - 1)) // align) * align
    for T, E, k, align in ((-1, 1, 1, 1), (1, 0, 1, 1), (1, 1, 0, 1), (1, 1, 1, 0), (2 ** 26, 1, 32, 1),
                           (2 ** 27 - 1, 1024, 16, 1024), (1, 1, 1, 1025), (1, 1, 65, 1)):
        assert lib.moe_plan_rows(T, E, k, align) == -1


SHARED = [(dict(p=None), NULL), (dict(T=-1), SIZE), (dict(T=2 ** 27), SIZE), (dict(H=0), SIZE),
          (dict(H=2 ** 24 + 1, xs=2 ** 25, ys=2 ** 25, gs=2 ** 25, os=2 ** 25, dys=2 ** 25), SIZE), (dict(k=0), SIZE),
          (dict(k=65, ws=65, dws=65), SIZE), (dict(rows=-1), SIZE), (dict(rows=2 ** 31), SIZE), (dict(T=2 ** 26, k=32, ws=32, dws=32), SIZE),
          (dict(dtype=3), DTYPE), (dict(p=FAKE + 2), ALIGN)]


@pytest.mark.parametrize("kw,code", SHARED + [
    (dict(x=None), NULL), (dict(s=None), NULL), (dict(out=None), NULL), (dict(xs=63), SIZE), (dict(os=63), SIZE),
    (dict(x=FAKE + 1), ALIGN), (dict(out=FAKE + 1), ALIGN), (dict(s=FAKE + 2), ALIGN)])
def test_moe_dispatch_refuses(lib, kw, code):
    assert lib.moe_dispatch(*dispatch(**{n: v for n, v in kw.items() if n not in ("ys", "gs", "dys", "ws", "dws")})) == code


@pytest.mark.parametrize("kw,code", SHARED + [
    (dict(y=None), NULL), (dict(out=None), NULL), (dict(ys=63), SIZE), (dict(os=63), SIZE), (dict(ws=1), SIZE),
    (dict(wt=2), DTYPE), (dict(wt=3), DTYPE), (dict(y=FAKE + 1), ALIGN), (dict(out=FAKE + 1), ALIGN),
    (dict(w=FAKE + 2), ALIGN), (dict(w=FAKE + 1, wt=1), ALIGN)])
def test_moe_combine_refuses(lib, kw, code):
    assert lib.moe_combine(*combine(**{n: v for n, v in kw.items() if n not in ("xs", "gs", "dys", "dws")})) == code


@pytest.mark.parametrize("kw,code", SHARED + [
    (dict(g=None), NULL), (dict(y=None), NULL), (dict(s=None), NULL), (dict(w=None), NULL), (dict(dy=None, dw=None), NULL),
    (dict(gs=63), SIZE), (dict(ys=63), SIZE), (dict(dys=63), SIZE), (dict(ws=1), SIZE), (dict(dws=1), SIZE),
    (dict(wt=2), DTYPE), (dict(g=FAKE + 1), ALIGN), (dict(y=FAKE + 1), ALIGN), (dict(dy=FAKE + 1), ALIGN),
    (dict(w=FAKE + 2), ALIGN), (dict(dw=FAKE + 2), ALIGN), (dict(s=FAKE + 2), ALIGN)])
def test_moe_combine_bwd_refuses(lib, kw, code):
    assert lib.moe_combine_bwd(*combine_bwd(**{n: v for n, v in kw.items() if n not in ("xs", "os")})) == code


def norm_args(pointers, sizes, types, outs=None, n=None):
    n = len(pointers) if n is None else n
    m = max(len(pointers), 1)
    args = [(ctypes.c_void_p * m)(*pointers), (ctypes.c_int64 * m)(*sizes), (ctypes.c_int * m)(*types), n]
    if outs is not None:
        args.insert(1, (ctypes.c_void_p * m)(*outs))
    return args


GOOD = dict(pointers=[FAKE, FAKE + 4096], sizes=[64, 64], types=[0, 1])


@pytest.mark.parametrize("kw,kind,norm,code", [
    ({}, 3, FAKE, REDUCTION), ({}, -1, FAKE, REDUCTION), ({}, 0, None, NULL), ({}, 0, FAKE + 2, ALIGN),
    (dict(n=-1), 0, FAKE, SIZE), (dict(n=2 ** 20 + 1), 0, FAKE, SIZE), (dict(pointers=[FAKE, None]), 0, FAKE, NULL),
    (dict(sizes=[64, -1]), 0, FAKE, SIZE), (dict(sizes=[2 ** 40 + 1, 1]), 0, FAKE, SIZE),
    (dict(types=[0, 3]), 0, FAKE, DTYPE), (dict(pointers=[FAKE + 2, FAKE]), 0, FAKE, ALIGN),
    (dict(pointers=[FAKE, FAKE + 1]), 0, FAKE, ALIGN)])
def test_grad_norm_refuses(lib, kw, kind, norm, code):
    assert lib.grad_norm(*norm_args(**{**GOOD, **kw}), kind, norm, None) == code


@pytest.mark.parametrize("outs,limit,eps,norm,code", [
    ([FAKE, None], 1.0, 0.0, 2 * FAKE, NULL), ([FAKE + 2, FAKE], 1.0, 0.0, 2 * FAKE, ALIGN),
    ([FAKE, FAKE + 4096], -1.0, 0.0, 2 * FAKE, SIZE), ([FAKE, FAKE + 4096], float("nan"), 0.0, 2 * FAKE, SIZE),
    ([FAKE, FAKE + 4096], 1.0, -1.0, 2 * FAKE, SIZE),
    ([FAKE + 4096, FAKE], 1.0, 0.0, 2 * FAKE, OVERLAP),       # each over the other's tensor
    ([FAKE + 4, FAKE + 4096], 1.0, 0.0, 2 * FAKE, OVERLAP),   # its own tensor, not from its start
    ([FAKE, FAKE], 1.0, 0.0, 2 * FAKE, OVERLAP), ([8 * FAKE, 8 * FAKE + 254], 1.0, 0.0, 2 * FAKE, OVERLAP),
    ([FAKE, FAKE + 4096], 1.0, 0.0, FAKE + 252, OVERLAP), ([8 * FAKE, FAKE + 4096 + 126], 1.0, 0.0, 2 * FAKE, OVERLAP)])
def test_clip_grad_norm_refuses(lib, outs, limit, eps, norm, code):
    assert lib.clip_grad_norm(*norm_args(**GOOD, outs=outs), 0, limit, eps, norm, None) == code


def test_binding_refuses_before_any_launch():
    x, e = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int64)
    ints = [torch.zeros(s, dtype=torch.int32) for s in ((4, 2), 8, 5, 4)]
    for call in (lambda: gbce.moe_sort(e, 4), lambda: gbce.MoePlan(*ints), lambda: gbce.grad_norm([x]),
                 lambda: gbce.clip_grad_norm([x], 1.0)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(ValueError, match="int64"):
        gbce.moe_sort(e.int(), 4)
    with pytest.raises(ValueError, match="norm_type"):
        gbce.grad_norm([x], 0.5)


def test_dense_tensors_in_any_order_of_axes():
    x = torch.zeros(4, 6, 5)
    for t in (x, x.permute(2, 0, 1), x[:, :, :0], x[2:], x[:1].transpose(0, 2), torch.zeros(())):
        assert gbce._dense(t)
    for t in (x[:, :, :4], x[:, ::2], x[:1].expand(3, 6, 5), x[:, :3]):
        assert not gbce._dense(t)
