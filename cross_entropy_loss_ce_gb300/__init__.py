"""Fused hard-label cross-entropy and row softmax on GB300 (sm_103a), the
cross-entropy of hidden states through an output layer, a router's balance loss, its
tokens sorted by expert and back, and the norm of all gradients.

Thin ctypes binding of ``_lib/libgbce.so`` (C ABI in ``include/gbce.h``): it
checks tensor shapes, takes raw device pointers, row strides and the current
CUDA stream from torch, and calls the library.  Every step of the computation
runs in the library's own CUDA kernels; there is no CPU or PyTorch fallback.
Loading fails loudly when the library has not been built
(``python -m cross_entropy_loss_ce_gb300.build``).

A call with ``stream=`` works as one under ``torch.cuda.stream(stream)``: it reads its
operands, and makes its outputs, on that stream.  Operands from another stream have to
be ready on it, and kept until it is done; outputs are used elsewhere after it.
"""
import array
import ctypes
import os

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_lib", "libgbce.so")

GBCE_F32, GBCE_BF16, GBCE_F16 = 0, 1, 2
DTYPES = {torch.float32: GBCE_F32, torch.bfloat16: GBCE_BF16, torch.float16: GBCE_F16}
REDUCTIONS = {"mean": 0, "sum": 1, "none": 2}
NORMS = {2.0: 0, 1.0: 1, float("inf"): 2}

OK, ERR_NULL, ERR_SIZE, ERR_DTYPE, ERR_ALIGN, ERR_CUDA, ERR_BAD_TARGET, ERR_TIMEOUT, \
    ERR_NO_DEVICE, ERR_REDUCTION, ERR_BAD_TABLE, ERR_OVERLAP = range(12)
# bits a call ORs into its own status word (gbce_status_bit)
STATUS_TIMEOUT, STATUS_BAD_TABLE = 1, 2

_lib = None


class GbceError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: gbce status {code}: {status_string(code)}")


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libgbce.so once (raises if it is missing)."""
    global _lib
    if _lib is None:
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it with "
                               "`python -m cross_entropy_loss_ce_gb300.build`")
        lib = ctypes.CDLL(path)
        i64, p, ci = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int
        lib.ce_fwd_bwd.argtypes = [p, i64, p, p, i64, i64, i64, ci, p]
        lib.softmax_fwd.argtypes = [p, i64, p, i64, i64, i64, ci, p]
        lib.softmax_bwd.argtypes = [p, i64, p, i64, p, i64, i64, i64, ci, p]
        lib.softmax_fwd_ex.argtypes = [p, i64, p, i64, i64, i64, ci, p, p]
        lib.softmax_bwd_ex.argtypes = [p, i64, p, i64, p, i64, i64, i64, ci, p, p]
        lib.ce_fwd_bwd_ex.argtypes = [p, i64, p, p, p, p, i64, i64, i64, ci, ci, p]
        lib.scale_rows.argtypes = [p, i64, i64, i64, ci, p, ci, p]
        lib.gbce_plan.argtypes = [ci, i64, i64, ci, ci, ctypes.POINTER(ci)]
        lib.gbce_plan.restype = ctypes.c_char_p
        lib.gbce_last_error.argtypes = [p]
        lib.gbce_status_string.argtypes = [ci]
        lib.gbce_status_string.restype = ctypes.c_char_p
        lib.gbce_timing_enable.argtypes = [ci]
        lib.softmax_bwd_bsr.argtypes = [p, i64, p, i64, p, i64, p, i64, i64, i64, i64, i64, i64,
                                        ctypes.c_float, ci, p]
        lib.softmax_bwd_bsr_ex.argtypes = [p, i64, p, i64, p, i64, p, i64, i64, i64, i64, i64, i64,
                                           ctypes.c_float, ci, p, p]
        lib.gbce_bsr_plan.argtypes = [i64, i64, ci, ci, ctypes.POINTER(ci)]
        lib.gbce_bsr_plan.restype = ctypes.c_char_p
        lib.gbce_timing_read.argtypes = [ctypes.POINTER(ctypes.c_double),
                                         ctypes.POINTER(ctypes.c_int64)]
        lib.linear_ce_fwd.argtypes = [p, i64, p, i64, p, p, p, p, i64, i64, i64, i64, ci, ci, p]
        lib.linear_ce_bwd.argtypes = [p, i64, p, i64, p, p, p, p, i64, p, i64, i64, i64, i64, i64,
                                      ci, ci, p]
        lib.linear_ce_bwd_ex.argtypes = [p, i64, p, i64, p, p, p, p, p, i64, p, i64, i64, i64, i64, i64,
                                         ci, ci, p]
        lib.linear_greedy.argtypes = [p, i64, p, i64, p, p, i64, i64, i64, ci, p]
        lib.moe_balance.argtypes = [p, i64, p, i64, p, p, p, i64, p, i64, i64, i64, ctypes.c_float,
                                    ctypes.c_float, ci, p]
        lib.moe_plan_rows.argtypes = [i64, i64, i64, i64]
        lib.moe_plan_rows.restype = i64
        lib.moe_sort.argtypes = [p, i64, p, p, p, p, i64, i64, i64, i64, p]
        lib.moe_dispatch.argtypes = [p, i64, p, p, p, i64, i64, i64, i64, i64, ci, p]
        lib.moe_combine.argtypes = [p, i64, p, p, i64, ci, p, i64, i64, i64, i64, i64, ci, p]
        lib.moe_combine_bwd.argtypes = [p, i64, p, i64, p, p, p, i64, ci, p, i64, p, i64, i64, i64, i64,
                                        i64, ci, p]
        lib.grad_norm.argtypes = [p, p, p, i64, ci, p, p]
        lib.clip_grad_norm.argtypes = [p, p, p, p, i64, ci, ctypes.c_double, ctypes.c_double, p, p]
        for f in ("ce_fwd_bwd", "softmax_fwd", "softmax_bwd", "gbce_last_error",
                  "gbce_timing_enable", "gbce_timing_read", "ce_fwd_bwd_ex", "scale_rows",
                  "softmax_bwd_bsr", "linear_ce_fwd", "linear_ce_bwd", "linear_ce_bwd_ex",
                  "linear_greedy", "moe_balance", "moe_sort", "moe_dispatch", "moe_combine",
                  "moe_combine_bwd", "grad_norm", "clip_grad_norm"):
            getattr(lib, f).restype = ci
        _lib = lib
    return _lib


def status_string(code: int) -> str:
    return load_library().gbce_status_string(code).decode()


def _call_device(*named):
    """The one CUDA device that every tensor of a call lives on.

    ``named`` holds (name, tensor) pairs; None tensors are skipped.  Raises
    ValueError, before anything is launched, when a tensor is on the host or
    on another device than the first one: the library works on the current
    device, so a pointer of another GPU would be handed to the wrong one.
    """
    dev = None
    for name, t in named:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError(f"{name} is on {t.device}, the call's other tensors on {dev}")
    return dev


class _OnDevice:
    """Makes `device` current for a library call; a no-op (no context-manager
    round trip through torch) when it already is, the common case."""
    __slots__ = ("index", "prev")

    def __init__(self, device):
        self.index = device.index if device.index is not None else torch.cuda.current_device()
        self.prev = None

    def __enter__(self):
        cur = torch.cuda.current_device()
        if cur != self.index:
            self.prev = cur
            torch.cuda.set_device(self.index)
        return self

    def __exit__(self, *exc):
        if self.prev is not None:
            torch.cuda.set_device(self.prev)
        return False


def _stream_handle(stream, device) -> ctypes.c_void_p:
    """The stream of a call on ``device``: the given one (which must belong to
    that device) or the device's current torch stream."""
    if stream is None:  # the handle itself: no Stream object for it
        return ctypes.c_void_p(torch._C._cuda_getCurrentRawStream(device.index))
    if stream.device != device:
        raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
    return ctypes.c_void_p(stream.cuda_stream)


def _matrix(t: torch.Tensor, name: str):
    """(pointer, row stride in elements, rows, cols) of a 2-D CUDA fp32/bf16 tensor."""
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D, got shape {tuple(t.shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype not in DTYPES:
        raise TypeError(f"{name} must be float32, bfloat16 or float16, not {t.dtype}")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} needs unit column stride")
    stride = t.stride(0) if t.shape[0] > 1 else t.shape[1]
    return t.data_ptr(), max(stride, t.shape[1]), t.shape[0], t.shape[1]


def _check(rc: int, where: str):
    if rc != OK:
        raise GbceError(rc, where)


def ce_fwd_bwd(logits: torch.Tensor, targets: torch.Tensor, ignore_index: int = -100,
               loss: torch.Tensor = None, stream=None) -> torch.Tensor:
    """Mean cross-entropy of ``logits`` [M, V] against int64 ``targets`` [M].

    ``logits`` is overwritten in place with d(loss)/d(logits).  Returns a
    0-dim float32 CUDA tensor (``loss`` when given); nothing is synchronised.
    """
    lp, stride, M, V = _matrix(logits, "logits")
    if targets.dtype != torch.int64 or targets.dim() != 1 or targets.shape[0] != M:
        raise ValueError("targets must be int64 of shape [M]")
    if M and (not targets.is_cuda or not targets.is_contiguous()):
        raise ValueError("targets must be a contiguous CUDA tensor")
    if loss is None:
        loss = _empty((), torch.float32, logits.device, stream)
    elif loss.dtype != torch.float32 or loss.numel() != 1 or not loss.is_cuda:
        raise ValueError("loss must be a one-element float32 CUDA tensor")
    dev = _call_device(("logits", logits), ("targets", targets if M else None), ("loss", loss))
    with _OnDevice(dev):
        rc = load_library().ce_fwd_bwd(lp, stride, targets.data_ptr(), loss.data_ptr(), M, V,
                                       int(ignore_index), DTYPES[logits.dtype],
                                       _stream_handle(stream, dev))
    _check(rc, "ce_fwd_bwd")
    return loss


def _empty(shape, dtype, device, stream):
    """An output that a call makes for itself.  Like all that it allocates or fills, it belongs
    to the call's stream: made on the current stream, it might be a block that work queued there
    has yet to leave.  The current stream is noted as its user, so its memory is not given to a
    later call of the stream while work queued here by the time it is dropped still reads it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        out = torch.empty(shape, dtype=dtype, device=device)
    if out.is_cuda:
        out.record_stream(torch.cuda.current_stream(out.device))
    return out


def _device_floats(v, n: int, device, name: str, stream):
    """A float32 CUDA tensor of n values on `device` from a tensor or a number (filled on the
    call's stream)."""
    if not torch.is_tensor(v):
        with torch.cuda.stream(stream):  # None: the current one
            v = torch.full((n,), float(v), dtype=torch.float32, device=device)
    if v.dtype != torch.float32 or not v.is_cuda or v.numel() != n or not v.is_contiguous():
        raise ValueError(f"{name} must be {n} contiguous float32 CUDA value(s)")
    return v


def ce_fwd_bwd_ex(logits: torch.Tensor, targets: torch.Tensor, ignore_index: int = -100,
                  reduction: str = "mean", grad_scale=None, want_row_loss: bool = False,
                  loss: torch.Tensor = None, row_loss: torch.Tensor = None, stream=None):
    """Cross-entropy with a reduction ('mean', 'sum', 'none'), optional per-row
    losses, and grad_scale (None, a number or a float32 CUDA tensor: one value,
    or one per row for 'none') folded into the in-place gradient.

    Returns (loss, row_loss): loss is a 0-dim float32 CUDA tensor (None for
    'none'); row_loss is [M] float32 when requested or for 'none', else None.
    """
    lp, stride, M, V = _matrix(logits, "logits")
    if reduction not in REDUCTIONS:
        raise ValueError(f"reduction must be one of {sorted(REDUCTIONS)}")
    if targets.dtype != torch.int64 or targets.dim() != 1 or targets.shape[0] != M:
        raise ValueError("targets must be int64 of shape [M]")
    if M and (not targets.is_cuda or not targets.is_contiguous()):
        raise ValueError("targets must be a contiguous CUDA tensor")
    dev = logits.device
    if reduction != "none" and loss is None:
        loss = _empty((), torch.float32, dev, stream)
    if (want_row_loss or reduction == "none") and row_loss is None:
        row_loss = _empty((M,), torch.float32, dev, stream)
    gs = None
    if grad_scale is not None:
        gs = _device_floats(grad_scale, M if reduction == "none" else 1, dev, "grad_scale", stream)
    dev = _call_device(("logits", logits), ("targets", targets if M else None), ("loss", loss),
                       ("row_loss", row_loss), ("grad_scale", gs))
    with _OnDevice(dev):
        rc = load_library().ce_fwd_bwd_ex(
            lp, stride, targets.data_ptr(), None if loss is None else loss.data_ptr(),
            None if row_loss is None else row_loss.data_ptr(),
            None if gs is None else gs.data_ptr(), M, V, int(ignore_index),
            DTYPES[logits.dtype], REDUCTIONS[reduction], _stream_handle(stream, dev))
    _check(rc, "ce_fwd_bwd_ex")
    return (None if reduction == "none" else loss), row_loss


def scale_rows(x: torch.Tensor, scale, stream=None) -> torch.Tensor:
    """x *= scale in place; scale is a number, a one-element float32 CUDA tensor,
    or one value per row ([M]).  A single scale of 1 costs only the launch."""
    xp, stride, M, N = _matrix(x, "x")
    per_row = torch.is_tensor(scale) and scale.numel() == M and M != 1
    sc = _device_floats(scale, M if per_row else 1, x.device, "scale", stream)
    dev = _call_device(("x", x), ("scale", sc))
    with _OnDevice(dev):
        rc = load_library().scale_rows(xp, stride, M, N, DTYPES[x.dtype], sc.data_ptr(),
                                       1 if per_row else 0, _stream_handle(stream, dev))
    _check(rc, "scale_rows")
    return x


class FusedCrossEntropy(torch.autograd.Function):
    """Autograd form of the fused call (the behaviour of Liger-Kernel's
    LigerCrossEntropyFunction): the forward computes the loss and writes the
    gradient into the logits' storage, which it saves; the backward scales that
    gradient in place by grad_output (a device-side no-op when it is 1, so no
    host synchronisation) and returns it.  The logits' values are consumed:
    read them before this call, and call backward once.
    """

    @staticmethod
    def forward(ctx, logits, targets, ignore_index=-100, reduction="mean"):
        buf = logits.detach()
        loss, row_loss = ce_fwd_bwd_ex(buf, targets, ignore_index, reduction)
        ctx.save_for_backward(buf)
        ctx.reduction = reduction
        return row_loss if reduction == "none" else loss

    @staticmethod
    def backward(ctx, grad_output):
        (grad,) = ctx.saved_tensors
        scale_rows(grad, grad_output.detach().to(torch.float32).contiguous().reshape(-1))
        return grad, None, None, None


def cross_entropy(logits: torch.Tensor, targets: torch.Tensor, ignore_index: int = -100,
                  reduction: str = "mean", inplace: bool = True) -> torch.Tensor:
    """Hard-label cross-entropy of [M, V] logits, differentiable.  With
    inplace=True the logits' storage is reused for the gradient (no extra
    M x V buffer); with inplace=False the logits are copied first."""
    if not inplace:
        logits = logits.clone(memory_format=torch.contiguous_format)
    return FusedCrossEntropy.apply(logits, targets, ignore_index, reduction)


class CrossEntropyLoss(torch.nn.Module):
    """nn.Module form of cross_entropy (hard labels, ignore_index, reduction)."""

    def __init__(self, ignore_index: int = -100, reduction: str = "mean", inplace: bool = True):
        super().__init__()
        if reduction not in REDUCTIONS:
            raise ValueError(f"reduction must be one of {sorted(REDUCTIONS)}")
        self.ignore_index, self.reduction, self.inplace = ignore_index, reduction, inplace

    def forward(self, logits, targets):
        return cross_entropy(logits, targets, self.ignore_index, self.reduction, self.inplace)


def _status_word(status, name="status"):
    """Device address of a per-call status word: a CUDA int32 tensor of one element."""
    if status is None:
        return None
    if not status.is_cuda or status.dtype != torch.int32 or status.numel() != 1:
        raise ValueError(f"{name} must be a one-element int32 CUDA tensor")
    return status.data_ptr()


def softmax_fwd(x: torch.Tensor, y: torch.Tensor = None, stream=None) -> torch.Tensor:
    """Row softmax of ``x`` [M, N] into ``y`` (allocated when None; may be ``x``)."""
    return softmax_fwd_ex(x, y, None, stream)


def softmax_fwd_ex(x: torch.Tensor, y: torch.Tensor = None, status: torch.Tensor = None,
                   stream=None) -> torch.Tensor:
    """softmax_fwd with a status word of the call's own: ``status`` (a one-element
    int32 CUDA tensor the caller cleared) gets STATUS_TIMEOUT when one of the
    call's bounded waits gave up."""
    if y is None:
        y = _empty(x.shape, x.dtype, x.device, stream)
    xp, xs, M, N = _matrix(x, "x")
    yp, ys, My, Ny = _matrix(y, "y")
    if (My, Ny) != (M, N) or y.dtype != x.dtype:
        raise ValueError("y must match x in shape and dtype")
    sp = _status_word(status)
    dev = _call_device(("x", x), ("y", y), ("status", status))
    with _OnDevice(dev):
        rc = load_library().softmax_fwd_ex(xp, xs, yp, ys, M, N, DTYPES[x.dtype], sp,
                                           _stream_handle(stream, dev))
    _check(rc, "softmax_fwd")
    return y


def softmax_bwd(y: torch.Tensor, dy: torch.Tensor, dx: torch.Tensor = None,
                stream=None) -> torch.Tensor:
    """dx = y * (dy - sum(y * dy, row)) for [M, N] operands (dx may be ``dy``)."""
    return softmax_bwd_ex(y, dy, dx, None, stream)


def softmax_bwd_ex(y: torch.Tensor, dy: torch.Tensor, dx: torch.Tensor = None,
                   status: torch.Tensor = None, stream=None) -> torch.Tensor:
    """softmax_bwd with a status word of the call's own (as softmax_fwd_ex)."""
    if dx is None:
        dx = _empty(dy.shape, dy.dtype, dy.device, stream)
    yp, ys, M, N = _matrix(y, "y")
    dp, ds, Md, Nd = _matrix(dy, "dy")
    xp, xs, Mx, Nx = _matrix(dx, "dx")
    if (Md, Nd) != (M, N) or (Mx, Nx) != (M, N) or not (y.dtype == dy.dtype == dx.dtype):
        raise ValueError("y, dy and dx must share shape and dtype")
    sp = _status_word(status)
    dev = _call_device(("y", y), ("dy", dy), ("dx", dx), ("status", status))
    with _OnDevice(dev):
        rc = load_library().softmax_bwd_ex(yp, ys, dp, ds, xp, xs, M, N, DTYPES[y.dtype], sp,
                                           _stream_handle(stream, dev))
    _check(rc, "softmax_bwd")
    return dx


def softmax_bwd_bsr(y: torch.Tensor, dy: torch.Tensor, lut: torch.Tensor, n_block_rows: int,
                    nblocks: int, block: int, sizemax: int, scale: float = 1.0,
                    dx: torch.Tensor = None, stream=None) -> torch.Tensor:
    """Block-sparse softmax backward, dx = y * (dy - sum(y * dy)) * scale per row.

    ``y``, ``dy`` and ``dx`` are [Z, zstride] CUDA tensors (unit inner stride)
    whose first nblocks * block^2 elements per batch item hold the blocks;
    ``lut`` is the int32 look-up table (a contiguous CUDA tensor).  ``dx``
    defaults to ``dy`` (in place, as the page's kernel stores); only the
    positions the table names are written.
    """
    return softmax_bwd_bsr_ex(y, dy, lut, n_block_rows, nblocks, block, sizemax, scale, dx,
                              None, stream)


def softmax_bwd_bsr_ex(y: torch.Tensor, dy: torch.Tensor, lut: torch.Tensor, n_block_rows: int,
                       nblocks: int, block: int, sizemax: int, scale: float = 1.0,
                       dx: torch.Tensor = None, status: torch.Tensor = None,
                       stream=None) -> torch.Tensor:
    """softmax_bwd_bsr with a status word of the call's own: ``status`` (a
    one-element int32 CUDA tensor the caller cleared) gets STATUS_BAD_TABLE when
    the call finds a malformed table entry."""
    if dx is None:
        dx = dy
    yp, ys, Z, Ly = _matrix(y, "y")
    dp, ds, Zd, Ld = _matrix(dy, "dy")
    xp, xs, Zx, Lx = _matrix(dx, "dx")
    if Zd != Z or Zx != Z or not (y.dtype == dy.dtype == dx.dtype):
        raise ValueError("y, dy and dx must share the batch size and dtype")
    if min(Ly, Ld, Lx) < nblocks * block * block:
        raise ValueError("y, dy and dx must hold nblocks * block^2 elements per batch item")
    if lut.dtype != torch.int32 or lut.dim() != 1 or not lut.is_cuda or not lut.is_contiguous():
        raise ValueError("lut must be a contiguous 1-D int32 CUDA tensor")
    sp = _status_word(status)
    dev = _call_device(("y", y), ("dy", dy), ("dx", dx), ("lut", lut), ("status", status))
    with _OnDevice(dev):
        rc = load_library().softmax_bwd_bsr_ex(yp, ys, dp, ds, xp, xs, lut.data_ptr(), lut.numel(),
                                               n_block_rows, nblocks, block, sizemax, Z,
                                               float(scale), DTYPES[y.dtype], sp,
                                               _stream_handle(stream, dev))
    _check(rc, "softmax_bwd_bsr")
    return dx


def bsr_plan(block: int, sizemax: int, dtype: torch.dtype, aligned: bool = True):
    """(kernel name, rows per slab of a block-row of sizemax blocks) that
    softmax_bwd_bsr uses for this block size, longest block-row and dtype."""
    r = ctypes.c_int(0)
    name = load_library().gbce_bsr_plan(block, sizemax, DTYPES[dtype], 1 if aligned else 0,
                                        ctypes.byref(r))
    if name is None:
        raise ValueError("invalid block-sparse plan query")
    return name.decode(), r.value


def plan(op: str, M: int, cols: int, dtype: torch.dtype, same_phase: bool = True):
    """(row-kernel family, CTAs per row) the library picks for M rows of `cols`
    elements on the current device; op is 'ce', 'softmax_fwd' or 'softmax_bwd'.
    M matters only for batches of at most one row per SM (gbce_plan)."""
    c = ctypes.c_int(0)
    name = load_library().gbce_plan({"ce": 0, "softmax_fwd": 1, "softmax_bwd": 2}[op], M, cols,
                                    DTYPES[dtype], 1 if same_phase else 0, ctypes.byref(c))
    if name is None:
        raise ValueError("invalid plan query")
    return name.decode(), c.value


def last_error(stream=None) -> int:
    """Synchronise the stream and read-and-clear the error flags of its device
    (the current device when no stream is given)."""
    dev = stream.device if stream is not None else torch.device("cuda", torch.cuda.current_device())
    with _OnDevice(dev):
        return load_library().gbce_last_error(_stream_handle(stream, dev))


def timing_enable(on: bool = True):
    _check(load_library().gbce_timing_enable(1 if on else 0), "gbce_timing_enable")


def timing_read():
    """(summed row-kernel milliseconds, bracketed launches) since the last read."""
    ms, n = ctypes.c_double(), ctypes.c_int64()
    _check(load_library().gbce_timing_read(ctypes.byref(ms), ctypes.byref(n)), "gbce_timing_read")
    return ms.value, n.value


def ce_fwd_bwd_host(logits_host: torch.Tensor, targets_host: torch.Tensor,
                    ignore_index: int = -100, grad: torch.Tensor = None,
                    loss_host: torch.Tensor = None, stream=None):
    """ce_fwd_bwd from host memory: (grad, loss_host).

    ``logits_host`` [M, V] and ``targets_host`` [M] (int64) are CPU tensors
    (pinned memory makes the copies asynchronous).  ``grad`` is a CUDA tensor of
    the logits' shape and dtype (allocated when not given) that receives the
    logits and then, in place, the gradient; ``loss_host`` is a one-element
    CPU float32 tensor (pinned when allocated here) that holds the mean loss
    once the stream has reached the end of the call.
    """
    if logits_host.is_cuda or targets_host.is_cuda:
        raise ValueError("logits_host and targets_host must be CPU tensors")
    if logits_host.dim() != 2 or (logits_host.shape[1] > 1 and logits_host.stride(1) != 1):
        raise ValueError("logits_host must be 2-D with unit column stride")
    if logits_host.dtype not in DTYPES:
        raise TypeError(f"logits_host must be float32, bfloat16 or float16, not {logits_host.dtype}")
    M, V = logits_host.shape
    if targets_host.dtype != torch.int64 or targets_host.shape != (M,) or \
            not targets_host.is_contiguous():
        raise ValueError("targets_host must be a contiguous int64 tensor of shape [M]")
    hs = logits_host.stride(0) if M > 1 else V
    if grad is None:
        grad = _empty((M, V), logits_host.dtype, "cuda", stream)
    gp, gs, Mg, Vg = _matrix(grad, "grad")
    if (Mg, Vg) != (M, V) or grad.dtype != logits_host.dtype:
        raise ValueError("grad must match the logits' shape and dtype")
    if loss_host is None:
        loss_host = torch.empty((), dtype=torch.float32).pin_memory()
    elif loss_host.dtype != torch.float32 or loss_host.numel() != 1 or loss_host.is_cuda:
        raise ValueError("loss_host must be a one-element float32 CPU tensor")
    lib = load_library()
    fn = lib.ce_fwd_bwd_host
    fn.argtypes = [ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p,
                   ctypes.c_int64, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64,
                   ctypes.c_int64, ctypes.c_int, ctypes.c_void_p]
    fn.restype = ctypes.c_int
    dev = _call_device(("grad", grad))
    with _OnDevice(dev):
        rc = fn(logits_host.data_ptr(), max(hs, V), targets_host.data_ptr(), gp, gs,
                loss_host.data_ptr(), M, V, int(ignore_index), DTYPES[logits_host.dtype],
                _stream_handle(stream, dev))
    _check(rc, "ce_fwd_bwd_host")
    return grad, loss_host


def ce_fwd_bwd_noalloc(logits: torch.Tensor, targets: torch.Tensor, ignore_index: int = -100,
                       loss: torch.Tensor = None, stream=None) -> torch.Tensor:
    """ce_fwd_bwd for callers that cannot let the library allocate device memory.

    Same results; the temporary storage is a fixed static device array inside
    the library (M <= 65536 rows), shared by every call on the device, so
    calls that overlap on the GPU must be serialised by the caller.  ``loss``
    is allocated here by torch when not given.
    """
    lp, stride, M, V = _matrix(logits, "logits")
    if targets.dtype != torch.int64 or targets.dim() != 1 or targets.shape[0] != M:
        raise ValueError("targets must be int64 of shape [M]")
    if M and (not targets.is_cuda or not targets.is_contiguous()):
        raise ValueError("targets must be a contiguous CUDA tensor")
    if loss is None:
        loss = _empty((), torch.float32, logits.device, stream)
    elif loss.dtype != torch.float32 or loss.numel() != 1 or not loss.is_cuda:
        raise ValueError("loss must be a one-element float32 CUDA tensor")
    dev = _call_device(("logits", logits), ("targets", targets if M else None), ("loss", loss))
    fn = load_library().ce_fwd_bwd_noalloc
    fn.argtypes = [ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p,
                   ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_int, ctypes.c_void_p]
    fn.restype = ctypes.c_int
    with _OnDevice(dev):
        rc = fn(lp, stride, targets.data_ptr(), loss.data_ptr(), M, V, int(ignore_index),
                DTYPES[logits.dtype], _stream_handle(stream, dev))
    _check(rc, "ce_fwd_bwd_noalloc")
    return loss


# ---------------------------------------------------------------------------
# the output layer: losses and tokens from hidden states, the logits not stored


def _rows(t: torch.Tensor, name: str):
    """_matrix for operands whose rows must not share memory (no expanded rows)."""
    if t.dim() == 2 and t.is_cuda and t.dtype in DTYPES:
        (rows, cols), (step, unit) = t.shape, t.stride()
        if unit == 1 and step >= cols:
            return t.data_ptr(), step, rows, cols
        if rows > 1 and step < cols and (unit == 1 or cols == 1):
            raise ValueError(f"{name} has overlapping rows (stride {step} for {cols} columns)")
    return _matrix(t, name)


def _head(hidden, weight):
    hp, hs, M, K = _rows(hidden, "hidden")
    wp, ws, V, Kw = _rows(weight, "weight")
    if Kw != K:
        raise ValueError(f"hidden has {K} columns, weight {Kw}")
    if hidden.dtype != weight.dtype:
        raise TypeError(f"hidden is {hidden.dtype}, weight {weight.dtype}")
    return hp, hs, wp, ws, M, K, V


def _class_ids(targets, M):
    if targets.dtype != torch.int64 or targets.dim() != 1 or targets.shape[0] != M:
        raise ValueError("targets must be int64 of shape [M]")
    if M and (not targets.is_cuda or not targets.is_contiguous()):
        raise ValueError("targets must be a contiguous CUDA tensor")
    return targets if M else None


def _row_values(t, M, name):
    if t.dtype != torch.float32 or t.shape != (M,) or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous float32 of shape [M]")
    return t


def _apart(name, out, *inputs):
    """Raises ValueError when the matrix ``out`` shares memory with an input.  (Columns of one
    buffer share none: rows of one stride, side by side.)"""
    def span(t):
        last = sum((n - 1) * s for n, s in zip(t.shape, t.stride())) if t.numel() else -1
        return t.data_ptr(), t.data_ptr() + (last + 1) * t.element_size()
    lo, hi = span(out)
    for other, t in inputs:
        if t is None:
            continue
        a, b = span(t)
        if not (lo < b and a < hi):
            continue
        if out.dim() == t.dim() == 2 and out.shape[0] > 1 and t.shape[0] > 1:
            step = out.stride(0) * out.element_size()
            beside = (a - lo) % step if step else 0
            if step == t.stride(0) * t.element_size() and \
                    beside >= out.shape[1] * out.element_size() and \
                    beside + t.shape[1] * t.element_size() <= step:
                continue
        raise ValueError(f"{name} shares memory with {other}")


def _ptr(t):
    return None if t is None else t.data_ptr()


def linear_ce_fwd(hidden: torch.Tensor, weight: torch.Tensor, targets: torch.Tensor,
                  ignore_index: int = -100, reduction: str = "mean", loss: torch.Tensor = None,
                  row_loss: torch.Tensor = None, lse: torch.Tensor = None, stream=None):
    """Cross-entropy of ``hidden`` [M, K] through the output layer ``weight``
    [V, K] (both bfloat16 or both float16) against int64 ``targets`` [M]; the
    [M, V] logits are never stored.

    Returns (loss, row_loss, lse): a 0-dim float32 CUDA tensor (None for the
    reduction 'none'), the [M] row losses and the [M] log-sum-exps (0 for ignored
    rows) that linear_ce_bwd takes.
    """
    hp, hs, wp, ws, M, K, V = _head(hidden, weight)
    if reduction not in REDUCTIONS:
        raise ValueError(f"reduction must be one of {sorted(REDUCTIONS)}")
    ids = _class_ids(targets, M)
    dev = hidden.device
    if reduction == "none":
        loss = None
    elif loss is None:
        loss = _empty((), torch.float32, dev, stream)
    elif loss.dtype != torch.float32 or loss.numel() != 1:
        raise ValueError("loss must be a one-element float32 CUDA tensor")
    row_loss = _empty((M,), torch.float32, dev, stream) if row_loss is None else \
        _row_values(row_loss, M, "row_loss")
    lse = _empty((M,), torch.float32, dev, stream) if lse is None else \
        _row_values(lse, M, "lse")
    dev = _call_device(("hidden", hidden), ("weight", weight), ("targets", ids), ("loss", loss),
                       ("row_loss", row_loss), ("lse", lse))
    with _OnDevice(dev):
        rc = load_library().linear_ce_fwd(
            hp, hs, wp, ws, targets.data_ptr(), _ptr(loss), row_loss.data_ptr(), lse.data_ptr(), M, K,
            V, int(ignore_index), DTYPES[hidden.dtype], REDUCTIONS[reduction],
            _stream_handle(stream, dev))
    _check(rc, "linear_ce_fwd")
    return loss, row_loss, lse


def linear_ce_bwd(hidden: torch.Tensor, weight: torch.Tensor, targets: torch.Tensor,
                  lse: torch.Tensor, grad_scale=None, ignore_index: int = -100,
                  reduction: str = "mean", want_hidden: bool = True, want_weight: bool = True,
                  d_hidden: torch.Tensor = None, d_weight: torch.Tensor = None, stream=None,
                  row_loss: torch.Tensor = None):
    """(d_hidden, d_weight) of linear_ce_fwd's loss, in the operands' type.

    ``lse`` and ``row_loss`` are what the forward returned; without the row losses
    the gradients of nearly certain rows lose their precision (a loss of 1e-4 about 1%
    of it, one of 1e-6 all: it is less than a step of lse).  ``grad_scale`` the incoming gradient
    (None, a number or a float32 CUDA tensor: one value, or one per row for
    'none').  A gradient that is not wanted is None and costs nothing.
    """
    hp, hs, wp, ws, M, K, V = _head(hidden, weight)
    if reduction not in REDUCTIONS:
        raise ValueError(f"reduction must be one of {sorted(REDUCTIONS)}")
    ids = _class_ids(targets, M)
    lse = _row_values(lse, M, "lse")
    if row_loss is not None:
        row_loss = _row_values(row_loss, M, "row_loss")
    dev, outs = hidden.device, []
    for name, want, out, like in (("d_hidden", want_hidden, d_hidden, hidden),
                                  ("d_weight", want_weight, d_weight, weight)):
        if not want:
            out = None
        elif out is None:
            out = _empty(like.shape, like.dtype, dev, stream)
        elif out.shape != like.shape or out.dtype != like.dtype:
            raise ValueError(f"{name} must have the shape and dtype of {name[2:]}")
        else:
            _apart(name, out, ("hidden", hidden), ("weight", weight), ("targets", targets),
                   ("lse", lse), ("row_loss", row_loss),
                   ("grad_scale", grad_scale if torch.is_tensor(grad_scale) else None))
        outs.append(out)
    d_hidden, d_weight = outs
    if d_hidden is not None and d_weight is not None:
        _apart("d_hidden", d_hidden, ("d_weight", d_weight))
    gs = None
    if grad_scale is not None:
        gs = _device_floats(grad_scale, M if reduction == "none" else 1, dev, "grad_scale", stream)
    dhp, dhs = _rows(d_hidden, "d_hidden")[:2] if d_hidden is not None else (None, 0)
    dwp, dws = _rows(d_weight, "d_weight")[:2] if d_weight is not None else (None, 0)
    dev = _call_device(("hidden", hidden), ("weight", weight), ("targets", ids), ("lse", lse),
                       ("row_loss", row_loss), ("grad_scale", gs if M else None),
                       ("d_hidden", d_hidden), ("d_weight", d_weight))
    if d_hidden is None and d_weight is None:
        return None, None
    with _OnDevice(dev):
        rc = load_library().linear_ce_bwd_ex(
            hp, hs, wp, ws, targets.data_ptr(), lse.data_ptr(), _ptr(row_loss), _ptr(gs), dhp, dhs,
            dwp, dws, M, K, V, int(ignore_index), DTYPES[hidden.dtype], REDUCTIONS[reduction],
            _stream_handle(stream, dev))
    _check(rc, "linear_ce_bwd")
    return d_hidden, d_weight


def linear_greedy(hidden: torch.Tensor, weight: torch.Tensor, tokens: torch.Tensor = None,
                  logprob: torch.Tensor = None, stream=None):
    """The most probable class of each row of ``hidden`` [M, K] @ ``weight``
    [V, K].T (the lowest index of equal ones) and its log-probability, the logits
    never stored: (tokens [M] int64, logprob [M] float32)."""
    hp, hs, wp, ws, M, K, V = _head(hidden, weight)
    dev = hidden.device
    if tokens is None:
        tokens = _empty((M,), torch.int64, dev, stream)
    elif tokens.dtype != torch.int64 or tokens.shape != (M,) or not tokens.is_contiguous():
        raise ValueError("tokens must be contiguous int64 of shape [M]")
    logprob = _empty((M,), torch.float32, dev, stream) if logprob is None else \
        _row_values(logprob, M, "logprob")
    dev = _call_device(("hidden", hidden), ("weight", weight), ("tokens", tokens), ("logprob", logprob))
    with _OnDevice(dev):
        rc = load_library().linear_greedy(hp, hs, wp, ws, tokens.data_ptr(), logprob.data_ptr(), M, K, V,
                                          DTYPES[hidden.dtype], _stream_handle(stream, dev))
    _check(rc, "linear_greedy")
    return tokens, logprob


def _unit_rows(t):
    """t itself where the library can read its rows, else a contiguous copy."""
    ok = (t.shape[1] == 1 or t.stride(1) == 1) and (t.shape[0] <= 1 or t.stride(0) >= t.shape[1])
    return t if ok else t.contiguous()


class FusedLinearCrossEntropy(torch.autograd.Function):
    """Autograd form of linear_ce_fwd / linear_ce_bwd.  Saves the hidden states,
    the weights and two numbers per row; nothing is overwritten, so backward may
    run more than once."""

    @staticmethod
    def forward(ctx, hidden, weight, targets, ignore_index=-100, reduction="mean"):
        h, w = _unit_rows(hidden.detach()), _unit_rows(weight.detach())
        loss, row_loss, lse = linear_ce_fwd(h, w, targets, ignore_index, reduction)
        # a copy where the row losses are the output: a caller may change those
        ctx.save_for_backward(h, w, targets, lse, row_loss.clone() if reduction == "none" else row_loss)
        ctx.ignore_index, ctx.reduction = ignore_index, reduction
        return row_loss if reduction == "none" else loss

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_output):
        h, w, targets, lse, row_loss = ctx.saved_tensors
        gs = grad_output.detach().to(torch.float32).contiguous().reshape(-1)
        dh, dw = linear_ce_bwd(h, w, targets, lse, gs, ctx.ignore_index, ctx.reduction,
                               want_hidden=ctx.needs_input_grad[0],
                               want_weight=ctx.needs_input_grad[1], row_loss=row_loss)
        return dh, dw, None, None, None


def linear_cross_entropy(hidden: torch.Tensor, weight: torch.Tensor, targets: torch.Tensor,
                         ignore_index: int = -100, reduction: str = "mean") -> torch.Tensor:
    """Hard-label cross-entropy of the logits hidden @ weight.T, differentiable in
    both, without forming the logits.  (Captured into a CUDA graph with its
    backward: torch refuses while an eager graph of the same leaves, built on
    another stream, is alive; linear_ce_fwd and linear_ce_bwd know no leaves.)  ``hidden`` is [..., K] and ``targets`` [...]
    (the same leading shape); 'none' returns row losses of the targets' shape."""
    if hidden.shape[:-1] != targets.shape:
        raise ValueError(f"hidden has rows {tuple(hidden.shape[:-1])}, targets {tuple(targets.shape)}")
    out = FusedLinearCrossEntropy.apply(hidden.reshape(-1, hidden.shape[-1]), weight,
                                        targets.reshape(-1).contiguous(), ignore_index, reduction)
    return out.reshape(targets.shape) if reduction == "none" else out


class LinearCrossEntropyLoss(torch.nn.Module):
    """nn.Module form of linear_cross_entropy; the output layer's weights are an
    argument, so they can be shared with an embedding."""

    def __init__(self, ignore_index: int = -100, reduction: str = "mean"):
        super().__init__()
        if reduction not in REDUCTIONS:
            raise ValueError(f"reduction must be one of {sorted(REDUCTIONS)}")
        self.ignore_index, self.reduction = ignore_index, reduction

    def forward(self, hidden, weight, targets):
        return linear_cross_entropy(hidden, weight, targets, self.ignore_index, self.reduction)


# ---------------------------------------------------------------------------
# a router's balance loss


def moe_balance(logits: torch.Tensor, experts: torch.Tensor, balance_coef: float,
                z_coef: float = 0.0, grad_scale=None, want_loss: bool = True,
                want_grad: bool = True, grad: torch.Tensor = None, stream=None):
    """Balance loss and z-loss of router ``logits`` [T, E] whose tokens were sent to
    ``experts`` [T, k] (int64, -1 for an empty slot), in one call:
    (loss, counts, grad).

    loss is balance_coef * E * sum_e (counts_e / (k n)) * mean_t softmax(logits_t)_e
    + z_coef * mean_t logsumexp(logits_t)^2 over the n tokens with a slot in use;
    counts is [E] int64; grad is d(loss)/d(logits) times grad_scale (a number or a
    one-element float32 CUDA tensor), written to ``grad`` when given (which may be
    ``logits`` itself, and shares no memory with the operands otherwise).  loss and grad are None when not wanted.
    """
    lp, ls, T, E = _rows(logits, "logits")
    if experts.dtype != torch.int64 or experts.dim() != 2 or experts.shape[0] != T or \
            experts.shape[1] < 1:
        raise ValueError("experts must be int64 of shape [T, k]")
    k = experts.shape[1]
    es, unit = experts.stride()
    if (k > 1 and unit != 1) or (T > 1 and es < k):
        raise ValueError("experts needs unit column stride and rows that do not overlap")
    dev = logits.device
    gp, gstride = None, 0
    if not want_grad:
        grad = None
    elif grad is None:
        grad = _empty((T, E), logits.dtype, dev, stream)
        gp, gstride = grad.data_ptr(), E
    elif grad.shape != logits.shape or grad.dtype != logits.dtype:
        raise ValueError("grad must match the logits' shape and dtype")
    else:
        gp, gstride = _rows(grad, "grad")[:2]
        if gp != lp or (gstride != ls and T > 1):  # a row is read while others are written
            _apart("grad", grad, ("logits", logits))
        _apart("grad", grad, ("experts", experts),
               ("grad_scale", grad_scale if torch.is_tensor(grad_scale) else None))
    gs = None if grad_scale is None else _device_floats(grad_scale, 1, dev, "grad_scale", stream)
    loss = _empty((), torch.float32, dev, stream) if want_loss else None
    counts = _empty((E,), torch.int64, dev, stream)
    dev = _call_device(("logits", logits), ("experts", experts if T else None), ("grad", grad),
                       ("grad_scale", gs))
    with _OnDevice(dev):
        rc = load_library().moe_balance(lp, ls, experts.data_ptr(), max(es, k), counts.data_ptr(),
                                        _ptr(loss), gp, gstride, _ptr(gs), T, E, k, balance_coef,
                                        z_coef, DTYPES[logits.dtype], _stream_handle(stream, dev))
    _check(rc, "moe_balance")
    return loss, counts, grad


class MoeBalance(torch.autograd.Function):
    """Autograd form of moe_balance: the forward computes the loss and the counts,
    the backward the gradient with the incoming one folded in."""

    @staticmethod
    def forward(ctx, logits, experts, balance_coef, z_coef=0.0):
        x = _unit_rows(logits.detach())
        loss, counts, _ = moe_balance(x, experts, balance_coef, z_coef, want_grad=False)
        ctx.save_for_backward(x, experts)
        ctx.coefs = balance_coef, z_coef
        ctx.mark_non_differentiable(counts)
        return loss, counts

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_output, _):
        x, experts = ctx.saved_tensors
        gs = grad_output.detach().to(torch.float32).contiguous().reshape(-1)
        grad = moe_balance(x, experts, *ctx.coefs, grad_scale=gs, want_loss=False)[2]
        return grad, None, None, None


def moe_balance_loss(logits: torch.Tensor, experts: torch.Tensor, balance_coef: float,
                     z_coef: float = 0.0):
    """(loss, counts) of moe_balance with the loss differentiable in the logits;
    ``logits`` is [..., E], ``experts`` [..., k] with the same leading shape."""
    if logits.shape[:-1] != experts.shape[:-1]:
        raise ValueError(f"logits have tokens {tuple(logits.shape[:-1])}, experts "
                         f"{tuple(experts.shape[:-1])}")
    return MoeBalance.apply(logits.reshape(-1, logits.shape[-1]),
                            experts.reshape(-1, experts.shape[-1]).contiguous(), balance_coef, z_coef)


# ---------------------------------------------------------------------------
# a router's tokens sorted by expert and back


def _launch(where, device, stream, *args):
    """The library's call `where` on `device` and a stream; raises on an error.  (Small calls are
    host time: no objects are made on the common way.)"""
    fn = getattr(load_library(), where)
    if stream is None:
        handle = torch._C._cuda_getCurrentRawStream(device.index)
    else:
        handle = _stream_handle(stream, device)
    if torch._C._cuda_getDevice() == device.index:
        rc = fn(*args, handle)
    else:
        with _OnDevice(device):
            rc = fn(*args, handle)
    if rc != OK:
        raise GbceError(rc, where)


class MoePlan:
    """Where a router's tokens go: ``position`` [T, k], ``source`` [R], ``offsets`` [E + 1] and
    ``counts`` [E], all int32 on one device, as moe_sort makes them (expert e's rows are
    offsets[e] .. offsets[e] + counts[e], offsets[e + 1] being a multiple of ``align``)."""
    __slots__ = ("_position", "_source", "_offsets", "_counts", "_buffer", "_kept", "_places", "tokens",
                 "slots", "rows", "experts", "align", "device")

    def __init__(self, position, source, offsets, counts, align: int = 1):
        index = position.get_device()
        for t, dim in ((position, 2), (source, 1), (offsets, 1), (counts, 1)):
            if t.dtype is not torch.int32 or t.dim() != dim or not t.is_contiguous():
                raise ValueError("position must be contiguous int32 and 2-D, source, offsets and counts 1-D")
            if t.get_device() != index or index < 0:
                _call_device(("position", position), ("source", source), ("offsets", offsets),
                             ("counts", counts))  # says which is where
        if offsets.numel() != counts.numel() + 1:
            raise ValueError("offsets must hold one value more than counts")
        self._position, self._source, self._offsets, self._counts = position, source, offsets, counts
        self._buffer, self._kept = None, (position, source)
        self._places = position.data_ptr(), source.data_ptr()
        self.tokens, self.slots = position.shape
        self.rows, self.experts, self.align = source.numel(), counts.numel(), align
        self.device = position.device

    @classmethod
    def _packed(cls, T, k, rows, E, align, device, stream):
        """A plan whose four parts lie in one buffer, made here."""
        return cls._in_buffer(_empty((T * k + rows + 2 * E + 1,), torch.int32, device, stream), T, k, rows, E, align)

    @classmethod
    def _in_buffer(cls, buffer, T, k, rows, E, align):
        """A plan whose four parts lie in one buffer; tensors are made of them when one is asked for."""
        self = cls.__new__(cls)
        self._buffer, self._kept = buffer, (buffer,)
        p = buffer.data_ptr()
        self._places = p, p + 4 * T * k, p + 4 * (T * k + rows), p + 4 * (T * k + rows + E + 1)
        self.tokens, self.slots, self.rows, self.experts = T, k, rows, E
        self.align, self.device = align, buffer.device
        return self

    def _of(self, kept):
        """The plan of what autograd saved of it (its ``_kept``): itself, or one of the copies that hooks
        on saved tensors gave back."""
        if all(a.data_ptr() == b.data_ptr() for a, b in zip(kept, self._kept)):
            return self
        if len(kept) == 1:
            return MoePlan._in_buffer(*kept, self.tokens, self.slots, self.rows, self.experts, self.align)
        return MoePlan(*kept, self._offsets, self._counts, self.align)

    def _parts(self):
        buffer, slots, rows, E = self._buffer, self.tokens * self.slots, self.rows, self.experts
        if buffer is None:  # another thread has been here
            return
        flat, self._source, self._offsets, self._counts = buffer.split_with_sizes((slots, rows, E + 1, E))
        self._position = flat.view(self.tokens, self.slots)
        self._buffer = None

    @property
    def position(self):
        if self._buffer is not None:
            self._parts()
        return self._position

    @property
    def source(self):
        if self._buffer is not None:
            self._parts()
        return self._source

    @property
    def offsets(self):
        if self._buffer is not None:
            self._parts()
        return self._offsets

    @property
    def counts(self):
        if self._buffer is not None:
            self._parts()
        return self._counts


def moe_sort(experts: torch.Tensor, n_experts: int, align: int = 1, stream=None) -> MoePlan:
    """The plan by which tokens go to ``experts`` [T, k] (int64, -1 for an empty slot) of
    ``n_experts``, each expert's rows padded to a multiple of ``align``: slots sorted by expert,
    an expert's in their order."""
    if experts.dtype != torch.int64 or experts.dim() != 2 or experts.shape[1] < 1:
        raise ValueError("experts must be int64 of shape [T, k]")
    T, k = experts.shape
    es, unit = experts.stride()
    if (k > 1 and unit != 1) or (T > 1 and es < k):
        raise ValueError("experts needs unit column stride and rows that do not overlap")
    dev = _call_device(("experts", experts))
    rows = load_library().moe_plan_rows(T, n_experts, k, align)
    if rows < 0:
        raise GbceError(ERR_SIZE, "moe_sort")
    plan = MoePlan._packed(T, k, rows, n_experts, align, dev, stream)
    _launch("moe_sort", dev, stream, experts.data_ptr(), max(es, k), *plan._places, T, n_experts, k, align)
    return plan


def _plan_matrix(t, rows, plan, name):
    """Pointer and row stride of a matrix with `rows` rows on the plan's device."""
    if t.dim() == 2 and t.dtype in DTYPES and t.get_device() == plan.device.index:
        (n, cols), (step, unit) = t.shape, t.stride()
        if n == rows and unit == 1 and step >= cols:
            return t.data_ptr(), step
    p, step, n, _ = _rows(t, name)  # other strides that will do, or what is wrong
    if n != rows:
        raise ValueError(f"{name} has {n} rows, the plan asks for {rows}")
    if t.device != plan.device:
        raise ValueError(f"{name} is on {t.device}, the plan on {plan.device}")
    return p, step


def _plan_output(out, name, rows, H, like, plan, stream, *inputs):
    """(out, pointer, row stride): allocated when None, else checked against the inputs."""
    if out is None:
        out = torch.empty((rows, H), dtype=like.dtype, device=plan.device) if stream is None else \
            _empty((rows, H), like.dtype, plan.device, stream)
        return out, out.data_ptr(), H
    p, step = _plan_matrix(out, rows, plan, name)
    if out.shape[1] != H or out.dtype != like.dtype:
        raise ValueError(f"{name} must be {like.dtype} of {H} columns")
    _apart(name, out, *inputs, ("position", plan.position), ("source", plan.source))
    return out, p, step


def _plan_weights(w, plan, like, name):
    """(pointer, row stride, dtype) of a [T, k] matrix of float32 or of the rows' type."""
    if w.dtype != torch.float32 and w.dtype != like.dtype:
        raise TypeError(f"{name} must be float32 or {like.dtype}, not {w.dtype}")
    p, step = _plan_matrix(w, plan.tokens, plan, name)
    if w.shape[1] != plan.slots:
        raise ValueError(f"{name} must have {plan.slots} columns, one for each slot")
    return p, step, DTYPES[w.dtype]


def moe_dispatch(x: torch.Tensor, plan: MoePlan, out: torch.Tensor = None, stream=None) -> torch.Tensor:
    """Rows of ``x`` [T, H] in the plan's order, [R, H]: row position[t, j] is x[t]; rows that
    are no slot's are zeros.  (Its gradient is moe_combine without weights.)"""
    xp, xs = _plan_matrix(x, plan.tokens, plan, "x")
    H = x.shape[1]
    out, op, os_ = _plan_output(out, "out", plan.rows, H, x, plan, stream, ("x", x))
    _launch("moe_dispatch", plan.device, stream, xp, xs, plan._places[0], plan._places[1], op, os_,
            plan.tokens, H, plan.slots, plan.rows, DTYPES[x.dtype])
    return out


def moe_combine(y: torch.Tensor, plan: MoePlan, weights: torch.Tensor = None, out: torch.Tensor = None,
                stream=None) -> torch.Tensor:
    """Rows of ``y`` [R, H] back by token, [T, H]: row t is the sum over t's slots of
    weights[t, j] * y[position[t, j]] (weights [T, k] in float32 or y's type; None: 1)."""
    yp, ys = _plan_matrix(y, plan.rows, plan, "y")
    H = y.shape[1]
    wp, ws, wt = (None, 0, 0) if weights is None else _plan_weights(weights, plan, y, "weights")
    out, op, os_ = _plan_output(out, "out", plan.tokens, H, y, plan, stream, ("y", y), ("weights", weights))
    _launch("moe_combine", plan.device, stream, yp, ys, plan._places[0], wp, ws, wt, op, os_, plan.tokens, H,
            plan.slots, plan.rows, DTYPES[y.dtype])
    return out


def moe_combine_bwd(d_out: torch.Tensor, y: torch.Tensor, plan: MoePlan, weights: torch.Tensor,
                    want_y: bool = True, want_weights: bool = True, d_y: torch.Tensor = None,
                    d_weights: torch.Tensor = None, stream=None):
    """(d_y, d_weights) of moe_combine with weights, for the incoming ``d_out`` [T, H]; rows of
    d_y that are no slot's are zeros, and so are the gradients of empty slots' weights.  A
    gradient that is not wanted is None; ``y`` is read for the weights' only, and may be None
    without."""
    dp, ds = _plan_matrix(d_out, plan.tokens, plan, "d_out")
    H = d_out.shape[1]
    yp, ys = None, 0
    if y is not None:
        yp, ys = _plan_matrix(y, plan.rows, plan, "y")
        if y.shape[1] != H or d_out.dtype != y.dtype:
            raise ValueError(f"d_out must be {y.dtype} of {y.shape[1]} columns, as y")
    elif want_weights:
        raise ValueError("y is needed for the weights' gradient")
    wp, ws, wt = _plan_weights(weights, plan, d_out, "weights")
    inputs = ("d_out", d_out), ("y", y), ("weights", weights)
    dyp, dys, dwp, dws = None, 0, None, 0
    if want_y:
        d_y, dyp, dys = _plan_output(d_y, "d_y", plan.rows, H, d_out, plan, stream, *inputs)
    else:
        d_y = None
    if want_weights:
        d_weights, dwp, dws = _plan_output(d_weights, "d_weights", plan.tokens, plan.slots, weights, plan,
                                           stream, *inputs, ("d_y", d_y))
    else:
        d_weights = None
    if d_y is None and d_weights is None:
        return None, None
    _launch("moe_combine_bwd", plan.device, stream, dp, ds, yp, ys, plan._places[0], plan._places[1], wp, ws, wt,
            dyp, dys, dwp, dws, plan.tokens, H, plan.slots, plan.rows, DTYPES[d_out.dtype])
    return d_y, d_weights


class DispatchTokens(torch.autograd.Function):
    """Autograd form of moe_dispatch; saves the plan's memory, so one that is written to before
    the backward is refused there."""

    @staticmethod
    def forward(ctx, x, plan):
        ctx.plan = plan
        ctx.save_for_backward(*plan._kept)
        return moe_dispatch(_unit_rows(x.detach()), plan)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_output):
        return moe_combine(_unit_rows(grad_output.detach()), ctx.plan._of(ctx.saved_tensors)), None


class CombineTokens(torch.autograd.Function):
    """Autograd form of moe_combine; saves the weights, the plan's memory and, where the weights
    need a gradient, the rows, so backward may run more than once and refuses what was written to
    before it."""

    @staticmethod
    def forward(ctx, y, plan, weights=None):
        y = _unit_rows(y.detach())
        w = None if weights is None else _unit_rows(weights.detach())
        ctx.plan = plan
        rows = (y,) if w is not None and ctx.needs_input_grad[2] else ()
        ctx.save_for_backward(*plan._kept, *(() if w is None else (w,)), *rows)
        return moe_combine(y, plan, w)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_output):
        g = _unit_rows(grad_output.detach())
        saved = ctx.saved_tensors  # once: a recomputed forward's can be unpacked no second time
        n = len(ctx.plan._kept)
        plan, saved = ctx.plan._of(saved[:n]), saved[n:]
        if not saved:
            return moe_dispatch(g, plan), None, None
        w, y = saved if len(saved) == 2 else (*saved, None)
        dy, dw = moe_combine_bwd(g, y, plan, w, want_y=ctx.needs_input_grad[0],
                                 want_weights=ctx.needs_input_grad[2])
        return dy, None, dw


def dispatch_tokens(x: torch.Tensor, plan: MoePlan) -> torch.Tensor:
    """moe_dispatch of ``x`` [..., H], differentiable (the leading sizes hold the plan's tokens).
    (Captured into a CUDA graph with its backward: as for linear_cross_entropy.)"""
    return DispatchTokens.apply(x.reshape(-1, x.shape[-1]), plan)


def combine_tokens(y: torch.Tensor, plan: MoePlan, weights: torch.Tensor = None) -> torch.Tensor:
    """moe_combine of ``y`` [R, H] with ``weights`` [T, k] or None, differentiable in both:
    [T, H].  (Captured into a CUDA graph with its backward: as for linear_cross_entropy.)"""
    return CombineTokens.apply(y, plan, weights)


# ---------------------------------------------------------------------------
# the norm of all gradients


def _dense(t):
    """Do the tensor's values fill one stretch of memory, in whatever order of its axes?"""
    if t.is_contiguous():
        return True
    step = 1
    for size, stride in sorted(zip(t.shape, t.stride()), key=lambda p: p[1]):
        if size != 1 and stride != step:
            return False
        step *= size
    return True


def _same_order(t, o):
    """Do the values of two tensors that each fill one stretch of memory lie there in the same order?
    (The stride of an axis of one says nothing.)"""
    return t.is_contiguous() and o.is_contiguous() or t.shape == o.shape and \
        all(a == b for n, a, b in zip(t.shape, t.stride(), o.stride()) if n != 1)


def _tensor_list(tensors, name):
    """(device index or None, pointers, sizes, types, whether all are contiguous) of the tensors of
    a call on many; a list at a time, as a model has hundreds."""
    devices = set(map(torch.Tensor.get_device, tensors))
    if -1 in devices:
        raise ValueError(f"{name} must be CUDA tensors")
    if len(devices) > 1:
        raise ValueError(f"{name} are on several devices: {sorted(devices)}")
    try:
        types = array.array("i", [DTYPES[t.dtype] for t in tensors])
    except KeyError as e:
        raise TypeError(f"{name} must be float32, bfloat16 or float16, not {e.args[0]}") from None
    contiguous = all(map(torch.Tensor.is_contiguous, tensors))
    if not contiguous:
        for t in tensors:
            if not _dense(t):
                raise ValueError(f"{name} must each fill one stretch of memory, not strides {t.stride()} "
                                 f"of shape {tuple(t.shape)}")
    pointers = array.array("Q", map(torch.Tensor.data_ptr, tensors))
    sizes = array.array("q", map(torch.Tensor.numel, tensors))
    return next(iter(devices), None), pointers, sizes, types, contiguous


def _writable(tensors, name):
    """Raises ValueError where parameters would be written to: torch.nn.utils.clip_grad_norm_ takes
    parameters and scales their gradients, clip_grad_norm takes the gradients."""
    for t in tensors:
        if t.requires_grad and t.is_leaf:
            raise ValueError(f"{name} hold leaves that require gradients: clip_grad_norm takes gradients, "
                             "not their parameters")


def _norm_call(where, tensors, norm_type, norm, stream, max_norm=None, eps=0.0, outs=None):
    kind = NORMS.get(float(norm_type))
    if kind is None:
        raise ValueError(f"norm_type must be 1, 2 or inf, not {norm_type}")
    tensors = [tensors] if torch.is_tensor(tensors) else list(tensors)
    if outs is not None:
        outs = [outs] if torch.is_tensor(outs) else list(outs)
        if len(outs) != len(tensors):
            raise ValueError(f"{len(outs)} outs for {len(tensors)} tensors")
        outs = [o for o, t in zip(outs, tensors) if t is not None]
    tensors = [t for t in tensors if t is not None]
    index, pointers, sizes, types, contiguous = _tensor_list(tensors, "tensors")
    if norm is None:
        norm = _empty((), torch.float32, "cuda" if index is None else tensors[0].device, stream)
    elif norm.dtype != torch.float32 or norm.numel() != 1:
        raise ValueError("norm must be a one-element float32 CUDA tensor")
    dev = _call_device(("norm", norm), ("tensors", tensors[0] if tensors else None))
    args = [pointers.buffer_info()[0], sizes.buffer_info()[0], types.buffer_info()[0], len(tensors), kind]
    if max_norm is not None:
        _writable(tensors if outs is None else outs, "tensors" if outs is None else "outs")
        results = pointers
        if outs is not None:
            out_index, results, out_sizes, out_types, out_contiguous = _tensor_list(outs, "outs")
            if out_index != index or out_types != types or out_sizes != sizes or \
                    not (contiguous and out_contiguous or all(map(_same_order, tensors, outs))):
                raise ValueError("outs must match the tensors in size, order of values, dtype and device")
        args.insert(1, results.buffer_info()[0])
        args += [float(max_norm), float(eps)]
    _launch(where, dev, stream, *args, norm.data_ptr())
    return norm


def grad_norm(tensors, norm_type: float = 2.0, norm: torch.Tensor = None, stream=None) -> torch.Tensor:
    """The norm (1, 2 or inf) of all ``tensors`` (float32, bfloat16 and float16 in any mixture;
    None entries are passed over) taken as one vector: a 0-dim float32 CUDA tensor.  Each tensor
    fills one stretch of memory, in whatever order of its axes; nothing is synchronised."""
    return _norm_call("grad_norm", tensors, norm_type, norm, stream)


def clip_grad_norm(tensors, max_norm: float, norm_type: float = 2.0, eps: float = 1e-6, outs=None,
                   norm: torch.Tensor = None, stream=None) -> torch.Tensor:
    """Scales ``tensors`` (gradients, not their parameters: leaves that require gradients are not
    written to) by min(1, max_norm / (norm + eps)), in place or into ``outs``, and returns the norm
    they had, as grad_norm does.  There is one out for each tensor, of the same type and, where they
    are not contiguous, the same shape and strides; it shares no memory with any other tensor.
    Where the norm keeps the limit, tensors in place are not written."""
    return _norm_call("clip_grad_norm", tensors, norm_type, norm, stream, max_norm, eps, outs)
