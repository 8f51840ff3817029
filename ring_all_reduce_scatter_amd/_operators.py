"""Operators next to the rings: global gradient norm and clipping, embedding
lookup and gradient, activation checkpoints in 8 bits, layer norm and the
gated feed-forward block forward and backward (include/rar.h states their
formulas).

Argument marshalling only, as in _binding: the caller owns every tensor,
outputs and workspaces included, and every step runs in the library's
kernels on the given stream (None: the current one).  A tensor of rows may
have any strides as long as its rows are whole (last dimension contiguous)
and equally far apart; what the kernels could not read or write in place is
refused with ValueError before any launch.
"""
from __future__ import annotations

import ctypes

from . import _binding
from ._binding import F32, GradPlan, GradSet, RarError, _sizes, dtype_code, lib

# These calls can take less time on the GPU than their Python does on the
# host (a layer norm of one row: 3 us), so the way to the library is kept
# short: types and functions are looked up once, the current stream is read
# as an address, and shapes are read once per tensor.

NORM_L2, NORM_MAX = 0, 1
ACT_SILU, ACT_GELU, ACT_GELU_TANH = 0, 1, 2
KEEP_NONE, KEEP_ROWS, KEEP_CHECKPOINT = 0, 1, 2
_I32, _I64 = 0, 1


def _width(t, what: str) -> int:
    shape = t.shape
    if not shape or shape[-1] == 0:
        raise ValueError(f"{what} must have rows of at least one element, got shape {tuple(shape)}")
    return shape[-1]


def _rows(t, dim: int, what: str):
    """(rows, elements between rows) of a tensor (..., dim)."""
    shape = t.shape
    if not shape or shape[-1] != dim:
        raise ValueError(f"{what} must have rows of {dim} elements, got shape {tuple(shape)}")
    if t.is_contiguous():
        return t.numel() // dim, dim
    if dim > 1 and t.stride(-1) != 1:
        raise ValueError(f"{what} must be contiguous along its last dimension")
    rows, stride = 1, dim
    # dimensions of one element have no step; the others must nest evenly
    for n, s in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
        if n == 1:
            continue
        if rows == 1:
            stride = s
        elif s != stride * rows:
            raise ValueError(f"{what} must have rows equally far apart, got strides {t.stride()}")
        rows *= n
    return rows, stride


def _out_rows(t, dim: int, rows: int, what: str):
    n, stride = _rows(t, dim, what)
    if n != rows:
        raise ValueError(f"{what} has {n} rows, {rows} are needed")
    if n > 1 and stride < dim:
        raise ValueError(f"{what} has rows that overlap")
    return stride if n > 1 else dim


def _vector(t, n: int, what: str):
    """Address of a contiguous tensor of n elements, None for None."""
    if t is None:
        return None
    if t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous with {n} elements, got shape {tuple(t.shape)}")
    return t.data_ptr()


def _floats(t, n: int, what: str):
    """Address of n contiguous float32 values, None for None."""
    if t is not None and dtype_code(t) != F32:
        raise ValueError(f"{what} must be float32, got {t.dtype}")
    return _vector(t, n, what)


def _on_gpu(*ts):
    """Refuses host tensors and tensors of two GPUs: a kernel reads all of them
    from one."""
    device = None
    for t in ts:
        if t is None:
            continue
        index = t.get_device()
        if index != device:
            if index < 0:
                raise ValueError(f"expected a GPU tensor, got one on {t.device}")
            if device is not None:
                raise ValueError(f"tensors must be on one device, got some on cuda:{device} and some on cuda:{index}")
            device = index


_id_codes: dict = {}  # filled by the first call, so importing needs no torch


def _ids(ids):
    if not _id_codes:
        import torch
        _id_codes.update({torch.int32: _I32, torch.int64: _I64})
    code = _id_codes.get(ids.dtype)
    if code is None:
        raise TypeError(f"ids must be int32 or int64, got {ids.dtype}")
    if not ids.is_contiguous():
        raise ValueError("ids must be contiguous")
    return code


_current_stream = _current_device = None


def _stream(stream, t):
    """Address of the given stream, or of the current one on t's device.  A
    device's default stream has no address of its own: a launch with none runs
    on the current device, which must then be t's."""
    if stream is not None:
        return stream if isinstance(stream, int) else stream.cuda_stream
    global _current_stream, _current_device
    if _current_stream is None:
        import torch
        # the address without a Stream object around it, where torch offers that
        if torch.cuda.device_count() > 1:  # the only one is the current one
            _current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
        _current_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                                  lambda index: torch.cuda.current_stream(index).cuda_stream)
    index = t.get_device()
    address = _current_stream(index)
    if not address and _current_device and _current_device() != index:
        raise ValueError(f"tensors on cuda:{index} need it as the current device (cuda:{_current_device()} is), or a "
                         "stream of it")
    return address


def _check(rc: int, what: str):
    if rc:
        raise RarError(rc, what)


def _workspace(ws):
    if ws is None:
        return None, 0
    if not ws.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return ws.data_ptr(), ws.numel() * ws.element_size()


# ------------------------------------------------------------------ norm and clip

def grad_clip_workspace_bytes(counts) -> int:
    """Workspace of a GradClip over tensors of these element counts."""
    return lib().rar_grad_workspace_bytes(_sizes(counts), len(counts))


def _is_dense(t) -> bool:
    """The elements fill one range of memory, in any order of dimensions."""
    if t.is_contiguous():
        return True
    want = 1
    for s, n in sorted((s, n) for s, n in zip(t.stride(), t.shape) if n != 1):
        if s != want:
            return False
        want *= n
    return True


def _same_steps(o, g) -> bool:
    """Equal strides wherever a dimension has a second element."""
    return all(a == b for a, b, n in zip(o.stride(), g.stride(), g.shape) if n != 1)


class GradClip:
    """Global norm and clipping of fixed gradient tensors, prepared once.

    grads: device tensors of any mix of float32, float16 and bfloat16, each
    filling one range of memory.  outs: where clip() writes, one tensor per
    gradient with its shape and strides (any of the three types); None clips
    in place.  norm_only: nothing is written and clip() is refused, so the
    gradients may overlap (one that is held twice counts twice).  workspace: grad_clip_workspace_bytes([g.numel() for g in
    grads]) bytes.  Everything must stay alive and keep its storage, and
    nothing else may write the workspace, while this object is used.  The
    preparation is work on `stream` that the host does not wait for, and all
    calls use the one workspace: a call must come after the preparation and
    after the calls before it (one stream, or streams that wait for each
    other).

    Preparing takes three short launches and one more for every 90 tensors,
    20 us of the host for 16 tensors and 110 us for 200, so a program whose
    gradients keep their storage prepares once."""

    def __init__(self, grads, workspace, outs=None, stream=None, norm_only: bool = False):
        grads = list(grads)
        outs = None if outs is None else list(outs)
        for g in grads:
            if not _is_dense(g):
                raise ValueError("gradients must fill one range of memory (no gaps, no expanded dimensions)")
        if outs is not None:
            if norm_only:
                raise ValueError("a set prepared for its norm alone has no outputs")
            if len(outs) != len(grads):
                raise ValueError("need one output per gradient")
            for g, o in zip(grads, outs):
                if o.shape != g.shape or (o.stride() != g.stride() and not (o.is_contiguous() and g.is_contiguous())
                                          and not _same_steps(o, g)):
                    raise ValueError("an output must have its gradient's shape and strides")
        if workspace is None:
            raise ValueError("a workspace is needed")
        _on_gpu(workspace, *grads, *(outs or ()))
        n = len(grads)
        ptrs = (ctypes.c_void_p * max(n, 1))(*[g.data_ptr() for g in grads])
        dts = (ctypes.c_int * max(n, 1))(*[dtype_code(g) for g in grads])
        optrs = odts = None
        if outs is not None:
            optrs = (ctypes.c_void_p * max(n, 1))(*[o.data_ptr() for o in outs])
            odts = (ctypes.c_int * max(n, 1))(*[dtype_code(o) for o in outs])
        ws, nbytes = _workspace(workspace)
        self._plan = GradPlan()
        counts, plan, st = _sizes([g.numel() for g in grads]), ctypes.byref(self._plan), _stream(stream, workspace)
        self._keep = (grads, outs, workspace, ptrs, optrs, counts, dts, odts)
        self._ws = workspace
        if norm_only:
            rc = (_binding._lib or lib()).rar_grad_prepare_norm(ptrs, counts, dts, n, ws, nbytes, plan, st)
        else:
            rc = (_binding._lib or lib()).rar_grad_prepare(ptrs, optrs, counts, dts, odts, n, ws, nbytes, plan, st)
        _check(rc, "rar_grad_prepare")
        # the calls compare norm's place with these
        self._set = GradSet(*(None if a is None else ctypes.addressof(a) for a in self._keep[3:]), n)
        self._plan.set = ctypes.pointer(self._set)
        self._ref = plan

    def norm(self, norm, norm_type: int = NORM_L2, scale: float = 1.0, stream=None):
        """norm (one float32 on the device, apart from the tensors) <- |scale|
        * the norm of all gradients."""
        address = _floats(norm, 1, "norm")
        _on_gpu(self._ws, norm)
        rc = (_binding._lib or lib()).rar_grad_norm(self._ref, norm_type, scale, address, _stream(stream, self._ws))
        _check(rc, "rar_grad_norm")

    def clip(self, max_norm: float, norm, norm_type: int = NORM_L2, scale: float = 1.0, stream=None):
        """The same norm, and every gradient times scale * min(1, max_norm / (norm + 1e-6))."""
        address = _floats(norm, 1, "norm")
        _on_gpu(self._ws, norm)
        rc = (_binding._lib or lib()).rar_grad_clip(
            self._ref, norm_type, scale, max_norm, address, _stream(stream, self._ws))
        _check(rc, "rar_grad_clip")


def grad_norm(grads, workspace, norm, norm_type: int = NORM_L2, scale: float = 1.0, stream=None):
    """One GradClip(grads, workspace, norm_only=True).norm(...): preparation
    and norm, 30 us for 16 small tensors (prepared 5), 133 us for 200 tensors
    of 378 million elements in all (prepared 114)."""
    GradClip(grads, workspace, stream=stream, norm_only=True).norm(norm, norm_type, scale, stream)


def clip_grad_norm(grads, max_norm: float, workspace, norm, outs=None, norm_type: int = NORM_L2, scale: float = 1.0,
                   stream=None):
    """One GradClip(grads, workspace, outs).clip(...): preparation, norm and clip."""
    GradClip(grads, workspace, outs, stream).clip(max_norm, norm, norm_type, scale, stream)


# ------------------------------------------------------------------ embedding

def embedding_forward(weight, ids, out, scale: float = 1.0, stream=None):
    """out[..., :] <- scale * weight[ids[...], :]; ids outside the table give zeros."""
    code = _ids(ids)
    if weight.dim() != 2:
        raise ValueError(f"weight must be (vocab, dim), got shape {tuple(weight.shape)}")
    vocab, dim = weight.shape[0], _width(weight, "weight")
    tokens = ids.numel()
    ostride = _out_rows(out, dim, tokens, "out")
    wstride = _out_rows(weight, dim, vocab, "weight")
    _on_gpu(weight, ids, out)
    rc = (_binding._lib or lib()).rar_embedding_forward(
        weight.data_ptr(), wstride, dtype_code(weight), vocab, dim, ids.data_ptr(), code, tokens, scale,
        out.data_ptr(), ostride, dtype_code(out), _stream(stream, out))
    _check(rc, "rar_embedding_forward")


def embedding_workspace_bytes(tokens: int, vocab: int, dim: int) -> int:
    return lib().rar_embedding_workspace_bytes(tokens, vocab, dim)


def embedding_backward(dout, ids, dweight, workspace, scale: float = 1.0, padding_id: int | None = None,
                       accumulate: bool = False, stream=None):
    """dweight[v, :] <- scale * the sum of dout[..., :] where ids == v (plus
    dweight[v, :] with accumulate); padding_id and ids outside the table
    contribute nothing."""
    code = _ids(ids)
    if dweight.dim() != 2:
        raise ValueError(f"dweight must be (vocab, dim), got shape {tuple(dweight.shape)}")
    vocab, dim = dweight.shape[0], _width(dweight, "dweight")
    tokens = ids.numel()
    n, dstride = _rows(dout, dim, "dout")
    if n != tokens:
        raise ValueError(f"dout has {n} rows for {tokens} ids")
    wstride = _out_rows(dweight, dim, vocab, "dweight")
    ws, nbytes = _workspace(workspace)
    _on_gpu(dout, ids, dweight, workspace)
    rc = (_binding._lib or lib()).rar_embedding_backward(
        dout.data_ptr(), dstride, dtype_code(dout), ids.data_ptr(), code, tokens, vocab, dim, scale,
        -1 if padding_id is None else padding_id, int(accumulate), dweight.data_ptr(), wstride, dtype_code(dweight),
        ws, nbytes, _stream(stream, dweight))
    _check(rc, "rar_embedding_backward")


# ------------------------------------------------------------------ activation checkpoints

def checkpoint_bytes(rows: int, dim: int) -> int:
    """Bytes of a checkpoint of rows x dim: 33 for every 32 columns begun of a row."""
    return lib().rar_checkpoint_bytes(rows, dim)


def _checkpoint(t, rows: int, dim: int, what: str = "checkpoint"):
    """(address, bytes) of a checkpoint's buffer."""
    if t.element_size() != 1 or t.is_floating_point() or not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous bytes (uint8)")
    n, need = t.numel(), rows * 33 * ((dim + 31) // 32)
    if n < need:
        raise ValueError(f"{what} holds {n} bytes, {need} are needed")
    return t.data_ptr(), n


def checkpoint_pack(x, checkpoint, stream=None):
    """checkpoint (checkpoint_bytes(rows, dim) bytes or more) <- x (..., dim)
    in 8 bits: blocks of 32 columns of a row share a power-of-two step, 1/64
    to 1/128 of the block's largest value.  A block with an infinity or NaN
    comes back as NaN."""
    dim = _width(x, "x")
    rows, stride = _rows(x, dim, "x")
    ck, nbytes = _checkpoint(checkpoint, rows, dim)
    code = dtype_code(x)
    _on_gpu(x, checkpoint)
    rc = (_binding._lib or lib()).rar_checkpoint_pack(x.data_ptr(), stride, rows, dim, code, ck, nbytes,
                                                      _stream(stream, x))
    _check(rc, "rar_checkpoint_pack")


def checkpoint_unpack(checkpoint, out, stream=None):
    """out (..., dim), of any of the three types, <- the values that a
    checkpoint of its shape stands for."""
    dim = _width(out, "out")
    rows, stride = _rows(out, dim, "out")
    if rows > 1 and stride < dim:
        raise ValueError("out has rows that overlap")
    ck, nbytes = _checkpoint(checkpoint, rows, dim)
    code = dtype_code(out)
    _on_gpu(checkpoint, out)
    rc = (_binding._lib or lib()).rar_checkpoint_unpack(ck, nbytes, rows, dim, out.data_ptr(),
                                                        stride if rows > 1 else dim, code, _stream(stream, out))
    _check(rc, "rar_checkpoint_unpack")


# ------------------------------------------------------------------ layer norm

def _weight_type(default: int, *ts):
    code = None
    for t in ts:
        if t is not None:
            if code is not None and dtype_code(t) != code:
                raise ValueError("weight, bias and their gradients must share one type")
            code = dtype_code(t)
    return default if code is None else code


def layernorm_forward(x, weight, bias, out, eps: float = 1e-5, mean=None, rstd=None, stream=None):
    """out <- (x - mean) * rstd * weight + bias over the last dimension.
    weight and bias may be None; mean and rstd (float32, one per row) receive
    the statistics that layernorm_backward needs."""
    dim = _width(x, "x")
    rows, xstride = _rows(x, dim, "x")
    ystride = _out_rows(out, dim, rows, "out")
    if out.dtype != x.dtype:
        raise ValueError("out must have x's type")
    w, b = _vector(weight, dim, "weight"), _vector(bias, dim, "bias")
    m, r = _floats(mean, rows, "mean"), _floats(rstd, rows, "rstd")
    dt = dtype_code(x)
    wdt = _weight_type(dt, weight, bias)
    _on_gpu(x, weight, bias, out, mean, rstd)
    rc = (_binding._lib or lib()).rar_layernorm_forward(
        x.data_ptr(), xstride, w, b, rows, dim, dt, wdt, eps, out.data_ptr(), ystride, m, r, _stream(stream, x))
    _check(rc, "rar_layernorm_forward")


def layernorm_workspace_bytes(rows: int, dim: int) -> int:
    return lib().rar_layernorm_workspace_bytes(rows, dim)


def layernorm_backward(dout, x, weight, mean, rstd, dx, dweight, dbias, workspace, accumulate: bool = False,
                       stream=None):
    """Gradients of layernorm_forward.  dx, dweight and dbias may be None;
    with accumulate the sums are added to what dweight and dbias hold."""
    dim = _width(x, "x")
    rows, xstride = _rows(x, dim, "x")
    n, dstride = _rows(dout, dim, "dout")
    if n != rows:
        raise ValueError(f"dout has {n} rows, x has {rows}")
    if dout.dtype != x.dtype or (dx is not None and dx.dtype != x.dtype):
        raise ValueError("dout and dx must have x's type")
    gstride = dim if dx is None else _out_rows(dx, dim, rows, "dx")
    w, dw, db = _vector(weight, dim, "weight"), _vector(dweight, dim, "dweight"), _vector(dbias, dim, "dbias")
    m, r = _floats(mean, rows, "mean"), _floats(rstd, rows, "rstd")
    dt = dtype_code(x)
    wdt = _weight_type(dt, weight, dweight, dbias)
    ws, nbytes = _workspace(workspace)
    _on_gpu(dout, x, weight, mean, rstd, dx, dweight, dbias, workspace)
    rc = (_binding._lib or lib()).rar_layernorm_backward(
        dout.data_ptr(), dstride, x.data_ptr(), xstride, w, m, r, rows, dim, dt, wdt,
        None if dx is None else dx.data_ptr(), gstride, dw, db, int(accumulate), ws, nbytes, _stream(stream, x))
    _check(rc, "rar_layernorm_backward")


def layernorm_forward_checkpoint(x, weight, bias, out, checkpoint, eps: float = 1e-5, mean=None, rstd=None,
                                 stream=None):
    """layernorm_forward that also writes x's checkpoint (checkpoint_pack's
    bytes) from the same reading of x."""
    dim = _width(x, "x")
    rows, xstride = _rows(x, dim, "x")
    ystride = _out_rows(out, dim, rows, "out")
    if out.dtype != x.dtype:
        raise ValueError("out must have x's type")
    ck, nbytes = _checkpoint(checkpoint, rows, dim)
    w, b = _vector(weight, dim, "weight"), _vector(bias, dim, "bias")
    m, r = _floats(mean, rows, "mean"), _floats(rstd, rows, "rstd")
    dt = dtype_code(x)
    wdt = _weight_type(dt, weight, bias)
    _on_gpu(x, weight, bias, out, checkpoint, mean, rstd)
    rc = (_binding._lib or lib()).rar_layernorm_forward_checkpoint(
        x.data_ptr(), xstride, w, b, rows, dim, dt, wdt, eps, out.data_ptr(), ystride, m, r, ck, nbytes,
        _stream(stream, x))
    _check(rc, "rar_layernorm_forward_checkpoint")


def layernorm_backward_checkpoint(dout, checkpoint, weight, mean, rstd, dx, dweight, dbias, workspace,
                                  accumulate: bool = False, stream=None):
    """layernorm_backward with the values of x's checkpoint in x's place."""
    dim = _width(dout, "dout")
    rows, dstride = _rows(dout, dim, "dout")
    if dx is not None and dx.dtype != dout.dtype:
        raise ValueError("dx must have dout's type")
    ck, cbytes = _checkpoint(checkpoint, rows, dim)
    gstride = dim if dx is None else _out_rows(dx, dim, rows, "dx")
    w, dw, db = _vector(weight, dim, "weight"), _vector(dweight, dim, "dweight"), _vector(dbias, dim, "dbias")
    m, r = _floats(mean, rows, "mean"), _floats(rstd, rows, "rstd")
    dt = dtype_code(dout)
    wdt = _weight_type(dt, weight, dweight, dbias)
    ws, nbytes = _workspace(workspace)
    _on_gpu(dout, checkpoint, weight, mean, rstd, dx, dweight, dbias, workspace)
    rc = (_binding._lib or lib()).rar_layernorm_backward_checkpoint(
        dout.data_ptr(), dstride, ck, cbytes, w, m, r, rows, dim, dt, wdt, None if dx is None else dx.data_ptr(),
        gstride, dw, db, int(accumulate), ws, nbytes, _stream(stream, dout))
    _check(rc, "rar_layernorm_backward_checkpoint")


# ------------------------------------------------------------------ gated feed-forward

def _ff_weights(x, wgate, wup):
    """(dim, hidden, rows between wgate's, wup's rows)"""
    dim = _width(x, "x")
    if wgate.dim() != 2 or wgate.shape[0] == 0 or wup.shape != wgate.shape:
        raise ValueError(f"wgate and wup must both be (hidden, {dim}), got shapes {tuple(wgate.shape)} and "
                         f"{tuple(wup.shape)}")
    if wgate.dtype != x.dtype or wup.dtype != x.dtype:
        raise ValueError("wgate and wup must have x's type")
    return dim, wgate.shape[0], _rows(wgate, dim, "wgate")[1], _rows(wup, dim, "wup")[1]


def _ff_kept(gate, up, rows: int, hidden: int, dtype, written: bool):
    """(keep, address and stride or bytes of gate, the same of up)"""
    if gate is None and up is None:
        return KEEP_NONE, None, 0, None, 0
    if gate is None or up is None or gate.dtype != up.dtype:
        raise ValueError("gate and up must be of one kind")
    if gate.dtype != dtype:
        return (KEEP_CHECKPOINT, *_checkpoint(gate, rows, hidden, "gate"), *_checkpoint(up, rows, hidden, "up"))
    steps = []
    for t, what in ((gate, "gate"), (up, "up")):
        if written:
            steps.append(_out_rows(t, hidden, rows, what))
            continue
        n, stride = _rows(t, hidden, what)
        if n != rows:
            raise ValueError(f"{what} has {n} rows, {rows} are needed")
        steps.append(stride)
    return KEEP_ROWS, gate.data_ptr(), steps[0], up.data_ptr(), steps[1]


def gated_ff_forward(x, wgate, wup, out, act: int = ACT_SILU, gate=None, up=None, stream=None):
    """out (..., hidden) <- act(x wgate^T) * (x wup^T) for x (..., dim) and
    weights (hidden, dim) of its type; they may be the halves of one matrix.
    gate and up receive the two projections for gated_ff_backward: tensors of
    out's shape and type, or checkpoints in 8 bits (checkpoint_bytes(rows,
    hidden) bytes each), written straight from the sums."""
    dim, hidden, gstride, ustride = _ff_weights(x, wgate, wup)
    rows, xstride = _rows(x, dim, "x")
    ostride = _out_rows(out, hidden, rows, "out")
    if out.dtype != x.dtype:
        raise ValueError("out must have x's type")
    keep, g, gs, u, us = _ff_kept(gate, up, rows, hidden, x.dtype, True)
    dt = dtype_code(x)
    _on_gpu(x, wgate, wup, out, gate, up)
    rc = (_binding._lib or lib()).rar_gated_ff_forward(
        x.data_ptr(), xstride, wgate.data_ptr(), gstride, wup.data_ptr(), ustride, rows, dim, hidden, dt, act,
        out.data_ptr(), ostride, keep, g, gs, u, us, _stream(stream, x))
    _check(rc, "rar_gated_ff_forward")


def gated_ff_workspace_bytes(rows: int, dim: int, hidden: int, dtype) -> int:
    """Workspace of gated_ff_backward for activations of this torch type."""
    import torch
    return lib().rar_gated_ff_workspace_bytes(rows, dim, hidden, dtype_code(torch.empty(0, dtype=dtype)))


def gated_ff_backward(dout, x, wgate, wup, gate, up, dx, dwgate, dwup, workspace, act: int = ACT_SILU,
                      accumulate: bool = False, stream=None):
    """Gradients of gated_ff_forward from what it kept in gate and up.  dx (x's
    shape and type) may be None, dwgate and dwup (the weights' shape, x's type
    or float32) may both be None; with accumulate the weights' gradients are
    added to what they hold.  The projections' own gradients are rounded to
    x's type on the way: in float16 one beyond 65,504 becomes infinite."""
    dim, hidden, gstride, ustride = _ff_weights(x, wgate, wup)
    rows, xstride = _rows(x, dim, "x")
    n, dstride = _rows(dout, hidden, "dout")
    if n != rows:
        raise ValueError(f"dout has {n} rows, x has {rows}")
    if dout.dtype != x.dtype or (dx is not None and dx.dtype != x.dtype):
        raise ValueError("dout and dx must have x's type")
    keep, g, gs, u, us = _ff_kept(gate, up, rows, hidden, x.dtype, False)
    if keep == KEEP_NONE:
        raise ValueError("gate and up are needed")
    if (dwgate is None) != (dwup is None) or (dwup is not None and dwup.dtype != dwgate.dtype):
        raise ValueError("dwgate and dwup must be of one kind")
    dt = dtype_code(x)
    xs = dim if dx is None else _out_rows(dx, dim, rows, "dx")
    wdt, dg, dgs, du, dus = dt, None, dim, None, dim
    if dwgate is not None:
        wdt = dtype_code(dwgate)
        if wdt != dt and wdt != F32:
            raise ValueError("dwgate and dwup must have x's type or be float32")
        if dwgate.dim() != 2 or dwup.dim() != 2:
            raise ValueError("dwgate and dwup must have the weights' shape")
        dgs, dus = _out_rows(dwgate, dim, hidden, "dwgate"), _out_rows(dwup, dim, hidden, "dwup")
        dg, du = dwgate.data_ptr(), dwup.data_ptr()
    ws, nbytes = _workspace(workspace)
    _on_gpu(dout, x, wgate, wup, gate, up, dx, dwgate, dwup, workspace)
    rc = (_binding._lib or lib()).rar_gated_ff_backward(
        dout.data_ptr(), dstride, x.data_ptr(), xstride, wgate.data_ptr(), gstride, wup.data_ptr(), ustride, keep, g,
        gs, u, us, rows, dim, hidden, dt, act, None if dx is None else dx.data_ptr(), xs, dg, dgs, du, dus, wdt,
        int(accumulate), ws, nbytes, _stream(stream, x))
    _check(rc, "rar_gated_ff_backward")
