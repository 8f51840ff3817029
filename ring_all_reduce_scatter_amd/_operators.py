"""Operators next to the rings: global gradient norm and clipping, embedding
lookup and gradient, layer norm forward and backward (include/rar.h states
their formulas).

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
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError(f"expected a GPU tensor, got one on {t.device}")


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


_current_stream = None


def _stream(stream, t):
    """Address of the given stream, or of the current one on t's device."""
    if stream is not None:
        return stream if isinstance(stream, int) else stream.cuda_stream
    global _current_stream
    if _current_stream is None:
        import torch
        # the address without a Stream object around it, where torch offers that
        _current_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                                  lambda index: torch.cuda.current_stream(index).cuda_stream)
    return _current_stream(t.get_device())


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
        _on_gpu(norm)
        rc = (_binding._lib or lib()).rar_grad_norm(self._ref, norm_type, scale, address, _stream(stream, self._ws))
        _check(rc, "rar_grad_norm")

    def clip(self, max_norm: float, norm, norm_type: int = NORM_L2, scale: float = 1.0, stream=None):
        """The same norm, and every gradient times scale * min(1, max_norm / (norm + 1e-6))."""
        address = _floats(norm, 1, "norm")
        _on_gpu(norm)
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
