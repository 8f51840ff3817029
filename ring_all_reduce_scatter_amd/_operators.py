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
from ._binding import F32, GradPlan, RarError, _sizes, dtype_code, lib

# These calls can take less time on the GPU than their Python does on the
# host (a layer norm of one row: 3 us), so the way to the library is kept
# short: types and functions are looked up once, the current stream is read
# as an address, and shapes are read once per tensor.

NORM_L2, NORM_MAX = 0, 1
_I32, _I64 = 0, 1


def _width(t, what: str) -> int:
    if t.dim() == 0 or t.shape[-1] == 0:
        raise ValueError(f"{what} must have rows of at least one element, got shape {tuple(t.shape)}")
    return t.shape[-1]


def _rows(t, dim: int, what: str):
    """(rows, elements between rows) of a tensor (..., dim)."""
    if t.dim() == 0 or t.shape[-1] != dim:
        raise ValueError(f"{what} must have rows of {dim} elements, got shape {tuple(t.shape)}")
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
    """A contiguous tensor of n elements, or None."""
    if t is not None and (t.numel() != n or not t.is_contiguous()):
        raise ValueError(f"{what} must be contiguous with {n} elements, got shape {tuple(t.shape)}")


def _floats(t, n: int, what: str):
    """n contiguous float32 values, or None."""
    _vector(t, n, what)
    if t is not None and dtype_code(t) != F32:
        raise ValueError(f"{what} must be float32, got {t.dtype}")


def _dptr(t) -> int:
    if not t.is_cuda:
        raise ValueError(f"expected a GPU tensor, got one on {t.device}")
    return t.data_ptr()


def _ptr(t):
    return None if t is None else _dptr(t)


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


def _call(name: str, *args):
    rc = getattr(_binding._lib or lib(), name)(*args)
    if rc:
        raise RarError(rc, name)


def _workspace(ws):
    if ws is None:
        return None, 0
    if not ws.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return _dptr(ws), ws.numel() * ws.element_size()


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


class GradClip:
    """Global norm and clipping of fixed gradient tensors, prepared once.

    grads: device tensors of any mix of float32, float16 and bfloat16, each
    filling one range of memory.  outs: where clip() writes, one tensor per
    gradient with its shape and strides (any of the three types); None clips
    in place.  workspace: grad_clip_workspace_bytes([g.numel() for g in
    grads]) bytes.  Everything must stay alive and keep its storage, and
    nothing else may write the workspace, while this object is used; its
    calls use the one workspace, so they must follow one another (one stream,
    or streams that wait for each other)."""

    def __init__(self, grads, workspace, outs=None, stream=None):
        grads = list(grads)
        outs = None if outs is None else list(outs)
        for g in grads:
            if not _is_dense(g):
                raise ValueError("gradients must fill one range of memory (no gaps, no expanded dimensions)")
        if outs is not None:
            if len(outs) != len(grads):
                raise ValueError("need one output per gradient")
            for g, o in zip(grads, outs):
                if o.shape != g.shape or (o.stride() != g.stride() and not (o.is_contiguous() and g.is_contiguous())):
                    raise ValueError("an output must have its gradient's shape and strides")
        n = len(grads)
        ptrs = (ctypes.c_void_p * max(n, 1))(*[_dptr(g) for g in grads])
        dts = (ctypes.c_int * max(n, 1))(*[dtype_code(g) for g in grads])
        optrs = odts = None
        if outs is not None:
            optrs = (ctypes.c_void_p * max(n, 1))(*[_dptr(o) for o in outs])
            odts = (ctypes.c_int * max(n, 1))(*[dtype_code(o) for o in outs])
        if workspace is None:
            raise ValueError("a workspace is needed")
        ws, nbytes = _workspace(workspace)
        self._keep = (grads, outs, workspace)
        self._ws = workspace
        self._plan = GradPlan()
        _call("rar_grad_prepare", ptrs, optrs, _sizes([g.numel() for g in grads]), dts, odts, n, ws, nbytes,
              ctypes.byref(self._plan), _stream(stream, workspace))
        self._ref = ctypes.byref(self._plan)

    def norm(self, norm, norm_type: int = NORM_L2, scale: float = 1.0, stream=None):
        """norm (one float32 on the device) <- |scale| * the norm of all gradients."""
        _floats(norm, 1, "norm")
        _call("rar_grad_norm", self._ref, norm_type, scale, _ptr(norm), _stream(stream, self._ws))

    def clip(self, max_norm: float, norm, norm_type: int = NORM_L2, scale: float = 1.0, stream=None):
        """The same norm, and every gradient times scale * min(1, max_norm / (norm + 1e-6))."""
        _floats(norm, 1, "norm")
        _call("rar_grad_clip", self._ref, norm_type, scale, max_norm, _ptr(norm), _stream(stream, self._ws))


def grad_norm(grads, workspace, norm, norm_type: int = NORM_L2, scale: float = 1.0, stream=None):
    """One GradClip(grads, workspace).norm(...): preparation and norm."""
    GradClip(grads, workspace, stream=stream).norm(norm, norm_type, scale, stream)


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
    _call("rar_embedding_forward", _dptr(weight), wstride, dtype_code(weight), vocab, dim, _dptr(ids), code, tokens,
          scale, _dptr(out), ostride, dtype_code(out), _stream(stream, out))


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
    _call("rar_embedding_backward", _dptr(dout), dstride, dtype_code(dout), _dptr(ids), code, tokens, vocab, dim,
          scale, -1 if padding_id is None else padding_id, int(accumulate), _dptr(dweight), wstride,
          dtype_code(dweight), ws, nbytes, _stream(stream, dweight))


# ------------------------------------------------------------------ layer norm

def _weight_type(default: int, *ts):
    codes = {dtype_code(t) for t in ts if t is not None}
    if len(codes) > 1:
        raise ValueError("weight, bias and their gradients must share one type")
    return codes.pop() if codes else default


def layernorm_forward(x, weight, bias, out, eps: float = 1e-5, mean=None, rstd=None, stream=None):
    """out <- (x - mean) * rstd * weight + bias over the last dimension.
    weight and bias may be None; mean and rstd (float32, one per row) receive
    the statistics that layernorm_backward needs."""
    dim = _width(x, "x")
    rows, xstride = _rows(x, dim, "x")
    ystride = _out_rows(out, dim, rows, "out")
    if out.dtype != x.dtype:
        raise ValueError("out must have x's type")
    _vector(weight, dim, "weight")
    _vector(bias, dim, "bias")
    _floats(mean, rows, "mean")
    _floats(rstd, rows, "rstd")
    dt = dtype_code(x)
    wdt = _weight_type(dt, weight, bias)
    _call("rar_layernorm_forward", _dptr(x), xstride, _ptr(weight), _ptr(bias), rows, dim, dt, wdt, eps, _dptr(out),
          ystride, _ptr(mean), _ptr(rstd), _stream(stream, x))


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
    for t, name in ((weight, "weight"), (dweight, "dweight"), (dbias, "dbias")):
        _vector(t, dim, name)
    _floats(mean, rows, "mean")
    _floats(rstd, rows, "rstd")
    dt = dtype_code(x)
    wdt = _weight_type(dt, weight, dweight, dbias)
    ws, nbytes = _workspace(workspace)
    _call("rar_layernorm_backward", _dptr(dout), dstride, _dptr(x), xstride, _ptr(weight), _ptr(mean), _ptr(rstd),
          rows, dim, dt, wdt, _ptr(dx), gstride, _ptr(dweight), _ptr(dbias), int(accumulate), ws, nbytes,
          _stream(stream, x))
