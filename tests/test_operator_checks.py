"""Refusals of the operators next to the rings (norm and clip, embedding,
layer norm), by the binding and by the C entry points, before any launch.
CPU only: host tensors reach the binding's own checks, and the C calls get
addresses that are never read."""
import ctypes
import math

import pytest
import torch

import ring_all_reduce_scatter_amd as rar
from ring_all_reduce_scatter_amd import _binding as b

OK, EINVAL, EDTYPE, EALIGN, EWORKSPACE, ENOTSUP, EOVERLAP = 0, 1, 2, 3, 4, 6, 7
B = 1 << 40  # a base address; calls that would touch it must be refused first
G = 1 << 30


def _raises(match, fn, *a, **k):
    with pytest.raises((ValueError, TypeError), match=match):
        fn(*a, **k)


# ------------------------------------------------------------------ binding

def test_clip_binding_refusals():
    ws = torch.zeros(rar.grad_clip_workspace_bytes([64, 64]), dtype=torch.uint8)
    g = [torch.zeros(8, 8), torch.zeros(64)]
    _raises("range of memory", rar.GradClip, [g[0][:, :4]], ws)
    _raises("range of memory", rar.GradClip, [torch.zeros(8, 1).expand(8, 8)], ws)
    _raises("one output per gradient", rar.GradClip, g, ws, outs=g[:1])
    _raises("shape and strides", rar.GradClip, [g[0]], ws, outs=[torch.zeros(8, 8).t()])
    _raises("shape and strides", rar.GradClip, [g[0]], ws, outs=[torch.zeros(64)])
    _raises("unsupported dtype|GPU tensor", rar.GradClip, [torch.zeros(8, dtype=torch.float64)], ws)
    _raises("GPU tensor", rar.GradClip, [g[0].t()], ws)  # dense in another order: only the host check is left


def test_embedding_binding_refusals():
    w, ids, out = torch.zeros(10, 6), torch.zeros(4, dtype=torch.int64), torch.zeros(4, 6)
    f = rar.embedding_forward
    _raises("int32 or int64", f, w, ids.to(torch.int16), out)
    _raises("ids must be contiguous", f, w, torch.zeros(8, dtype=torch.int64)[::2], out)
    _raises("vocab, dim", f, w[0], ids, out)
    _raises("rows of 6", f, w, ids, torch.zeros(4, 5))
    _raises("3 rows, 4 are needed", f, w, ids, torch.zeros(3, 6))
    _raises("last dimension", f, w, ids, torch.zeros(4, 12)[:, ::2])
    _raises("overlap", f, w, ids, torch.zeros(1, 6).expand(4, 6))
    _raises("at least one element", f, torch.zeros(10, 0), ids, torch.zeros(4, 0))
    _raises("GPU tensor", f, w, ids, out)
    ws = torch.zeros(rar.embedding_workspace_bytes(4, 10, 6), dtype=torch.uint8)
    bw = rar.embedding_backward
    _raises("rows for 4 ids", bw, torch.zeros(5, 6), ids, w, ws)
    _raises("rows of 6", bw, torch.zeros(4, 7), ids, w, ws)
    _raises("equally far apart", bw, torch.zeros(2, 3, 6)[:, :2], ids, w, ws)
    _raises("workspace must be contiguous", bw, out, ids, w, torch.zeros(2048, dtype=torch.uint8)[::2])
    _raises("overlap", bw, out, ids, torch.zeros(1, 6).expand(10, 6), ws)
    _raises("GPU tensor", bw, out, ids, w, ws)


def test_layernorm_binding_refusals():
    x, w, s = torch.zeros(4, 6), torch.zeros(6), torch.zeros(4)
    f = rar.layernorm_forward
    _raises("at least one element", f, torch.tensor(1.0), w, w, x)
    _raises("out must have x's type", f, x, w, w, x.half())
    _raises("rows of 6", f, x, w, w, torch.zeros(4, 7))
    _raises("contiguous with 6", f, x, torch.zeros(7), w, torch.zeros(4, 6))
    _raises("contiguous with 6", f, x, torch.zeros(12)[::2], w, torch.zeros(4, 6))
    _raises("one type", f, x, w, w.half(), torch.zeros(4, 6))
    _raises("mean must be float32", f, x, w, w, torch.zeros(4, 6), mean=s.half())
    _raises("contiguous with 4", f, x, w, w, torch.zeros(4, 6), rstd=torch.zeros(5))
    bw = rar.layernorm_backward
    ws = torch.zeros(rar.layernorm_workspace_bytes(4, 6), dtype=torch.uint8)
    _raises("dout has 3 rows", bw, torch.zeros(3, 6), x, w, s, s, x, w, w, ws)
    _raises("x's type", bw, x.half(), x, w, s, s, x, w, w, ws)
    _raises("x's type", bw, x, x, w, s, s, x.half(), w, w, ws)
    _raises("one type", bw, x, x, w, s, s, x, w.half(), w, ws)
    _raises("overlap", bw, x, x, w, s, s, torch.zeros(1, 6).expand(4, 6), w, w, ws)


def test_rows_of_views():
    """What counts as rows equally far apart."""
    from ring_all_reduce_scatter_amd._operators import _is_dense, _rows
    big = torch.zeros(5, 7, 32)
    assert _rows(big, 32, "t") == (35, 32)
    assert _rows(big[:, :, 3:20], 17, "t") == (35, 32)
    assert _rows(big[1:3, 2, :], 32, "t") == (2, 7 * 32)
    assert _rows(big[:, 2:3, :], 32, "t") == (5, 7 * 32)
    assert _rows(big[2, 2, :9], 9, "t") == (1, 9)
    assert _rows(torch.zeros(1, 32).expand(6, 32), 32, "t") == (6, 0)
    assert _rows(torch.zeros(32).expand(2, 3, 32), 32, "t") == (6, 0)
    assert _rows(torch.zeros(6, 1), 1, "t") == (6, 1)
    assert _rows(torch.zeros(6, 9)[:, :1], 1, "t") == (6, 9)
    assert _rows(torch.zeros(0, 9), 9, "t") == (0, 9)
    for bad in (big.transpose(0, 1), big[:, ::2, :][:, :3], torch.zeros(9, 32).t()):
        with pytest.raises(ValueError):
            _rows(bad, bad.shape[-1], "t")
    assert _is_dense(big.permute(2, 0, 1)) and _is_dense(big[1:3]) and not _is_dense(big[:, 1:])


# ------------------------------------------------------------------ C entry points

def _arr(t, xs):
    return (t * max(1, len(xs)))(*xs)


def _prepare(grads, counts, dts, outs=None, odts=None, ws=B + 64 * G, nbytes=None, plan=True):
    L = rar.lib()
    cs = _arr(ctypes.c_size_t, counts)
    need = L.rar_grad_workspace_bytes(cs, len(counts)) if nbytes is None else nbytes
    p = b.GradPlan()
    return L.rar_grad_prepare(_arr(ctypes.c_void_p, grads), None if outs is None else _arr(ctypes.c_void_p, outs), cs,
                              _arr(ctypes.c_int, dts), None if odts is None else _arr(ctypes.c_int, odts), len(counts),
                              ws, need, ctypes.byref(p) if plan else None, None)


def test_grad_prepare_refusals():
    c = [1000, 3000]
    g, o = [B, B + G], [B + 2 * G, B + 3 * G]
    assert _prepare(g, c, [0, 0], plan=False) == EINVAL
    assert _prepare(g, c, [0, 3]) == EDTYPE
    assert _prepare(g, c, [0, 0], o, [0, -1]) == EDTYPE
    assert _prepare(g, c, [0, 0], o, None) == EINVAL
    assert _prepare([0, B], c, [0, 0]) == EOVERLAP
    assert _prepare([B + 2, B + G], c, [0, 0]) == EALIGN
    assert _prepare([B + 1, B + G], c, [1, 0]) == EALIGN
    assert _prepare(g, c, [0, 0], [B + 2 * G, B + 3 * G + 2], [0, 0]) == EALIGN
    assert _prepare(g, c, [0, 0], ws=0) == EWORKSPACE
    assert _prepare(g, c, [0, 0], nbytes=64) == EWORKSPACE
    assert _prepare(g, c, [0, 0], ws=B + 64 * G + 8) == EALIGN
    assert _prepare(g, [1 << 46, 1], [0, 0], nbytes=1 << 40) == EINVAL
    # overlaps: in place twice, an output in another input, types that differ in place, the workspace
    assert _prepare([B, B + 2000], c, [0, 0]) == EOVERLAP
    assert _prepare(g, c, [0, 0], [B + 2 * G, B + 2 * G + 2000], [0, 0]) == EOVERLAP
    assert _prepare(g, c, [0, 0], [B + G + 4, B + 3 * G], [0, 0]) == EOVERLAP
    assert _prepare(g, c, [0, 0], [B + 4, B + 3 * G], [0, 0]) == EOVERLAP
    assert _prepare(g, c, [0, 0], [B, B + 3 * G], [1, 0]) == EOVERLAP
    assert _prepare(g, c, [0, 0], [B + G, B], [0, 0]) == EOVERLAP
    assert _prepare(g, c, [0, 0], ws=B + 512) == EOVERLAP
    assert _prepare(g, c, [0, 0], o, [0, 0], ws=B + G - 256) == EOVERLAP
    assert _prepare(g, c, [0, 0], o, [0, 0], ws=B + 3 * G - 256) == EOVERLAP


def test_grad_plan_of_an_empty_set_and_launch_refusals():
    L = rar.lib()
    p = b.GradPlan()
    need = L.rar_grad_workspace_bytes(None, 0)
    assert need > 0
    assert L.rar_grad_workspace_bytes(None, 3) == 0
    assert L.rar_grad_prepare(None, None, None, None, None, 0, B, need, ctypes.byref(p), None) == OK
    assert p.ntiles == 0
    counts = _arr(ctypes.c_size_t, [0, 0])
    ptrs, dts = _arr(ctypes.c_void_p, [0, 0]), _arr(ctypes.c_int, [0, 1])
    assert L.rar_grad_prepare(ptrs, None, counts, dts, None, 2, B, 1 << 20, ctypes.byref(p), None) == OK
    assert p.ntiles == 0
    ref = ctypes.byref(p)
    assert L.rar_grad_norm(None, 0, 1.0, B + G, None) == EINVAL
    assert L.rar_grad_norm(ref, 2, 1.0, B + G, None) == EINVAL
    assert L.rar_grad_norm(ref, 0, math.nan, B + G, None) == EINVAL
    assert L.rar_grad_norm(ref, 0, math.inf, B + G, None) == EINVAL
    assert L.rar_grad_norm(ref, 0, 1.0, None, None) == EOVERLAP
    assert L.rar_grad_norm(ref, 0, 1.0, B + G + 2, None) == EALIGN
    assert L.rar_grad_clip(ref, 0, 1.0, -1.0, B + G, None) == EINVAL
    assert L.rar_grad_clip(ref, 0, 1.0, math.nan, B + G, None) == EINVAL
    assert L.rar_grad_norm(ctypes.byref(b.GradPlan()), 0, 1.0, B + G, None) == EINVAL


def _embed(w=B, ws=64, wd=2, vocab=100, dim=64, ids=B + G, idt=1, tokens=10, out=B + 2 * G, os_=64, od=2):
    return rar.lib().rar_embedding_forward(w, ws, wd, vocab, dim, ids, idt, tokens, 1.0, out, os_, od, None)


def test_embedding_forward_refusals():
    assert _embed(tokens=0) == OK
    assert _embed(tokens=0, w=None, ids=None, out=None) == OK
    assert _embed(vocab=0) == EINVAL and _embed(dim=0) == EINVAL
    assert _embed(ws=63) == EINVAL and _embed(os_=63) == EINVAL
    assert _embed(wd=3) == EDTYPE and _embed(od=-1) == EDTYPE and _embed(idt=2) == EDTYPE
    assert _embed(w=None) == EOVERLAP and _embed(ids=None) == EOVERLAP and _embed(out=None) == EOVERLAP
    assert _embed(w=B + 1) == EALIGN and _embed(ids=B + G + 4) == EALIGN and _embed(out=B + 1, od=0) == EALIGN
    assert _embed(out=B + 99 * 128) == EOVERLAP and _embed(out=B + G - 100) == EOVERLAP
    assert _embed(tokens=1 << 31) == ENOTSUP and _embed(vocab=1 << 31) == ENOTSUP
    assert _embed(ws=1 << 62, vocab=8) == EINVAL


def _embed_grad(d=B, ds=64, dd=2, ids=B + G, idt=1, tokens=10, vocab=100, dim=64, dw=B + 2 * G, ws=64, wd=0,
                work=B + 3 * G, nbytes=None, pad=-1):
    L = rar.lib()
    need = L.rar_embedding_workspace_bytes(tokens, vocab, dim) if nbytes is None else nbytes
    return L.rar_embedding_backward(d, ds, dd, ids, idt, tokens, vocab, dim, 1.0, pad, 0, dw, ws, wd, work, need, None)


def test_embedding_backward_refusals():
    assert _embed_grad(vocab=0) == EINVAL and _embed_grad(dim=0) == EINVAL and _embed_grad(ws=63) == EINVAL
    assert _embed_grad(dd=4) == EDTYPE and _embed_grad(wd=4) == EDTYPE and _embed_grad(idt=-1) == EDTYPE
    assert _embed_grad(d=None) == EOVERLAP and _embed_grad(ids=None) == EOVERLAP and _embed_grad(dw=None) == EOVERLAP
    assert _embed_grad(d=B + 1) == EALIGN and _embed_grad(dw=B + 2) == EALIGN and _embed_grad(work=B + 8) == EALIGN
    assert _embed_grad(work=None) == EWORKSPACE and _embed_grad(nbytes=16) == EWORKSPACE
    assert _embed_grad(dw=B + 128) == EOVERLAP and _embed_grad(work=B + G - 16) == EOVERLAP
    assert _embed_grad(work=B + 2 * G + 256) == EOVERLAP
    assert _embed_grad(tokens=1 << 31, nbytes=1 << 40) == ENOTSUP
    L = rar.lib()
    assert L.rar_embedding_workspace_bytes(1 << 31, 10, 10) == 0 and L.rar_embedding_workspace_bytes(1, 0, 10) == 0


def _ln(x=B, xs=64, w=B + G, bias=B + G + 4096, rows=10, dim=64, dt=2, wd=0, eps=1e-5, y=B + 2 * G, ys=64,
        mean=B + 3 * G, rstd=B + 4 * G):
    return rar.lib().rar_layernorm_forward(x, xs, w, bias, rows, dim, dt, wd, eps, y, ys, mean, rstd, None)


def test_layernorm_forward_refusals():
    assert _ln(rows=0) == OK and _ln(rows=0, x=None, y=None) == OK
    assert _ln(dim=0) == EINVAL and _ln(ys=63) == EINVAL
    assert _ln(eps=-1.0) == EINVAL and _ln(eps=math.nan) == EINVAL
    assert _ln(dt=3) == EDTYPE and _ln(wd=3) == EDTYPE
    assert _ln(x=None) == EOVERLAP and _ln(y=None) == EOVERLAP
    assert _ln(x=B + 1) == EALIGN and _ln(w=B + G + 2) == EALIGN and _ln(mean=B + 3 * G + 2) == EALIGN
    assert _ln(y=B + 2) == EOVERLAP and _ln(y=B, ys=65) == EOVERLAP  # not x itself
    assert _ln(mean=B + 16) == EOVERLAP and _ln(rstd=B + 3 * G + 4) == EOVERLAP and _ln(y=B + G) == EOVERLAP
    assert _ln(rows=1 << 50) == EINVAL


def _ln_grad(dy=B, dys=64, x=B + G, xs=64, w=B + 2 * G, mean=B + 3 * G, rstd=B + 4 * G, rows=10, dim=64, dt=2, wd=0,
             dx=B + 5 * G, dxs=64, dw=B + 6 * G, db=B + 7 * G, ws=B + 8 * G, nbytes=None):
    L = rar.lib()
    need = L.rar_layernorm_workspace_bytes(rows, dim) if nbytes is None else nbytes
    return L.rar_layernorm_backward(dy, dys, x, xs, w, mean, rstd, rows, dim, dt, wd, dx, dxs, dw, db, 0, ws, need,
                                    None)


def test_layernorm_backward_refusals():
    assert _ln_grad(dim=0) == EINVAL and _ln_grad(dxs=63) == EINVAL
    assert _ln_grad(dt=-1) == EDTYPE and _ln_grad(wd=7) == EDTYPE
    for name in ("dy", "x", "mean", "rstd"):
        assert _ln_grad(**{name: None}) == EOVERLAP, name
    assert _ln_grad(dy=B + 1) == EALIGN and _ln_grad(dw=B + 6 * G + 2) == EALIGN and _ln_grad(ws=B + 8) == EALIGN
    assert _ln_grad(ws=None) == EWORKSPACE and _ln_grad(nbytes=8) == EWORKSPACE
    assert _ln_grad(dx=B + 2) == EOVERLAP and _ln_grad(dx=B, dxs=70) == EOVERLAP and _ln_grad(dx=B + G + 64) == EOVERLAP
    assert _ln_grad(dw=B + 7 * G + 4) == EOVERLAP and _ln_grad(ws=B + 6 * G + 16) == EOVERLAP
    assert _ln_grad(db=B + 2 * G + 4) == EOVERLAP and _ln_grad(dw=B + 3 * G) == EOVERLAP
    assert rar.lib().rar_layernorm_workspace_bytes(5, 0) == 0


def test_sizes_that_no_launch_holds():
    """Refused before anything is enqueued: a launch holds fewer than 2^32 threads."""
    big = (1 << 24) * 8192  # 2^24 tiles of bf16 elements
    L = rar.lib()
    need = L.rar_grad_workspace_bytes(_arr(ctypes.c_size_t, [big]), 1)
    assert need > 0
    assert _prepare([B], [big], [2], ws=B - (1 << 36), nbytes=need) == ENOTSUP
    assert _embed(tokens=(1 << 30) + 1) == ENOTSUP
    assert _embed(tokens=1 << 30, dim=4096, ws=4096, os_=4096, vocab=8, out=1 << 45) == ENOTSUP
    assert _embed_grad(tokens=(1 << 30) + 1, nbytes=1 << 40) == ENOTSUP
    assert _embed_grad(vocab=1 << 30, dim=4096, ws=4096, ds=4096, dw=1 << 45, work=1 << 44) == ENOTSUP
    assert _ln(dim=1 << 31, ys=1 << 31) == ENOTSUP and _ln_grad(dim=1 << 31) == ENOTSUP
    assert L.rar_layernorm_workspace_bytes(5, 1 << 31) == 0
