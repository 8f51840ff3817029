"""Overlaps that the gradient operators' calls refuse or serve, before any
launch.  CPU only: the addresses are never read."""
import ctypes

import pytest
import torch

import ring_all_reduce_scatter_amd as rar
from ring_all_reduce_scatter_amd import _binding as b

OK, EINVAL, EDTYPE, EALIGN, EWORKSPACE, EOVERLAP = 0, 1, 2, 3, 4, 7
B, G = 1 << 40, 1 << 30


def _empty_plan():
    L, p = rar.lib(), b.GradPlan()
    need = L.rar_grad_workspace_bytes(None, 0)
    assert L.rar_grad_prepare(None, None, None, None, None, 0, B, need, ctypes.byref(p), None) == OK
    return p, need


def test_norm_in_the_workspace_is_refused():
    """Written there it would change descriptors (addresses) or counts that
    the same call reads."""
    L = rar.lib()
    p, need = _empty_plan()
    for at in (B, B + 4, B + p.desc_offset, B + p.partial_offset + 8, B + p.result_offset, B + need - 4):
        assert L.rar_grad_norm(ctypes.byref(p), 0, 1.0, at, None) == EOVERLAP, hex(at)
        assert L.rar_grad_clip(ctypes.byref(p), 1, 1.0, 1.0, at, None) == EOVERLAP, hex(at)


def test_norm_among_the_tensors_is_refused():
    """Where the plan points to the set's host arrays."""
    L = rar.lib()
    p, _ = _empty_plan()
    assert not p.set
    grads, outs = (ctypes.c_void_p * 3)(B + G, B + G + 256, None), (ctypes.c_void_p * 3)(B + G + 512, B + G, None)
    counts = (ctypes.c_size_t * 3)(32, 1, 0)
    f16, f32 = (ctypes.c_int * 3)(1, 1, 1), (ctypes.c_int * 3)(0, 0, 0)

    def refused(offset, outs=None, odts=None, dts=f32):
        s = b.GradSet(*(None if a is None else ctypes.addressof(a) for a in (grads, outs, counts, dts, odts)), 3)
        p.set = ctypes.pointer(s)
        # the limit is refused afterwards, so that nothing is launched
        rc = L.rar_grad_clip(ctypes.byref(p), 0, 1.0, -1.0, B + G + offset, None)
        assert rc in (EINVAL, EOVERLAP)
        return rc == EOVERLAP

    for dts, es in ((f32, 4), (f16, 2)):
        for bad in (0, 32 * es - 4, 256):
            assert refused(bad, dts=dts), bad
        for good in (-4, 32 * es, 252, 260, 512):
            assert not refused(good, dts=dts), good
    assert refused(512, outs, f16) and refused(512 + 60, outs, f16) and not refused(512 + 64, outs, f16)
    assert refused(512 + 64, outs, f32)
    grads[0] = B + G + 2  # an element inside, the other beside the four bytes
    counts[0] = 1
    assert refused(0, dts=f16) and not refused(4, dts=f16)
    assert L.rar_grad_norm(ctypes.byref(p), 0, 1.0, B + G, None) == EOVERLAP


def test_set_prepared_for_its_norm_alone():
    """Tensors that are read only may overlap, but for the workspace."""
    L, p = rar.lib(), b.GradPlan()
    counts = (ctypes.c_size_t * 2)(0, 3000)
    dts = (ctypes.c_int * 2)(0, 0)
    need = L.rar_grad_workspace_bytes(counts, 2)

    def prepare(grads, n=2, ws=B + 2 * G, nbytes=need, dts=dts):
        return L.rar_grad_prepare_norm((ctypes.c_void_p * 2)(*grads), counts, dts, n, ws, nbytes, ctypes.byref(p), None)

    assert L.rar_grad_prepare_norm(None, None, None, 0, B, need, ctypes.byref(p), None) == OK and p.clips == 0
    assert prepare([None, None], n=1) == OK and p.ntiles == 0
    assert L.rar_grad_clip(ctypes.byref(p), 0, 1.0, 1.0, B + 5 * G, None) == EINVAL
    assert prepare([None, B + 2 * G + 256]) == EOVERLAP and prepare([None, B + 2 * G - 4]) == EOVERLAP
    assert prepare([None, None]) == EOVERLAP and prepare([None, B + 2]) == EALIGN
    assert prepare([None, B], ws=None) == EWORKSPACE and prepare([None, B], nbytes=64) == EWORKSPACE
    assert prepare([None, B], dts=(ctypes.c_int * 2)(0, 3)) == EDTYPE
    assert L.rar_grad_prepare(None, None, None, None, None, 0, B, need, ctypes.byref(p), None) == OK and p.clips == 1
    with pytest.raises(ValueError, match="norm alone"):
        rar.GradClip([torch.zeros(4)], torch.zeros(1 << 16, dtype=torch.uint8), outs=[torch.zeros(4)], norm_only=True)


def _ln(x, y, rows=10, dim=64, xs=200, ys=200, dt=2):
    return rar.lib().rar_layernorm_forward(x, xs, None, None, rows, dim, dt, 0, 1e-5, y, ys, None, None, None)


def test_rows_that_share_bytes_are_refused():
    """Columns of one matrix are apart only where neither reaches the other's
    columns, in its own row or the next."""
    e = 2
    for off in (1, 63, 137, 199, 200 + 63, 5 * 200 + 137):
        assert _ln(B, B + off * e) == EOVERLAP, off
        assert _ln(B + off * e, B) == EOVERLAP, -off
    assert _ln(B, B + 64 * e, xs=199) == EOVERLAP
    assert _ln(B, B + 100 * e, xs=100) == EOVERLAP  # every second row of x is a row of y's
    assert _ln(B, B + 64 * e, xs=32) == EOVERLAP  # x's rows overlap


def test_dimensions_of_one_element_have_no_step():
    """An output in its gradient's order, whatever the strides of dimensions
    of one element say."""
    ws = torch.zeros(rar.grad_clip_workspace_bytes([32]), dtype=torch.uint8)
    g = torch.zeros(8, 4).t()[None]
    o = torch.zeros(1, 8, 4).as_strided((1, 4, 8), (1, 1, 4))
    assert g.stride() != o.stride() and not g.is_contiguous() and not o.is_contiguous()
    with pytest.raises(ValueError, match="GPU tensor"):  # only the host check is left
        rar.GradClip([g], ws, outs=[o])
    for bad in (torch.zeros(1, 4, 8), torch.zeros(4, 8), torch.zeros(4, 1, 8).transpose(0, 1)):
        with pytest.raises(ValueError, match="shape and strides"):
            rar.GradClip([g], ws, outs=[bad])
