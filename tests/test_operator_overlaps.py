"""Overlaps that the gradient operators' calls refuse or serve, before any
launch.  CPU only: the addresses are never read."""
import ctypes

import pytest
import torch

import ring_all_reduce_scatter_amd as rar
from ring_all_reduce_scatter_amd import _binding as b
from ring_all_reduce_scatter_amd import _operators as op

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


def test_merged_ranges():
    begins, ends = op._merged([(100, 200), (300, 304), (150, 260), (200, 210), (260, 264)])
    assert list(zip(begins, ends)) == [(100, 260), (260, 264), (300, 304)]
    for a, n, hit in ((96, 4, False), (97, 4, True), (256, 4, True), (260, 4, True), (264, 4, False), (296, 4, False),
                      (297, 4, True), (300, 4, True), (304, 4, False), (0, 4, False), (0, 1000, True)):
        assert op._touches(begins, ends, a, n) == hit, (a, n)
    assert not op._touches([], [], 5, 4)


def test_norm_among_the_tensors_is_refused_by_the_binding():
    clip = op.GradClip.__new__(op.GradClip)  # without a device there is no plan to prepare
    flat, outs = torch.zeros(64), torch.zeros(32, dtype=torch.float16)
    clip._keep = ([flat[:32], flat[40:41], torch.empty(0)], [outs[:16], outs[20:21]], None)
    clip._ranges = None
    for bad in (flat[:1], flat[31:32], flat[40:41], outs[14:16].view(torch.float32), outs[20:22].view(torch.float32)):
        with pytest.raises(ValueError, match="apart from"):
            clip._norm_address(bad)
    for good in (flat[32:33], flat[39:40], flat[41:42], torch.zeros(1)):
        assert clip._norm_address(good) == good.data_ptr()


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
