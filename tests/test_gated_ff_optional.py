"""Outputs of rar_gated_ff_backward that a caller leaves out: what stands in
their strides does not count.  CPU only: a workspace that is too small ends
each call before a launch."""
import pytest

import ring_all_reduce_scatter_amd as rar

OK, EINVAL, EWORKSPACE = 0, 1, 4
G = 1 << 32
B = 1 << 40  # addresses that are never read


def _backward(dx=B + 6 * G, dxs=48, dg=B + 7 * G, dgs=48, du=B + 8 * G, dus=48, ws=0, n=0):
    return rar.lib().rar_gated_ff_backward(B, 80, B + G, 48, B + 2 * G, 48, B + 3 * G, 48, rar.KEEP_ROWS, B + 4 * G, 80,
                                           B + 5 * G, 80, 70, 48, 80, rar.BF16, rar.ACT_SILU, dx, dxs, dg, dgs, du, dus,
                                           rar.BF16, 0, ws, n, None)


@pytest.mark.parametrize("stride", [0, 1, 47, 48, 1 << 63])
def test_strides_of_outputs_left_out(stride):
    # past the strides' checks, up to the missing workspace
    assert _backward(dx=0, dxs=stride) == EWORKSPACE
    assert _backward(dg=0, du=0, dgs=stride, dus=stride) == EWORKSPACE
    assert _backward(dx=0, dg=0, du=0, dxs=stride, dgs=stride, dus=stride, ws=B + 9 * G, n=1 << 30) == OK


def test_strides_of_outputs_given():
    for name in ("dxs", "dgs", "dus"):
        assert _backward(**{name: 47}) == EINVAL and _backward(**{name: 1 << 63}) == EINVAL
    assert _backward(dg=0, dgs=0) == EINVAL and _backward(du=0, dus=0) == EINVAL  # both or none
