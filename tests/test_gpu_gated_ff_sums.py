"""How far long sums of the gated feed-forward block in binary32 are off.

Of n terms of one size and any sign, the i-th partial sum is sqrt(i) times as
large, and each addition rounds it by at most u = 2^-24 of it, one way or the
other.  Chains of 512 terms and a chain of their sums are then off by u
sqrt(512 / 2 + n / 1024) of the result, in the root of the mean square over
many results; a single chain is off by u sqrt(n / 2).  The products' roundings
add 1 under the root, and 100 what dg and du are off by themselves, ten
roundings at most.
"""
import math

import pytest
import torch

import block_ref
import ring_all_reduce_scatter_amd as rar

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24


def _off(got, want):
    return float((got.double() - want).norm() / want.norm()) / U


def _bound(n, operands=0):
    return math.sqrt(256 + n / 1024 + 1 + operands)


# sums of 4096 (forward), 16,384 (dx) and 8192 terms (the weights' gradients)
# that no split shortens, and of few and odd numbers
@pytest.mark.parametrize("first", [0, 1])
@pytest.mark.parametrize("rows,dim,hidden", [(1024, 4096, 8192), (8192, 2048, 1024), (70, 8191, 300), (600, 513, 1025),
                                             (129, 33, 700)])
def test_sums_in_binary32(rows, dim, hidden, first):
    g = torch.Generator(device=DEV).manual_seed(rows + dim + hidden)
    rand = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    room = torch.empty(rows * dim + 8, device=DEV)  # from element `first` on: rows on and off 16 bytes
    x = room[first:first + rows * dim].view(rows, dim).copy_(rand(rows, dim))
    wg, wu, dh = rand(hidden, dim) * dim ** -0.5, rand(hidden, dim) * dim ** -0.5, rand(rows, hidden)
    out, gate, up = (torch.empty(rows, hidden, device=DEV) for _ in range(3))
    rar.gated_ff_forward(x, wg, wu, out, gate=gate, up=up)
    for got, w in ((gate, wg), (up, wu)):
        assert _off(got, x.double() @ w.double().t()) <= _bound(dim)
    dx, dwg, dwu = torch.empty(rows, dim, device=DEV), torch.empty_like(wg), torch.empty_like(wu)
    ws = torch.empty(rar.gated_ff_workspace_bytes(rows, dim, hidden, torch.float32), dtype=torch.uint8, device=DEV)
    rar.gated_ff_backward(dh, x, wg, wu, gate, up, dx, dwg, dwu, ws)
    a, d = block_ref.act(gate.double(), rar.ACT_SILU)
    dg, du = dh.double() * up.double() * d, dh.double() * a
    assert _off(dx, dg @ wg.double() + du @ wu.double()) <= _bound(2 * hidden, 100)
    assert _off(dwg, dg.t() @ x.double()) <= _bound(rows, 100)
    assert _off(dwu, du.t() @ x.double()) <= _bound(rows, 100)
