"""Global gradient norm and clipping on the GPU against the 64-bit formula."""
import math

import pytest
import torch

import operator_ref as ref
import ring_all_reduce_scatter_amd as rar
from operator_ref import DTYPES, U, assert_within

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def _ws(grads):
    return torch.empty(rar.grad_clip_workspace_bytes([g.numel() for g in grads]), dtype=torch.uint8, device=DEV)


def _grads(sizes, dts, seed, spread=1.0):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    return [(torch.randn(n, generator=gen, device=DEV) * spread).to(DTYPES[d]) for n, d in zip(sizes, dts)]


def _norm(grads, kind=0, scale=1.0):
    out = torch.full((1,), -7.0, device=DEV)
    rar.grad_norm(grads, _ws(grads), out, norm_type=kind, scale=scale)
    return out


def _check_norm(got, want, what):
    # one rounding to binary32 (the binary64 sum is off by far less)
    assert_within(got, torch.tensor([want], dtype=torch.float64),
                  torch.tensor(abs(want) * U * (1 + 2.0 ** -20) + 2.0 ** -150), what)


def _check_clip(grads, outs, norm, kind, scale, max_norm, what):
    want = ref.norm(grads, kind, scale)
    _check_norm(norm, want, what)
    for t, (g, o) in enumerate(zip(grads, outs)):
        r, tol = ref.clipped(g, want, max_norm, scale, o.dtype)
        assert_within(o, r, tol, f"{what} tensor {t}")


SETS = {
    "one": [1],
    "tail": [7, 0, 8, 9, 1, 0, 255],
    "tiles": [8192, 8191, 8193, 16384 + 5, 3],
    "many": [37 * (i % 50) + 1 for i in range(700)],
    "large": [3_000_017, 1_000_000, 65_537],
}


@pytest.mark.parametrize("kind", [rar.NORM_L2, rar.NORM_MAX])
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16", "mix"])
@pytest.mark.parametrize("name", sorted(SETS))
def test_norm_and_clip_match_formula(name, dt, kind):
    sizes = SETS[name]
    dts = [("f32", "bf16", "f16")[i % 3] if dt == "mix" else dt for i in range(len(sizes))]
    grads = _grads(sizes, dts, seed=len(name))
    scale = 1.0 / 3.0
    want = ref.norm(grads, kind, scale)
    _check_norm(_norm(grads, kind, scale), want, f"{name} norm")
    for max_norm in (want / 2, want * 2):
        ws, norm = _ws(grads), torch.zeros(1, device=DEV)
        for out in ("same", "f32", "bf16"):
            outs = [torch.full_like(g, 3.0, dtype=g.dtype if out == "same" else DTYPES[out]) for g in grads]
            keep = [g.clone() for g in grads]
            rar.clip_grad_norm(grads, max_norm, ws, norm, outs=outs, norm_type=kind, scale=scale)
            _check_clip(grads, outs, norm, kind, scale, max_norm, f"{name} {out} {max_norm}")
            assert all(torch.equal(a, b) for a, b in zip(keep, grads)), "inputs changed"
        again = [torch.empty_like(g) for g in grads]
        rar.clip_grad_norm(grads, max_norm, ws, norm, outs=again, norm_type=kind, scale=scale)
        rar.clip_grad_norm(grads, max_norm, ws, norm, norm_type=kind, scale=scale)  # in place
        assert all(torch.equal(a, b) for a, b in zip(again, grads)), "in place differs"
        for g, k in zip(grads, keep):
            g.copy_(k)


def test_empty_set():
    for grads in ([], [torch.empty(0, device=DEV), torch.empty(0, dtype=torch.float16, device=DEV)]):
        assert _norm(grads).item() == 0.0
        norm = torch.full((1,), 5.0, device=DEV)
        rar.clip_grad_norm(grads, 1.0, _ws(grads), norm)
        assert norm.item() == 0.0


def test_zero_gradients_stay_zero():
    grads = [torch.zeros(1000, device=DEV), torch.zeros(5000, dtype=torch.bfloat16, device=DEV)]
    norm = torch.ones(1, device=DEV)
    rar.clip_grad_norm(grads, 0.0, _ws(grads), norm)
    assert norm.item() == 0.0 and all(int((g != 0).sum()) == 0 for g in grads)


@pytest.mark.parametrize("mag", [1e30, 1e-30, 1e-42])
def test_norm_neither_overflows_nor_vanishes(mag):
    grads = [torch.full((4097,), mag, device=DEV)]
    got = _norm(grads)
    want = float(grads[0][0].double()) * math.sqrt(4097)
    _check_norm(got, want, f"{mag}")


@pytest.mark.parametrize("kind", [rar.NORM_L2, rar.NORM_MAX])
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_non_finite_gradients(bad, dt, kind):
    grads = _grads([100, 20_001, 5], [dt] * 3, seed=1)
    grads[1][20_000] = bad
    if math.isinf(bad):
        grads[2][0] = -bad
    outs = [torch.empty_like(g) for g in grads]
    norm = torch.zeros(1, device=DEV)
    rar.clip_grad_norm(grads, 1.0, _ws(grads), norm, outs=outs, norm_type=kind)
    if math.isnan(bad):
        assert math.isnan(norm.item()) and all(bool(o.isnan().all()) for o in outs)
    else:
        assert norm.item() == math.inf
        assert bool((outs[0] == 0).all()) and bool(outs[1][20_000].isnan()) and bool((outs[1][:20_000] == 0).all())


def test_scale_and_unlimited_max_norm():
    grads = _grads([5000], ["f32"], seed=2)
    for scale in (0.0, -0.5, 4.0):
        outs, norm = [torch.empty_like(grads[0])], torch.zeros(1, device=DEV)
        rar.clip_grad_norm(grads, math.inf, _ws(grads), norm, outs=outs, scale=scale)
        _check_norm(norm, ref.norm(grads, 0, scale), f"scale {scale}")
        assert torch.equal(outs[0], grads[0] * scale)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_unaligned_views_and_dense_permutations(dt):
    flat = torch.randn(70_000, device=DEV).to(DTYPES[dt])
    offs = [1, 1000, 9999, 30_001, 59_999]
    grads = [flat[a:b - 3] for a, b in zip(offs, offs[1:])]
    out = torch.full((80_000,), 9.0, device=DEV).to(DTYPES[dt])
    outs = [out[a + 1:a + 1 + g.numel()] for a, g in zip(offs, grads)]
    norm = torch.zeros(1, device=DEV)
    rar.clip_grad_norm(grads, 1.0, _ws(grads), norm, outs=outs)
    _check_clip(grads, outs, norm, 0, 1.0, 1.0, "views")
    touched = torch.zeros(80_000, dtype=torch.bool, device=DEV)
    for a, g in zip(offs, grads):
        touched[a + 1:a + 1 + g.numel()] = True
    assert bool((out[~touched] == 9.0).all()), "written outside the outputs"
    m = torch.randn(33, 65, 7, device=DEV).to(DTYPES[dt])
    perm = [m.permute(2, 0, 1), m.transpose(0, 1)[3:5].contiguous().transpose(0, 1)]
    want = [p.clone() for p in perm]
    rar.clip_grad_norm(perm, 1.0, _ws(perm), norm)
    _check_clip(want, perm, norm, 0, 1.0, 1.0, "permuted")


def test_same_bits_every_time_and_on_another_stream():
    grads = _grads([100_003, 77, 2_000_000], ["bf16", "f32", "bf16"], seed=5)
    ws, norm = _ws(grads), torch.zeros(1, device=DEV)
    outs = [torch.empty_like(g) for g in grads]
    clip = rar.GradClip(grads, ws, outs=outs)
    clip.clip(0.5, norm)
    first, n0 = [o.clone() for o in outs], norm.clone()
    side = torch.cuda.Stream()
    for k in range(6):
        for o in outs:
            o.zero_()
        if k % 2:
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                clip.clip(0.5, norm)
            torch.cuda.current_stream().wait_stream(side)
        else:
            clip.clip(0.5, norm, stream=torch.cuda.current_stream())
        assert torch.equal(norm, n0) and all(torch.equal(a, b) for a, b in zip(first, outs))


def test_norm_then_clip_of_one_plan_interleave():
    grads = _grads([50_000, 3], ["f32", "f16"], seed=6)
    keep = [g.clone() for g in grads]
    clip = rar.GradClip(grads, _ws(grads))
    a, c = torch.zeros(1, device=DEV), torch.zeros(1, device=DEV)
    clip.norm(a)
    clip.norm(c, norm_type=rar.NORM_MAX)
    _check_norm(a, ref.norm(keep, 0, 1.0), "l2")
    _check_norm(c, ref.norm(keep, 1, 1.0), "max")
    clip.clip(2.0, a, scale=0.25)
    _check_clip(keep, grads, a, 0, 0.25, 2.0, "clip")
    # afterwards the set's norm is at most max_norm, up to the outputs' roundings
    clip.norm(a)
    assert a.item() <= 2.0 * (1 + 2.0 ** -10)


def test_set_beyond_32_bit_offsets():
    """One tensor of more than 2^31 elements; its last elements count."""
    n = (1 << 31) + 12_345
    g = torch.zeros(n, dtype=torch.float16, device=DEV)
    g[0], g[1 << 31], g[n - 1] = 2.0, 3.0, 6.0
    norm = torch.zeros(1, device=DEV)
    rar.clip_grad_norm([g], 3.5, _ws([g]), norm)
    assert norm.item() == 7.0
    # f = 3.5 / (7 + 1e-6), a relative 2^-22.7 below one half: half precision rounds it away
    assert [g[0].item(), g[1 << 31].item(), g[n - 1].item()] == [1.0, 1.5, 3.0]
    assert int((g != 0).sum()) == 3


def test_replays_in_a_graph():
    grads = _grads([300_000, 1001], ["bf16", "f32"], seed=8)
    outs = [torch.empty_like(g) for g in grads]
    ws, norm = _ws(grads), torch.zeros(1, device=DEV)
    clip = rar.GradClip(grads, ws, outs=outs)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        clip.clip(0.7, norm, scale=0.5)
    for k in range(4):
        for x in grads:
            x.mul_(0.5 + k)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        got, n = [o.clone() for o in outs], norm.clone()
        clip.clip(0.7, norm, scale=0.5)
        assert torch.equal(n, norm) and all(torch.equal(a, b) for a, b in zip(got, outs)), f"replay {k}"
