"""The operators of a block one after the other, as a training step runs them:
embedding, layer norm that keeps its input in 8 bits, the feed-forward block
that keeps its projections in 8 bits, and back to the table's gradient."""
import pytest
import torch

import block_ref
import ring_all_reduce_scatter_amd as rar

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def test_gradients_of_a_run():
    """Against binary64 on the kept values, without the steps' roundings: each
    of binary32's is 2^-24 of sums of at most 300 terms, five operators deep,
    so 2^-11 of the largest gradient covers them."""
    tokens, vocab, dim, hidden = 150, 60, 72, 200
    gen = torch.Generator(device=DEV).manual_seed(3)
    rand = lambda *s: torch.randn(*s, generator=gen, device=DEV)  # noqa: E731
    table, w, b = rand(vocab, dim), 1 + 0.1 * rand(dim), 0.1 * rand(dim)
    wg, wu, dh = rand(hidden, dim) * dim ** -0.5, rand(hidden, dim) * dim ** -0.5, rand(tokens, hidden)
    ids = torch.randint(0, vocab, (tokens,), generator=gen, device=DEV)

    def new(*s, dtype=torch.float32):
        return torch.empty(s, dtype=dtype, device=DEV)

    def held(rows, cols):
        return new(rar.checkpoint_bytes(rows, cols), dtype=torch.uint8)

    x, y, h = new(tokens, dim), new(tokens, dim), new(tokens, hidden)
    mean, rstd = new(tokens), new(tokens)
    kx, kg, ku = held(tokens, dim), held(tokens, hidden), held(tokens, hidden)
    rar.embedding_forward(table, ids, x)
    rar.layernorm_forward_checkpoint(x, w, b, y, kx, mean=mean, rstd=rstd)
    rar.gated_ff_forward(y, wg, wu, h, gate=kg, up=ku)

    dy, dwg, dwu = new(tokens, dim), new(hidden, dim), new(hidden, dim)
    dx, dw, db, dtable = new(tokens, dim), new(dim), new(dim), new(vocab, dim)
    ws = new(rar.gated_ff_workspace_bytes(tokens, dim, hidden, torch.float32), dtype=torch.uint8)
    rar.gated_ff_backward(dh, y, wg, wu, kg, ku, dy, dwg, dwu, ws)
    ws2 = new(rar.layernorm_workspace_bytes(tokens, dim), dtype=torch.uint8)
    rar.layernorm_backward_checkpoint(dy, kx, w, mean, rstd, dx, dw, db, ws2)
    ws3 = new(rar.embedding_workspace_bytes(tokens, vocab, dim), dtype=torch.uint8)
    rar.embedding_backward(dx, ids, dtable, ws3)

    t64, w64, b64, wg64, wu64 = (t.double() for t in (table, w, b, wg, wu))
    x64 = t64[ids]
    mu = x64.mean(1, keepdim=True)
    r = (x64.var(1, unbiased=False, keepdim=True) + 1e-5).rsqrt()
    y64 = (x64 - mu) * r * w64 + b64
    g, u = (torch.empty(tokens, hidden, device=DEV) for _ in range(2))
    rar.checkpoint_unpack(kg, g)
    rar.checkpoint_unpack(ku, u)
    # the kept projections are the projections, to a step of their blocks
    for k, p in ((g, y64 @ wg64.t()), (u, y64 @ wu64.t())):
        top = torch.nn.functional.pad(p.abs(), (0, -hidden % 32)).view(tokens, -1, 32).amax(2, keepdim=True)
        step = top.expand(-1, -1, 32).reshape(tokens, -1)[:, :hidden] * 2.0 ** -6
        assert bool(((k.double() - p).abs() <= step).all())
    a, d = block_ref.act(g.double(), 0)
    dg, du = dh.double() * u.double() * d, dh.double() * a
    dy64 = dg @ wg64 + du @ wu64
    hx = (block_ref.held(x)[2].to(DEV) - mu) * r
    gy = dy64 * w64
    dx64 = r * (gy - gy.mean(1, keepdim=True) - hx * (gy * hx).mean(1, keepdim=True))
    dt64 = torch.zeros(vocab, dim, dtype=torch.float64, device=DEV).index_add_(0, ids, dx64)
    want = {"dwgate": (dwg, dg.t() @ y64), "dwup": (dwu, du.t() @ y64), "dw": (dw, (dy64 * hx).sum(0)),
            "db": (db, dy64.sum(0)), "dx": (dx, dx64), "dtable": (dtable, dt64)}
    for name, (got, ref) in want.items():
        assert float((got.double() - ref).abs().max()) <= 2.0 ** -11 * float(ref.abs().max()), name
    a64 = block_ref.act(y64 @ wg64.t(), 0)[0] * (y64 @ wu64.t())
    assert float((h.double() - a64).abs().max()) <= 2.0 ** -11 * float(a64.abs().max())
