"""The example's training step: its gradients against binary64 autograd on
the whole batch, and a loss that falls."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location("gradient_step", os.path.join(ROOT, "examples", "gradient_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _autograd(t, ids, targets):
    """Mean loss and mean gradients over the ranks, on the CPU in binary64."""
    ws = [w.double().cpu().requires_grad_() for w in t.weights]
    table, w, b, proj = ws
    total = 0.0
    for r in range(t.ranks):
        i, y = ids[r].cpu(), targets[r].cpu()
        # the padding row is used, but receives no gradient
        x = torch.where((i == t.padding)[:, None], table.detach()[i], table[i]) * t._scale
        mu = x.mean(1, keepdim=True)
        h = (x - mu) / torch.sqrt((x - mu).square().mean(1, keepdim=True) + 1e-5) * w + b
        logp = torch.log_softmax(h @ proj.t(), 1)
        total = total - (logp[torch.arange(i.numel()), y] * (i != t.padding)).sum() / t.tokens
    loss = total / t.ranks
    loss.backward()
    return loss.item(), [p.grad for p in ws]


@pytest.mark.parametrize("ranks", [1, 4])
def test_gradients_match_autograd(ranks):
    t = _example().Trainer(ranks=ranks, vocab=300, dim=70, tokens=129)
    ids, targets = t.batch(5)
    loss = t.gradients(ids, targets)
    want, grads = _autograd(t, ids, targets)
    # binary32 products over at most 300 terms, sums over 129 tokens and the
    # norms' own bounds: every step is off by less than 2^-24 times a few
    # hundred terms, and each gradient by less than 2^-12 of the largest
    assert abs(loss.item() - want) < 2.0 ** -16 * want
    norm = sum(g.square().sum() for g in grads).sqrt().item()
    assert abs(t.norm.item() - norm) < 2.0 ** -12 * norm
    factor = min(1.0, t.max_norm / (norm + 1e-6))
    for u, g in zip(t.updates, grads):
        assert (u.double().cpu() - g * factor).abs().max() <= 2.0 ** -12 * (g * factor).abs().max()
    for r in range(1, ranks):  # reduced gradients are the same on every rank
        assert all(torch.equal(a, b) for a, b in zip(t.grads[0], t.grads[r]))


def test_loss_falls():
    t = _example().Trainer(vocab=200)
    first = t.step(*t.batch(0)).item()
    for k in range(1, 40):
        last = t.step(*t.batch(k)).item()
    assert last < 0.5 * first, (first, last)
