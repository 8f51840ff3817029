"""Data-parallel training steps of a small next-token model on N simulated
ranks, every gradient made, reduced and finished by the library.

    python examples/gradient_step.py [--ranks 4] [--steps 20]

Per rank: tokens -> embedding -> layer norm -> projection -> cross entropy,
and back: the layer norm's gradients (dx, dweight, dbias) and the embedding's
(by sorted tokens) are written straight into the rank's gradient tensors.
Then the ranks' gradients are summed by the bucketed ring all-reduce, and the
mean's global norm is taken and clipped into the optimizer's buffers.  The
projection and the loss are torch's.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import ring_all_reduce_scatter_amd as rar  # noqa: E402


class Trainer:
    """Weights, per-rank gradients and the plans of one training run."""

    def __init__(self, ranks=4, vocab=1000, dim=256, tokens=512, max_norm=0.5, lr=2.0, padding=0, device="cuda"):
        self.ranks, self.vocab, self.dim, self.tokens = ranks, vocab, dim, tokens
        self.max_norm, self.lr, self.padding = max_norm, lr, padding
        gen = torch.Generator(device=device).manual_seed(1)
        rand = lambda *s: torch.randn(*s, generator=gen, device=device)  # noqa: E731
        # table, norm weight, norm bias, projection
        self.weights = [rand(vocab, dim) * 0.1, torch.ones(dim, device=device), torch.zeros(dim, device=device),
                        rand(vocab, dim) * dim ** -0.5]
        shapes = [w.shape for w in self.weights]
        counts = [w.numel() for w in self.weights]
        # rank r's gradients, the ranks' copies placed for the fold
        self._arena, flat = rar.rank_tensors(ranks, counts, torch.float32, device)
        self.grads = [[g.view(s) for g, s in zip(row, shapes)] for row in flat]
        cap = 1 << 20
        self._bucket_ws = self._bytes(rar.bucketed_workspace_bytes(counts, ranks, rar.F32, cap), device)
        self._reduce = rar.BucketedAllreduce(self.grads, cap, self._bucket_ws)
        # the reduced gradients are the same on every rank: rank 0's are clipped
        self.updates = [torch.empty_like(w) for w in self.weights]
        self._clip_ws = self._bytes(rar.grad_clip_workspace_bytes(counts), device)
        self._clip = rar.GradClip(self.grads[0], self._clip_ws, outs=self.updates)
        self.norm = torch.zeros(1, device=device)
        # activations, reused by every rank
        self._x, self._h, self._dx = (torch.empty(tokens, dim, device=device) for _ in range(3))
        self._mean, self._rstd = torch.empty(tokens, device=device), torch.empty(tokens, device=device)
        self._ln_ws = self._bytes(rar.layernorm_workspace_bytes(tokens, dim), device)
        self._emb_ws = self._bytes(rar.embedding_workspace_bytes(tokens, vocab, dim), device)
        self._scale = dim ** 0.5

    @staticmethod
    def _bytes(n, device):
        return torch.empty(n, dtype=torch.uint8, device=device)

    def _rank_gradients(self, ids, targets, grads):
        """One rank's loss, and its gradients into `grads`."""
        table, w, b, proj = self.weights
        dtable, dw, db, dproj = grads
        rar.embedding_forward(table, ids, self._x, scale=self._scale)
        rar.layernorm_forward(self._x, w, b, self._h, mean=self._mean, rstd=self._rstd)
        logp = torch.log_softmax(self._h @ proj.t(), dim=1)
        used = (ids != self.padding).float() / self.tokens  # padded positions have no target
        loss = -(logp.gather(1, targets[:, None])[:, 0] * used).sum()
        dlogits = logp.exp()
        dlogits.scatter_add_(1, targets[:, None], torch.full_like(used, -1.0)[:, None])
        dlogits *= used[:, None]
        torch.mm(dlogits.t(), self._h, out=dproj)
        rar.layernorm_backward(dlogits @ proj, self._x, w, self._mean, self._rstd, self._dx, dw, db, self._ln_ws)
        rar.embedding_backward(self._dx, ids, dtable, self._emb_ws, scale=self._scale, padding_id=self.padding)
        return loss

    def gradients(self, ids, targets):
        """ids[r], targets[r]: rank r's tokens.  Returns the mean loss; the
        clipped mean gradient is in self.updates, its norm in self.norm."""
        losses = [self._rank_gradients(ids[r], targets[r], self.grads[r]) for r in range(self.ranks)]
        self._reduce()
        self._clip.clip(self.max_norm, self.norm, scale=1.0 / self.ranks)
        return torch.stack(losses).mean()

    def step(self, ids, targets):
        loss = self.gradients(ids, targets)
        for w, u in zip(self.weights, self.updates):
            w.add_(u, alpha=-self.lr)
        return loss

    def batch(self, seed):
        """Tokens that follow a fixed rule (next = 7 t + 3 mod the vocabulary),
        a few of them padding."""
        gen = torch.Generator().manual_seed(seed)
        ids = torch.randint(1, self.vocab, (self.ranks, self.tokens), generator=gen)
        ids[torch.rand(ids.shape, generator=gen) < 0.05] = self.padding
        dev = self.weights[0].device
        return ids.to(dev), ((7 * ids + 3) % self.vocab).to(dev)


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--ranks", type=int, default=4)
    ap.add_argument("--steps", type=int, default=20)
    args = ap.parse_args()
    t = Trainer(ranks=args.ranks)
    for k in range(args.steps):
        loss = t.step(*t.batch(k))
        print(f"step {k:3d}  loss {loss.item():.4f}  gradient norm {t.norm.item():.4f}", flush=True)


if __name__ == "__main__":
    main()
