"""Trains a small residual language model with the library alone.

The model predicts the next token from the current one: an embedding, residual
blocks x += ffn(norm(x)), a final norm and the vocabulary loss.  Every gradient
comes from the library's operators and goes straight into its optimizer steps:
Muon for the gate, up and down matrices, AdamW for the embedding, the vocabulary
matrix and the norms.  The data is a random token map followed with probability
0.9, so the loss can fall from log(vocab) to about 1.

    python examples/train_residual_lm.py [--steps N] [--dtype bf16|fp32]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import matrix_orthogonalising_optimizer_gb300 as dm  # noqa: E402


class Model:
    def __init__(self, vocab, dim, hidden, layers, tokens, dtype, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, std):
            return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)

        def const(value, *shape):
            return torch.full(shape, value, dtype=dtype, device="cuda")

        name = "bf16" if dtype == torch.bfloat16 else "fp32"
        self.embed = normal(vocab, dim, std=1.0)
        self.head = normal(vocab, dim, std=dim ** -0.5)
        self.norms = [(const(1.0, dim), const(0.0, dim)) for _ in range(layers + 1)]
        self.ffns = [(normal(hidden, dim, std=dim ** -0.5), normal(hidden, dim, std=dim ** -0.5),
                      normal(dim, hidden, std=hidden ** -0.5)) for _ in range(layers)]
        # the optimizers: one Muon plan over all block matrices, AdamW on the rest
        self.matrices = [w for block in self.ffns for w in block]
        self.momenta = [torch.zeros_like(w) for w in self.matrices]
        self.muon = dm.Muon([(*w.shape, name) for w in self.matrices]).bind()
        self.others = [self.embed, self.head, *(t for pair in self.norms for t in pair)]
        self.avg = [torch.zeros_like(w) for w in self.others]
        self.sq = [torch.zeros_like(w) for w in self.others]
        # one workspace serves every operator of the step, one after the other
        need = max(dm.gated_ffn_workspace(tokens, dim, hidden, dtype, backward=True),
                   dm.vocab_loss_workspace(tokens, dim, vocab, dtype, grad=True),
                   dm.layer_norm_workspace(tokens, dim, dtype))
        self.space = torch.empty(need, dtype=torch.uint8, device="cuda")
        self.steps = 0

    def step(self, tokens, targets, lr_muon=0.02, lr_adam=3e-3):
        """One training step; the mean loss before it, as a device tensor."""
        ws = self.space
        x = self.embed[tokens]
        kept = []
        for (w, b), block in zip(self.norms, self.ffns):
            n, mean, rstd = dm.layer_norm(x, w, b)
            y, saved, h = dm.gated_ffn(n, *block, save=True, workspace=ws)
            kept.append((x, n, mean, rstd, saved, h))
            x = x + y
        w, b = self.norms[-1]
        n, mean, rstd = dm.layer_norm(x, w, b)
        coef = torch.full(targets.shape, 1.0 / targets.numel(), device="cuda")
        loss, _, dn, dhead = dm.vocab_loss_grad(n, self.head, targets, coef=coef, workspace=ws)
        dx, dw, db = dm.layer_norm_backward(dn, x, w, mean, rstd, workspace=ws)
        dnorms, dmatrices = [(dw, db)], []
        for (w, _), block, (x, n, mean, rstd, saved, h) in zip(self.norms[-2::-1], self.ffns[::-1], kept[::-1]):
            dn, *dblock = dm.gated_ffn_backward(dx, n, *block, saved, h, workspace=ws)
            dres, dw, db = dm.layer_norm_backward(dn, x, w, mean, rstd, workspace=ws)
            dx = dx + dres
            dnorms.insert(0, (dw, db))
            dmatrices = dblock + dmatrices
        dembed = torch.zeros_like(self.embed, dtype=torch.float32).index_add_(0, tokens, dx.float())
        dembed = dembed.to(self.embed.dtype)
        self.steps += 1
        self.muon.step(self.matrices, dmatrices, self.momenta, lr=lr_muon, beta=0.95, wd=0.0)
        dm.adamw_step(self.others, [dembed, dhead, *(t for pair in dnorms for t in pair)], self.avg, self.sq,
                      lr=lr_adam, beta1=0.9, beta2=0.95, eps=1e-8, wd=0.0, step=self.steps)
        return loss.mean()


def train(steps=100, vocab=1000, dim=256, hidden=768, layers=2, tokens=2048, dtype=torch.bfloat16, seed=0):
    """The mean losses of the steps, as a list."""
    model = Model(vocab, dim, hidden, layers, tokens, dtype, seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    follow = torch.randperm(vocab, generator=g, device="cuda")
    losses = []
    for _ in range(steps):
        cur = torch.randint(0, vocab, (tokens,), generator=g, device="cuda")
        noise = torch.randint(0, vocab, (tokens,), generator=g, device="cuda")
        keep = torch.rand(tokens, generator=g, device="cuda") < 0.9
        losses.append(model.step(cur, torch.where(keep, follow[cur], noise)))
    losses = [float(x) for x in losses]
    if dm.ops_status() != 0 or model.muon.device_status() != 0:
        raise RuntimeError("a device-side wait gave up")
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=100)
    ap.add_argument("--dtype", choices=("bf16", "fp32"), default="bf16")
    a = ap.parse_args()
    out = train(a.steps, dtype=torch.bfloat16 if a.dtype == "bf16" else torch.float32)
    for i in range(0, len(out), max(1, len(out) // 10)):
        print(f"step {i:4d}  loss {out[i]:.4f}")
    print(f"step {len(out) - 1:4d}  loss {out[-1]:.4f}")
