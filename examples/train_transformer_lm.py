"""Trains a small transformer on packed texts of different lengths.

Blocks x += attention(norm(x)) w_out, x += ffn(norm(x)); queries and keys are normalised
per head and turned by their positions, keys and values are shared by groups of query
heads, and a batch is a row of texts packed one behind the other.  Everything but the
attention's two projections (torch products) comes from the library's operators, every
gradient goes into its optimizer steps: Muon for the matrices, AdamW for the rest.  In the
data each token repeats the one before the last with probability 0.9, which only
attention can see.

    python examples/train_transformer_lm.py [--steps N] [--dtype bf16|fp32]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import matrix_orthogonalising_optimizer_gb300 as dm  # noqa: E402


class Model:
    def __init__(self, vocab, dim, hidden, heads, kv_heads, layers, tokens, sequences, dtype, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, std):
            return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)

        def const(value, *shape):
            return torch.full(shape, value, dtype=dtype, device="cuda")

        self.heads, self.kv, self.head_dim, self.sequences = heads, kv_heads, dim // heads, sequences
        d = self.head_dim
        # per block: the attention's matrices, its head norms, the feed-forward block, two norms
        self.blocks = [{
            "w_qkv": normal((heads + 2 * kv_heads) * d, dim, std=dim ** -0.5), "w_out": normal(dim, dim, std=dim ** -0.5),
            "w_gate": normal(hidden, dim, std=dim ** -0.5), "w_up": normal(hidden, dim, std=dim ** -0.5),
            "w_down": normal(dim, hidden, std=hidden ** -0.5), "q_norm": const(1.0, d), "k_norm": const(1.0, d),
            "norm1": const(1.0, dim), "norm2": const(1.0, dim)} for _ in range(layers)]
        self.top = {"embed": normal(vocab, dim, std=1.0), "head": normal(vocab, dim, std=dim ** -0.5),
                    "norm": const(1.0, dim)}
        self.table = dm.rotary_table(tokens, d)
        self.matrices = [b[k] for b in self.blocks for k in ("w_qkv", "w_out", "w_gate", "w_up", "w_down")]
        self.momenta = [torch.zeros_like(w) for w in self.matrices]
        name = "bf16" if dtype == torch.bfloat16 else "fp32"
        self.muon = dm.Muon([(*w.shape, name) for w in self.matrices]).bind()
        self.others = [b[k] for b in self.blocks for k in ("q_norm", "k_norm", "norm1", "norm2")] + list(self.top.values())
        self.avg = [torch.zeros_like(w) for w in self.others]
        self.sq = [torch.zeros_like(w) for w in self.others]
        need = max(dm.gated_ffn_workspace(tokens, dim, hidden, dtype, backward=True),
                   dm.vocab_loss_workspace(tokens, dim, vocab, dtype, grad=True),
                   dm.layer_norm_workspace(tokens, dim, dtype),
                   dm.qk_norm_rotary_workspace(tokens, heads, kv_heads, d, dtype),
                   dm.attention_workspace(tokens, heads, kv_heads, d, dtype, sequences=sequences, backward=True))
        self.space = torch.empty(need, dtype=torch.uint8, device="cuda")
        self.steps = 0

    def gradients(self, tokens, targets, offsets, positions):
        """The mean loss and the gradients, as the parameters are held: (loss, blocks, top)."""
        ws, h, kv, d = self.space, self.heads, self.kv, self.head_dim
        n = tokens.shape[0]
        x = self.top["embed"][tokens]
        kept = []
        for b in self.blocks:
            n1, m1, r1 = dm.layer_norm(x, b["norm1"])
            q, k, v = (n1 @ b["w_qkv"].T).split([h * d, kv * d, kv * d], 1)
            q, k, v = q.view(n, h, d), k.view(n, kv, d), v.view(n, kv, d)
            qr, kr = dm.qk_norm_rotary(q, k, positions, self.table, b["q_norm"], b["k_norm"])
            o, lse = dm.attention(qr, kr, v, offsets, workspace=ws)
            y = x + o.flatten(1) @ b["w_out"].T
            n2, m2, r2 = dm.layer_norm(y, b["norm2"])
            f, saved, inner = dm.gated_ffn(n2, b["w_gate"], b["w_up"], b["w_down"], save=True, workspace=ws)
            kept.append((x, n1, m1, r1, q, k, v, qr, kr, o, lse, y, n2, m2, r2, saved, inner))
            x = y + f
        z, m, r = dm.layer_norm(x, self.top["norm"])
        coef = torch.full(targets.shape, 1.0 / n, device="cuda")
        loss, _, dz, dhead = dm.vocab_loss_grad(z, self.top["head"], targets, coef=coef, workspace=ws)
        dx, dnorm, _ = dm.layer_norm_backward(dz, x, self.top["norm"], m, r, workspace=ws)
        grads = []
        for b, (x, n1, m1, r1, q, k, v, qr, kr, o, lse, y, n2, m2, r2, saved, inner) in zip(self.blocks[::-1], kept[::-1]):
            g = {}
            dn, g["w_gate"], g["w_up"], g["w_down"] = dm.gated_ffn_backward(
                dx, n2, b["w_gate"], b["w_up"], b["w_down"], saved, inner, workspace=ws)
            dy, g["norm2"], _ = dm.layer_norm_backward(dn, y, b["norm2"], m2, r2, workspace=ws)
            dy = dy + dx
            g["w_out"] = dy.T @ o.flatten(1)
            do = (dy @ b["w_out"]).view(n, h, d)
            dqr, dkr, dv = dm.attention_backward(do, qr, kr, v, o, lse, offsets, workspace=ws)
            dq, dk, g["q_norm"], g["k_norm"] = dm.qk_norm_rotary_backward(dqr, dkr, q, k, positions, self.table,
                                                                          b["q_norm"], b["k_norm"], workspace=ws)
            dqkv = torch.cat([dq.flatten(1), dk.flatten(1), dv.flatten(1)], 1)
            g["w_qkv"] = dqkv.T @ n1
            dres, g["norm1"], _ = dm.layer_norm_backward(dqkv @ b["w_qkv"], x, b["norm1"], m1, r1, workspace=ws)
            dx = dy + dres
            grads.insert(0, g)
        dembed = torch.zeros_like(self.top["embed"], dtype=torch.float32).index_add_(0, tokens, dx.float())
        return loss.mean(), grads, {"embed": dembed.to(dx.dtype), "head": dhead, "norm": dnorm}

    def step(self, tokens, targets, offsets, positions, lr_muon=0.02, lr_adam=3e-3):
        loss, blocks, top = self.gradients(tokens, targets, offsets, positions)
        self.steps += 1
        self.muon.step(self.matrices, [g[k].contiguous() for g in blocks for k in
                                       ("w_qkv", "w_out", "w_gate", "w_up", "w_down")], self.momenta, lr=lr_muon,
                       beta=0.95, wd=0.0)
        dm.adamw_step(self.others, [g[k] for g in blocks for k in ("q_norm", "k_norm", "norm1", "norm2")]
                      + [top[k] for k in self.top], self.avg, self.sq, lr=lr_adam, beta1=0.9, beta2=0.95, eps=1e-8, wd=0.0,
                      step=self.steps)
        return loss


def batch(g, vocab, tokens, sequences):
    """Tokens, targets, offsets and positions of `sequences` texts of random lengths."""
    cuts = torch.randperm(tokens - 1, generator=g, device="cuda")[:sequences - 1].sort().values + 1
    edge = torch.tensor([0], device="cuda"), torch.tensor([tokens], device="cuda")
    offsets = torch.cat([edge[0], cuts, edge[1]])
    at = torch.arange(tokens + 1, device="cuda")
    text = torch.randint(0, vocab, (tokens + 1,), generator=g, device="cuda")
    # token i repeats token i - 2 with probability 0.9; where several in a row do, the first counts
    keep = torch.rand(tokens + 1, generator=g, device="cuda") < 0.9
    keep[:2] = False
    for parity in (0, 1):
        start = torch.where(keep[parity::2], 0, at[parity::2]).cummax(0).values
        text[parity::2] = text[start]
    start = offsets[torch.searchsorted(offsets, at[:-1], right=True) - 1]
    return text[:-1].contiguous(), text[1:].contiguous(), offsets, at[:-1] - start


def train(steps=100, vocab=500, dim=256, hidden=768, heads=4, kv_heads=2, layers=2, tokens=2048, sequences=9,
          dtype=torch.bfloat16, seed=0):
    """The mean losses of the steps, as a list."""
    model = Model(vocab, dim, hidden, heads, kv_heads, layers, tokens, sequences, dtype, seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    losses = [model.step(*batch(g, vocab, tokens, sequences)) for _ in range(steps)]
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
