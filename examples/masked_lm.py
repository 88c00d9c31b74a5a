"""Trains a small masked language model whose contractions run through the
simulated multiplier (AMDense, AMAttention), with the exact operators between
and after them: BlockNorm around every block, VocabHead's loss over the
vocabulary (tokens that are not masked carry no target), and AdamW with 8-bit
moments.

    python examples/masked_lm.py [--steps 100] [--mantissa 7] [--kind mitchell]

The data is synthetic: each sequence repeats a short random phrase, so that a
masked token can be read off the sequence's other repeats."""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import approximate_multiplier_dnn_gb300 as am  # noqa: E402
from approximate_multiplier_dnn_gb300.layers import AMAttention, AMDense, BlockNorm, VocabHead  # noqa: E402
from approximate_multiplier_dnn_gb300.optim import AdamW  # noqa: E402

IGNORE = -100


class Attention(torch.nn.Module):
    def __init__(self, dim, heads, lut, gen):
        super().__init__()
        self.heads = heads
        self.q, self.k, self.v, self.o = (AMDense(dim, dim, lut, bias=False, generator=gen) for _ in range(4))
        self.attention = AMAttention(lut)

    def forward(self, n, batch, seq):
        def split(t):
            return t.view(batch, seq, self.heads, -1).transpose(1, 2).contiguous()
        out = self.attention(split(self.q(n)), split(self.k(n)), split(self.v(n)))
        return self.o(out.transpose(1, 2).reshape(batch * seq, -1))


class Mlp(torch.nn.Module):
    def __init__(self, dim, lut, gen):
        super().__init__()
        self.up, self.down = AMDense(dim, 4 * dim, lut, generator=gen), AMDense(4 * dim, dim, lut, generator=gen)

    def forward(self, n, batch, seq):
        return self.down(torch.nn.functional.gelu(self.up(n)))


class MaskedLm(torch.nn.Module):
    """Token and position embeddings, `layers` times attention and MLP, the
    vocabulary head.  The residual stream and the blocks are fp32; the last
    norm writes the bf16 that the head reads."""

    def __init__(self, vocab, dim, heads, layers, seq, lut, gen):
        super().__init__()
        self.tokens = torch.nn.Parameter((torch.randn((vocab + 1, dim), generator=gen) * 0.5).cuda())
        self.places = torch.nn.Parameter((torch.randn((seq, dim), generator=gen) * 0.5).cuda())
        blocks, norms = [], [BlockNorm(dim, post=False)]
        for i in range(layers):
            blocks += [Attention(dim, heads, lut, gen), Mlp(dim, lut, gen)]
            norms += [BlockNorm(dim, gate="channel", alpha=0.5),
                      BlockNorm(dim, gate="channel", alpha=0.5,
                                n_dtype=torch.bfloat16 if i == layers - 1 else None)]
        self.blocks, self.norms = torch.nn.ModuleList(blocks), torch.nn.ModuleList(norms)
        self.head = VocabHead(dim, vocab, ignore_index=IGNORE, generator=gen)

    def forward(self, ids, targets):
        batch, seq = ids.shape
        x = (self.tokens[ids] + self.places[:seq]).reshape(batch * seq, -1)
        x, n = self.norms[0](x)
        for block, norm in zip(self.blocks, list(self.norms)[1:]):
            x, n = norm(x, block(n, batch, seq))
        return self.head(n, targets)


def batch_of(vocab, batch, seq, gen, phrase=4):
    """Sequences of a repeated phrase, a seventh of their tokens masked (id `vocab`); targets at the masks only."""
    words = torch.randint(0, vocab, (batch, phrase), generator=gen)
    ids = words.repeat(1, -(-seq // phrase))[:, :seq]
    mask = torch.rand((batch, seq), generator=gen) < 1 / 7
    targets = torch.where(mask, ids, torch.full_like(ids, IGNORE))
    return torch.where(mask, torch.full_like(ids, vocab), ids).cuda(), targets.cuda()


def train(steps=60, kind="mitchell", mantissa=7, vocab=1000, dim=128, heads=4, layers=2, seq=64, batch=32, lr=1e-2,
          moment_bits=8, clip=1.0, seed=0, report=None):
    """Trains and returns the losses, one per step."""
    lut = am.Lut.build(kind, mantissa)
    gen = torch.Generator().manual_seed(seed)
    model = MaskedLm(vocab, dim, heads, layers, seq, lut, gen)
    vectors = [p for p in model.parameters() if p.dim() < 2 or p.shape[0] == 1]
    known = {id(p) for p in vectors}
    opt = AdamW([{"params": [p for p in model.parameters() if id(p) not in known]},
                 {"params": vectors, "weight_decay": 0.0}], lr=lr, moment_bits=moment_bits)
    losses = []
    for i in range(steps):
        ids, targets = batch_of(vocab, batch, seq, gen)
        loss = model(ids, targets)
        opt.zero_grad(set_to_none=False)
        loss.backward()
        norm = torch.stack([p.grad.float().square().sum() for p in model.parameters()]).sum().sqrt()
        opt.step(grad_scale=(clip / norm.clamp(min=clip)).reshape(1))
        losses.append(loss.detach())
        if report and (i % report == 0 or i == steps - 1):
            print(f"step {i}: loss {loss.item():.4f}, gradient norm {norm.item():.3f}", flush=True)
    return [float(x) for x in losses]


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=100)
    ap.add_argument("--kind", default="mitchell", choices=sorted(am.KINDS))
    ap.add_argument("--mantissa", type=int, default=7)
    ap.add_argument("--moment-bits", type=int, default=8, choices=(8, 32))
    ap.add_argument("--lr", type=float, default=3e-3)
    a = ap.parse_args()
    am.build()
    train(a.steps, a.kind, a.mantissa, moment_bits=a.moment_bits, lr=a.lr, report=10)
