"""Trains a small encoder with K-FAC: attention with a learned relative
position bias, linear layers that keep their inputs in 8 bits, and the
preconditioner.  Synthetic task: every token answers which half of the
vocabulary the token before it is from, which attention solves through the
position bias.

    python examples/train_encoder.py [--steps 60] [--layers 2] [--width 128]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from linear_algebra_amd import kfac_position_borders  # noqa: E402
from linear_algebra_amd.kfac_preconditioner import KFACPreconditioner  # noqa: E402
from linear_algebra_amd.training import CheckpointLinear, attention  # noqa: E402


class EncoderLayer(torch.nn.Module):
    def __init__(self, width, heads, borders):
        super().__init__()
        self.heads, self.borders = heads, borders
        self.norm1, self.norm2 = torch.nn.LayerNorm(width), torch.nn.LayerNorm(width)
        self.qkv, self.out = CheckpointLinear(width, 3 * width), CheckpointLinear(width, width)
        self.up, self.down = CheckpointLinear(width, 4 * width), CheckpointLinear(4 * width, width)
        # every head starts out looking at a distance of its own
        bias = torch.zeros(2 * (len(borders) + 1), heads)
        bias[torch.arange(heads) % bias.shape[0], torch.arange(heads)] = 4.0
        self.bias = torch.nn.Parameter(bias)

    def forward(self, x, lens):
        b, n, width = x.shape
        qkv = self.qkv(self.norm1(x)).view(b, n, 3, self.heads, width // self.heads)
        y = attention(qkv[:, :, 0], qkv[:, :, 1], qkv[:, :, 2], lens=lens, bias=self.bias, borders=self.borders)
        x = x + self.out(y.reshape(b, n, width))
        return x + self.down(torch.relu(self.up(self.norm2(x))))


class Encoder(torch.nn.Module):
    def __init__(self, width=128, heads=4, layers=2, vocabulary=32):
        super().__init__()
        borders = kfac_position_borders(8, 64)
        self.embed = torch.nn.Embedding(vocabulary, width)
        self.layers = torch.nn.ModuleList(EncoderLayer(width, heads, borders) for _ in range(layers))
        self.norm, self.head = torch.nn.LayerNorm(width), CheckpointLinear(width, 2)

    def forward(self, tokens, lens):
        x = self.embed(tokens)
        for layer in self.layers:
            x = layer(x, lens)
        return self.head(self.norm(x))


def batch_of(generator, batch=32, length=48, vocabulary=32):
    """Tokens, sequence lengths, which half of the vocabulary the token before
    each one is from, and the places that have an answer."""
    tokens = torch.randint(0, vocabulary, (batch, length), generator=generator)
    lens = torch.randint(length // 2, length + 1, (batch,), generator=generator)
    answer = (tokens.roll(1, dims=1) < vocabulary // 2).long()
    place = torch.arange(length)
    return tokens, lens.int(), answer, (place >= 1) & (place < lens[:, None])


def train(steps=60, width=128, layers=2, lr=0.3, seed=0, device="cuda:0", say=print):
    torch.manual_seed(seed)
    g = torch.Generator().manual_seed(seed)
    model = Encoder(width=width, layers=layers).to(device)
    pre = KFACPreconditioner(model, damping=1e-2, inv_update_freq=5)
    opt = torch.optim.SGD(model.parameters(), lr=lr)
    losses = []
    for step in range(steps):
        tokens, lens, answer, real = (t.to(device) for t in batch_of(g))
        loss = torch.nn.functional.cross_entropy(model(tokens, lens)[real], answer[real])
        opt.zero_grad()
        loss.backward()
        pre.step()
        torch.nn.utils.clip_grad_norm_(model.parameters(), 1.0)
        opt.step()
        losses.append(float(loss.detach()))
        if step % 10 == 0:
            say(f"step {step:4d}  loss {losses[-1]:.4f}")
    pre.remove()
    return losses


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--layers", type=int, default=2)
    ap.add_argument("--width", type=int, default=128)
    a = ap.parse_args()
    losses = train(a.steps, a.width, a.layers)
    print(f"last loss {losses[-1]:.4f}")


if __name__ == "__main__":
    main()
