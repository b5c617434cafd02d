"""Train a small language model with NVFP4 linear layers on a synthetic text: the
token embedding, FFN blocks on `NVFP4Linear`, the output head with its softmax
cross entropy, and gradient clipping, as they are used together; with --heads also
self-attention between an NVFP4 projection and another, over documents of --document tokens.

    python examples/train_lm.py [--steps 30] [--vocab 5000] [--hidden 256] [--tied] [--heads 4]

The text follows a fixed random successor of each word, three times out of four, so
the loss falls from log(vocab) towards about a quarter of it.  One line per step:
loss, gradient norm, milliseconds.
"""
import argparse
import math
import os
import sys
import time

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))

from bit_microscaled_numerics_amd.linear import NVFP4Linear, Seeds  # noqa: E402
from bit_microscaled_numerics_amd.lm import (CrossEntropyHead, ScaledEmbedding,  # noqa: E402
                                             SelfAttention, clip_grad_norm)


def norm(x: torch.Tensor) -> torch.Tensor:
    return torch.nn.functional.rms_norm(x.float(), x.shape[-1:]).to(torch.bfloat16)


class Attention(torch.nn.Module):
    """Queries, keys and values from one NVFP4 projection; half as many key heads."""

    def __init__(self, hidden: int, heads: int, document: int, seed: int, device):
        super().__init__()
        dim, kv_heads = hidden // heads, max(1, heads // 2)
        self.document = document
        self.qkv = NVFP4Linear(hidden, (heads + 2 * kv_heads) * dim, Seeds(rht=seed, sr=seed), device=device)
        self.mix = SelfAttention(heads, dim, kv_heads, device=device)
        self.out = NVFP4Linear(hidden, hidden, Seeds(rht=seed + 1, sr=seed + 1000), device=device)

    def forward(self, x):
        tokens = x.shape[0]
        starts = torch.arange(0, tokens, self.document, device=x.device)
        cu = torch.cat((starts, starts.new_full((1,), tokens))).to(torch.int32)
        y = self.mix(self.qkv(norm(x)).to(torch.bfloat16), cu=cu)
        return x + self.out(y).to(torch.bfloat16)


class Block(torch.nn.Module):
    def __init__(self, hidden: int, ffn: int, seed: int, device):
        super().__init__()
        self.up = NVFP4Linear(hidden, ffn, Seeds(rht=seed, sr=seed), device=device)
        self.down = NVFP4Linear(ffn, hidden, Seeds(rht=seed + 1, sr=seed + 1000), device=device)

    def forward(self, x):
        y = torch.relu(self.up(norm(x))).to(torch.bfloat16)
        return x + self.down(y).to(torch.bfloat16)


class Model(torch.nn.Module):
    def __init__(self, vocab: int, hidden: int, blocks: int = 2, tied: bool = False, device="cuda",
                 heads: int = 0, document: int = 512):
        super().__init__()
        self.embed = ScaledEmbedding(vocab, hidden, math.sqrt(hidden) if tied else 1.0, device)
        self.blocks = torch.nn.ModuleList()
        for i in range(blocks):
            if heads:
                self.blocks.append(Attention(hidden, heads, document, 10 * i + 5, device))
            self.blocks.append(Block(hidden, 4 * hidden, 10 * i + 1, device))
        self.head = CrossEntropyHead(hidden, vocab, device,
                                     weight=self.embed.weight if tied else None)

    def forward(self, ids, targets):
        x = self.embed(ids)
        for b in self.blocks:
            x = b(x)
        return self.head(norm(x), targets)


def text(tokens: int, vocab: int, generator: torch.Generator, successor: torch.Tensor):
    """(ids, targets): each target follows its id three times out of four; a few
    positions are padding, an id and a target of -100."""
    ids = torch.randint(0, vocab, (tokens,), generator=generator)
    other = torch.randint(0, vocab, (tokens,), generator=generator)
    targets = torch.where(torch.rand(tokens, generator=generator) < 0.75, successor[ids], other)
    pad = torch.rand(tokens, generator=generator) < 0.02
    ids[pad] = -100
    targets[pad] = -100
    return ids.cuda(), targets.cuda()


def train(steps: int, vocab: int, hidden: int, tokens: int, tied: bool = False, lr: float = 2.0,
          report=None, heads: int = 0, document: int = 512):
    """The losses and gradient norms of `steps` steps of plain SGD."""
    torch.manual_seed(0)
    g = torch.Generator().manual_seed(1)
    successor = torch.randperm(vocab, generator=g)
    model = Model(vocab, hidden, tied=tied, heads=heads, document=document)
    params = list(model.parameters())
    master = [p.detach().float() for p in params]   # FP32 copies take the updates
    history = []
    for step in range(steps):
        t0 = time.perf_counter()
        ids, targets = text(tokens, vocab, g, successor)
        loss = model(ids, targets)
        loss.backward()
        total = clip_grad_norm(params, 1.0)
        with torch.no_grad():
            for p, m in zip(params, master):
                m.sub_(p.grad.float(), alpha=lr)
                p.copy_(m)
                p.grad = None
        history.append((loss.item(), total.item()))
        if report:
            report(step, *history[-1], 1e3 * (time.perf_counter() - t0))
    return history


def main():
    ap = argparse.ArgumentParser(description=__doc__,
                                 formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=30)
    ap.add_argument("--vocab", type=int, default=5000)
    ap.add_argument("--hidden", type=int, default=256)
    ap.add_argument("--tokens", type=int, default=8192)
    ap.add_argument("--tied", action="store_true", help="share the embedding with the head")
    ap.add_argument("--heads", type=int, default=0, help="self-attention of so many heads (0: none)")
    ap.add_argument("--document", type=int, default=512, help="tokens that attend to each other")
    a = ap.parse_args()
    train(a.steps, a.vocab, a.hidden, a.tokens, a.tied, heads=a.heads, document=a.document,
          report=lambda s, l, n, ms: print(f"step {s:3d}  loss {l:7.4f}  norm {n:8.4f}  {ms:7.2f} ms",
                                           flush=True))


if __name__ == "__main__":
    main()
