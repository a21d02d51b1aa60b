"""A few training steps of residual feed-forward blocks under a language-model head,
on synthetic data: NVFP4 linear layers, the residual RMS norm with dropout between
them, and the linear cross entropy over the vocabulary.

    python examples/train_ffn_head.py [--steps 20] [--hidden 512] [--ffn 2048] [--blocks 2]
                                      [--vocab 8192] [--tokens 2048]

Each token's label is a fixed function of its input, so the loss falls.  The last
step's input is also scored in evaluation mode, with the final norm in 8 bits.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from bit_microscaled_quantized_amd.layers import AddRMSNorm, linear_cross_entropy, rms_norm_mx8  # noqa: E402
from bit_microscaled_quantized_amd.module import NVFP4Linear  # noqa: E402


class Block(torch.nn.Module):
    """y -> up -> SiLU -> down; the residual addition belongs to the next norm."""

    def __init__(self, hidden, ffn, seed):
        super().__init__()
        self.up, self.down = NVFP4Linear(hidden, ffn, seed=seed), NVFP4Linear(ffn, hidden, seed=seed + 1)

    def forward(self, y):
        return self.down(torch.nn.functional.silu(self.up(y)))


class Model(torch.nn.Module):
    def __init__(self, hidden, ffn, blocks, vocab, p=0.1):
        super().__init__()
        g = torch.Generator(device="cuda").manual_seed(0)
        rnd = lambda n: torch.randn(n, hidden, generator=g, device="cuda")
        self.embedding = torch.nn.Parameter(rnd(vocab).bfloat16())
        self.head = torch.nn.Parameter((rnd(vocab) * 0.02).bfloat16())
        self.blocks = torch.nn.ModuleList(Block(hidden, ffn, 10 * b + 1) for b in range(blocks))
        # the first norm normalizes the embedding, each later one adds a block's output
        self.norms = torch.nn.ModuleList(AddRMSNorm(hidden, p=p if b else 0.0, seed=b) for b in range(blocks + 1))

    def forward(self, tokens):
        h, y = self.norms[0](self.embedding[tokens])
        for block, norm in zip(self.blocks, self.norms[1:]):
            h, y = norm(block(y), h)
        return y

    def final_mx8(self, tokens):
        """The head's input in 8 bits (inference)."""
        h, y = self.norms[0](self.embedding[tokens])
        for block, norm in zip(self.blocks[:-1], self.norms[1:-1]):
            h, y = norm(block(y), h)
        return rms_norm_mx8(self.blocks[-1](y), h, self.norms[-1].gamma)[1:]


def train(steps=20, hidden=512, ffn=2048, blocks=2, vocab=8192, tokens=2048, lr=0.01, report=print):
    """(losses of the steps, largest difference of the 8-bit final norm from the BF16 one)."""
    torch.manual_seed(0)  # dropout's masks
    model = Model(hidden, ffn, blocks, vocab)
    opt = torch.optim.Adam(model.parameters(), lr=lr, foreach=False)
    g = torch.Generator(device="cuda").manual_seed(1)
    losses = []
    for step in range(steps):
        x = torch.randint(vocab // 8, (tokens,), generator=g, device="cuda")
        labels = (x * 7 + 3) % vocab
        labels[::16] = -100  # ignored
        opt.zero_grad()
        loss = linear_cross_entropy(model(x), model.head, labels)
        loss.backward()
        opt.step()
        losses.append(loss.item())
        if report:
            report(f"step {step}: loss {losses[-1]:.4f}")
    model.eval()
    with torch.no_grad():
        y = model(x).float()
        codes, scales = model.final_mx8(x)
        v = codes.float().view(tokens, -1, 32) * scales.float()[..., None]
        diff = float((v.view(tokens, -1) - y).abs().max() / y.abs().max())
    if report:
        report(f"8-bit final norm: largest difference {diff:.4f} of the largest value")
    return losses, diff


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, default in (("steps", 20), ("hidden", 512), ("ffn", 2048), ("blocks", 2), ("vocab", 8192),
                          ("tokens", 2048)):
        ap.add_argument(f"--{name}", type=int, default=default)
    train(**vars(ap.parse_args()))
