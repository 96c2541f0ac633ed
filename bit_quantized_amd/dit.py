"""A DiT block under 4-bit post-training: the quantized linears with what lies
between them (modulated norms with gates, rotation by positions on several
axes, attention over the packed samples of a batch) and the step that trains
their adapters.

    python -m bit_quantized_amd.dit [--steps 20] [--width 512] [--state q8]

trains the adapters of one block toward the outputs of a block with other
adapters, on synthetic inputs of two images of different size, and prints the
loss.  (FourTune, "3.1 Triple-Branch Hybrid-Precision Pipeline": only the
adapters learn; the frozen weights are 4-bit.)
"""
from __future__ import annotations

import argparse

import torch

from . import ops
from .block import (AdamW, AxialRotary, DocAttention, GatedNorm, GatedNormFunction, RotaryAttentionFunction)
from .layer import FourTuneLinearFunction, QuantizedLinear


class DiTBlock:
    """One block over rows packed sample after sample:

        h = (1 + scale1) LN(x) + shift1;  x = x + gate1 out(attention(rotate(qkv(h))))
        h = (1 + scale2) LN(x) + shift2;  x = x + gate2 fc2(gelu(fc1(h)))

    with the modulation (shift, scale, gate of both halves) from a quantized
    linear of the conditioning, as the linears are.  `linear(N, K, act_out)`
    makes a quantized linear."""

    def __init__(self, width: int, heads: int, axis_dims, linear):
        self.heads, self.dim = heads, width // heads
        self.qkv, self.out = linear(3 * width, width), linear(width, width)
        self.fc1, self.fc2 = linear(4 * width, width, ops.FT_ACT_GELU_TANH), linear(width, 4 * width)
        self.mod = linear(6 * width, width)
        self.norm = GatedNorm(norm="layer", eps=1e-6)
        one = torch.ones(self.dim, dtype=torch.bfloat16, device=self.qkv.device)
        self.rope = AxialRotary(self.dim, axis_dims, q_weight=one, k_weight=one)
        self.attn = DocAttention(self.dim)

    def linears(self):
        return [self.qkv, self.out, self.fc1, self.fc2, self.mod]

    def adapters(self):
        """The trainable tensors."""
        return [t for l in self.linears() for t in (l.At, l.B)]

    def __call__(self, x, cond, positions, segments):
        """x [M, width]; cond [samples, width]; positions int32 [M, axes]; segments
        int32 [samples + 1], the row offsets of the samples."""
        lin = lambda layer, t: FourTuneLinearFunction.apply(t, layer.At, layer.B, layer)
        shift1, scale1, gate1, shift2, scale2, gate2 = lin(self.mod, cond).chunk(6, 1)
        x, h = GatedNormFunction.apply(x, None, None, scale1, shift1, self.norm, segments)
        o = RotaryAttentionFunction.apply(lin(self.qkv, h), positions, self.rope, self.attn, self.heads, self.heads,
                                          segments)
        x, h = GatedNormFunction.apply(x, lin(self.out, o), gate1, scale2, shift2, self.norm, segments)
        x, _ = GatedNormFunction.apply(x, lin(self.fc2, lin(self.fc1, h)), gate2, None, None, self.norm, segments, False)
        return x


def quantized_linears(width_rank: int, generator: torch.Generator, device):
    """A maker of quantized linears with random frozen weights, a stabilizer and an adapter of that rank."""
    def make(N, K, act_out=ops.FT_ACT_NONE):
        n = lambda *s, std: (torch.randn(*s, generator=generator, device=device) * std).to(torch.bfloat16)
        r = width_rank
        layer = QuantizedLinear(n(N, K, std=K ** -0.5), n(r, K, std=K ** -0.5), n(r, N, std=0.1),
                                n(r, K, std=K ** -0.5), n(r, N, std=0.02), act_out=act_out)
        layer.At.requires_grad_(True)
        layer.B.requires_grad_(True)
        return layer
    return make


def grid_positions(text: int, height: int, width: int, device):
    """Positions on three axes of a sample: text tokens at 0, then the image's rows and columns."""
    pos = torch.zeros((text + height * width, 3), dtype=torch.int32, device=device)
    i = torch.arange(height * width, dtype=torch.int32, device=device)
    pos[text:, 1], pos[text:, 2] = i // width, i % width
    return pos


def train(steps: int = 20, width: int = 512, rank: int = 16, lr: float = 3e-3, state: str = "f32", seed: int = 0, say=print):
    """Train a block's adapters toward another's outputs; returns the losses."""
    dev = torch.device("cuda:0")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    heads, dim = width // 64, 64
    block = DiTBlock(width, heads, [dim // 4, dim // 2 - dim // 8, dim // 2 - dim // 8], quantized_linears(rank, gen, dev))
    sizes = [(32, 16, 16), (32, 12, 10)]                      # text tokens, height, width of each sample
    positions = torch.cat([grid_positions(*s, dev) for s in sizes])
    rows = [t + h * w for t, h, w in sizes]
    segments = torch.tensor([0, rows[0], sum(rows)], dtype=torch.int32, device=dev)
    x = torch.randn(sum(rows), width, generator=gen, device=dev).to(torch.bfloat16)
    cond = torch.randn(len(rows), width, generator=gen, device=dev).to(torch.bfloat16)
    params = block.adapters()
    with torch.no_grad():                                     # the target: the same block with other adapters
        start = [p.clone() for p in params]
        for p in params:
            p.add_((torch.randn(p.shape, generator=gen, device=dev) * 0.05).to(p.dtype))
        target = block(x, cond, positions, segments).float()
        for p, s in zip(params, start):
            p.copy_(s)
    for p in params:
        p.grad = torch.zeros_like(p)
    masters = [p.detach().float() for p in params] if state == "f32" else None
    opt = AdamW([p.detach() for p in params], [p.grad for p in params], lr=lr, weight_decay=0.0, masters=masters, state=state,
                seed=seed)
    losses = []
    for step in range(steps):
        for p in params:
            p.grad.zero_()
        out = block(x, cond, positions, segments)
        loss = (out.float() - target).square().mean()
        loss.backward()
        # clip to a gradient norm of 1 without a look at it from the host
        norm = torch.stack([p.grad.float().square().sum() for p in params]).sum().sqrt()
        opt.step(grad_scale=(1.0 / norm.clamp(min=1.0)).reshape(1))
        losses.append(loss.detach())
    losses = [float(v) for v in losses]
    if say:
        for i, v in enumerate(losses):
            say(f"step {i:3d}  loss {v:.6f}")
    return losses


def main():
    ap = argparse.ArgumentParser(description="Train the adapters of one quantized DiT block on synthetic inputs.")
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--width", type=int, default=512, help="channels, a multiple of 64")
    ap.add_argument("--rank", type=int, default=16)
    ap.add_argument("--lr", type=float, default=3e-3)
    ap.add_argument("--state", choices=("f32", "q8"), default="f32", help="optimizer states in 32 bits or in 8")
    a = ap.parse_args()
    train(a.steps, a.width, a.rank, a.lr, a.state)


if __name__ == "__main__":
    main()
