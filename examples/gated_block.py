"""A residual block of images trained for a few steps, then run on one token.

    a = rms(x)                               the norm before the block
    h = silu(a Wg^T + bg) * (a Wu^T + bu)    gated feed-forward layer
    f = conv1x1(h)                           back to the stream's width
    y = x + s * sigmoid(z) * layer(f)        norm after it, gate of each image
    o = rms(y)                               what the next block would read

The loss is the mean squared distance of ``o`` to a target; the gradients of all
weights are clipped by their global norm and taken as a plain step.  Everything
is channels-last (NHWC images, OHWI weights).

    python examples/gated_block.py [--steps N] [--device cuda:0]
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import convolution_implicit_gemm_conv2d_amd as cm


class GatedBlock:
    """The block's weights and its forward and backward pass."""

    def __init__(self, channels: int, hidden: int, dtype=torch.bfloat16, device="cuda:0", seed: int = 0):
        gen = torch.Generator().manual_seed(seed)

        def t(*shape, std=1.0, mean=0.0):
            return (torch.randn(shape, generator=gen) * std + mean).to(device, dtype)

        self.w = {
            "pre": t(channels, std=0.02, mean=1.0),
            "gate": t(hidden, 1, 1, channels, std=channels ** -0.5), "gate_bias": t(hidden, std=0.02),
            "up": t(hidden, 1, 1, channels, std=channels ** -0.5), "up_bias": t(hidden, std=0.02),
            "down": t(channels, 1, 1, hidden, std=hidden ** -0.5),
            "post": t(channels, std=0.02, mean=1.0), "post_bias": t(channels, std=0.02),
            "scale": t(channels, std=0.02, mean=0.5), "next": t(channels, std=0.02, mean=1.0),
        }

    def _norms(self, z):
        w = self.w
        return dict(gate=z, scale=w["scale"], post_weight=w["post"], post_bias=w["post_bias"], pre_weight=w["next"],
                    post="layer", pre="rms", gate_activation="sigmoid")

    def forward(self, x, z):
        """``x`` [N, H, W, C] and a gate ``z`` [N, C]: (y, o, what ``backward`` needs)."""
        w = self.w
        _, a = cm.block_norm(x, pre_weight=w["pre"], pre="rms")
        h = cm.gated_feed_forward(a, w["gate"], w["up"], w["gate_bias"], w["up_bias"], activation="silu")
        f = cm.conv2d(h, w["down"], None, layout="NHWC")
        y, o = cm.block_norm(x, f, **self._norms(z))
        return y, o, (x, z, a, h, f)

    def backward(self, do, kept):
        """Gradients of x, z and all weights, from the gradient of ``o``."""
        w = self.w
        x, z, a, h, f = kept
        d = cm.block_norm_grad(None, do, x, f, **self._norms(z))
        df = d["branch"]
        dh = cm.conv2d_input_grad(df, w["down"], tuple(h.shape), layout="NHWC")
        dw = {"down": cm.conv2d_weight_grad(h, df, tuple(w["down"].shape), layout="NHWC"), "scale": d["scale"],
              "post": d["post_weight"], "post_bias": d["post_bias"], "next": d["pre_weight"]}
        da, dw["gate"], dw["up"], dw["gate_bias"], dw["up_bias"] = cm.gated_feed_forward_grad(
            dh, a, w["gate"], w["up"], w["gate_bias"], w["up_bias"], activation="silu")
        first = cm.block_norm_grad(None, da, x, pre_weight=w["pre"], pre="rms")
        dw["pre"] = first["pre_weight"]
        return d["x"] + first["x"], d["gate"], dw

    def step(self, dw, rate: float, max_norm: float = 1.0):
        """Clips the gradients in place and takes a step; returns their norm."""
        norm = cm.clip_gradients([dw[k] for k in self.w], max_norm)
        for k, w in self.w.items():
            w.add_(dw[k], alpha=-rate)
        return norm


def train(steps: int = 20, images: int = 4, size: int = 14, channels: int = 128, hidden: int = 512, device="cuda:0"):
    """Losses of a few steps towards the output of another block."""
    gen = torch.Generator().manual_seed(1)
    x = torch.randn((images, size, size, channels), generator=gen).to(device, torch.bfloat16)
    z = torch.randn((images, channels), generator=gen).to(device, torch.bfloat16)
    _, target, _ = GatedBlock(channels, hidden, device=device, seed=2).forward(x, z)
    block, losses = GatedBlock(channels, hidden, device=device, seed=3), []
    for _ in range(steps):
        _, o, kept = block.forward(x, z)
        e = o.float() - target.float()
        losses.append((e * e).mean())
        _, _, dw = block.backward((2 * e).to(torch.bfloat16), kept)
        block.step(dw, rate=0.05)
    return block, [v.item() for v in losses]


def main() -> None:
    p = argparse.ArgumentParser()
    p.add_argument("--steps", type=int, default=20)
    p.add_argument("--device", default="cuda:0")
    a = p.parse_args()
    with torch.cuda.device(a.device):
        block, losses = train(a.steps, device=a.device)
        for i, v in enumerate(losses):
            print(f"step {i:3d}  loss {v:.5f}")
        channels = block.w["pre"].numel()
        token = torch.randn(1, 1, 1, channels).to(a.device, torch.bfloat16)
        y, o, _ = block.forward(token, torch.zeros(1, channels, dtype=torch.bfloat16, device=a.device))
        print("one token:", tuple(y.shape), tuple(o.shape), "finite" if torch.isfinite(o).all() else "not finite")


if __name__ == "__main__":
    main()
