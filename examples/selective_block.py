"""A residual block that mixes along the sequence, trained for a few steps, then
continued token by token.

    a = rms(x)                                 the norm before the block
    u, z = a Win^T                             inner channels and their gate
    v = silu(causal convolution of u)          four taps along the sequence
    r, B, C = v Wx^T                           rank of the step, states' in and out
    h = scan(v, r Wd^T, A, B, C, D) silu(z)    selective state space scan
    y = x + h Wout^T,  o = rms(y)              what the next block would read

All sequences of a batch lie packed in one tensor.  The loss is the mean squared
distance of ``o`` to a target; a step clips by the gradients' global norm inside
AdamW, on fp32 parameters with 8-bit states that leave bf16 weights for the next
forward pass.

    python examples/selective_block.py [--steps N] [--device cuda:0]
"""
from __future__ import annotations

import argparse
import math
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import convolution_implicit_gemm_conv2d_amd as cm

TAPS = 4
# Kept in float32 also where the block computes in bfloat16.
WIDE = ("A_log", "D", "step_bias")


def project(x, w):
    """``x`` [rows, C] through a 1x1 convolution with ``w`` [F, C]."""
    return cm.conv1d(x.unsqueeze(0), w.unsqueeze(1), None, layout="NLC")[0]


def project_grad(dy, x, w):
    """Gradients of ``project``: of ``x`` and of ``w``."""
    dy, x = dy[None, None], x[None, None]
    dx = cm.conv2d_input_grad(dy, w[:, None, None], tuple(x.shape), layout="NHWC")
    return dx[0, 0], cm.conv2d_weight_grad(x, dy, (w.shape[0], 1, 1, w.shape[1]), layout="NHWC").view(w.shape)


class SelectiveBlock:
    """The block's weights, its forward and backward pass, and its form for tokens."""

    def __init__(self, channels: int, inner: int, states: int = 16, dtype=torch.bfloat16, device="cuda:0", seed: int = 0):
        gen = torch.Generator().manual_seed(seed)
        rank = -(-channels // 16)
        self.inner, self.rank, self.states, self.dtype = inner, rank, states, dtype

        def t(*shape, std=1.0, mean=0.0, type_=None):
            return (torch.randn(shape, generator=gen) * std + mean).to(device, type_ or dtype)

        step = torch.exp(torch.rand(inner, generator=gen) * math.log(100.0) + math.log(1e-3))
        self.w = {
            "pre": t(channels, std=0.02, mean=1.0), "in": t(2 * inner, channels, std=channels ** -0.5),
            "conv": t(inner, TAPS, std=TAPS ** -0.5), "conv_bias": t(inner, std=0.02),
            "x": t(rank + 2 * states, inner, std=inner ** -0.5), "step": t(inner, rank, std=rank ** -0.5),
            "step_bias": (step + torch.log(-torch.expm1(-step))).to(device),
            "A_log": torch.log(torch.arange(1, states + 1.0)).repeat(inner, 1).to(device),
            "D": torch.ones(inner, device=device), "out": t(channels, inner, std=inner ** -0.5),
            "next": t(channels, std=0.02, mean=1.0),
        }

    def _inputs(self, x):
        """What the scan's channels are computed from: u, z."""
        _, a = cm.block_norm(x, pre_weight=self.w["pre"], pre="rms")
        uz = project(a, self.w["in"])
        return a, uz[:, :self.inner], uz[:, self.inner:]

    def _steps(self, v):
        p = project(v, self.w["x"])
        r = p[:, :self.rank].contiguous()
        delta = project(r, self.w["step"])
        return r, delta, p[:, self.rank:self.rank + self.states], p[:, self.rank + self.states:]

    def _scan(self, z):
        w = self.w
        return dict(D=w["D"], z=z, delta_bias=w["step_bias"])

    def _output(self, x, h):
        f = project(h, self.w["out"])
        return f, *cm.block_norm(x, f, pre_weight=self.w["next"], pre="rms")

    def forward(self, x, starts, conv_last=None, scan_last=None):
        """``x`` [rows, C] with the sequences of ``starts``: (y, o, what ``backward``
        needs).  ``conv_last`` and ``scan_last`` receive the states behind them."""
        a, u, z = self._inputs(x)
        v = cm.causal_conv(u, self.w["conv"], self.w["conv_bias"], activation="silu", starts=starts, last=conv_last)
        r, delta, B, C = self._steps(v)
        A = -torch.exp(self.w["A_log"])
        saved = cm.selective_scan_saved(v, A)
        h = cm.selective_scan(v, delta, A, B, C, starts=starts, last=scan_last, saved=saved, **self._scan(z))
        f, y, o = self._output(x, h)
        return y, o, (x, starts, a, u, z, v, r, delta, A, B, C, saved, h, f)

    def backward(self, do, kept):
        """Gradients of x and of all weights, from the gradient of ``o``."""
        w = self.w
        x, starts, a, u, z, v, r, delta, A, B, C, saved, h, f = kept
        n = cm.block_norm_grad(None, do, x, f, pre_weight=w["next"], pre="rms", post="none")
        dw = {"next": n["pre_weight"]}
        dh, dw["out"] = project_grad(n["branch"], h, w["out"])
        d = cm.selective_scan_grad(dh, v, delta, A, B, C, starts=starts, saved=saved, **self._scan(z))
        dw["A_log"], dw["D"], dw["step_bias"] = d["A"] * A, d["D"], d["delta_bias"]
        dr, dw["step"] = project_grad(d["delta"], r, w["step"])
        dv, dw["x"] = project_grad(torch.cat([dr, d["B"], d["C"]], 1), v, w["x"])
        c = cm.causal_conv_grad(d["x"] + dv, u, w["conv"], w["conv_bias"], activation="silu", starts=starts)
        dw["conv"], dw["conv_bias"] = c["weight"], c["bias"]
        da, dw["in"] = project_grad(torch.cat([c["x"], d["z"]], 1), a, w["in"])
        first = cm.block_norm_grad(None, da, x, pre_weight=w["pre"], pre="rms")
        dw["pre"] = first["pre_weight"]
        return n["x"] + first["x"], dw

    def token(self, x, conv_state, scan_state, slots=None):
        """One row [C] more for each of many sequences, whose states move on in place."""
        _, u, z = self._inputs(x)
        v = cm.causal_conv_step(u, self.w["conv"], conv_state, self.w["conv_bias"], activation="silu", slots=slots)
        _, delta, B, C = self._steps(v)
        h = cm.selective_step(v, delta, -torch.exp(self.w["A_log"]), B, C, scan_state, slots=slots, **self._scan(z))
        return self._output(x, h)[1:]

    def pool(self, count: int):
        """States of ``count`` sequences before their first row."""
        device = self.w["conv"].device
        return (torch.zeros(count, TAPS - 1, self.inner, dtype=self.dtype, device=device),
                torch.zeros(count, self.inner, self.states, device=device))


class Trainer:
    """fp32 parameters of a block, their 8-bit states, and the step."""

    def __init__(self, block: SelectiveBlock, bits: int = 8):
        self.block, self.names, self.count = block, list(block.w), 0
        self.params = [block.w[k].float() for k in self.names]
        # the block's own weights are the copies that a step leaves
        self.copies = [block.w[k] for k in self.names]
        self.state = cm.adamw_state(self.params, bits)

    def step(self, dw, rate: float, max_norm: float = 1.0):
        grads = [dw[k] for k in self.names]
        norm = cm.gradient_norm(grads)
        self.count += 1
        copies = [c if c.data_ptr() != p.data_ptr() else None for c, p in zip(self.copies, self.params)]
        cm.adamw_step(self.params, grads, self.state, self.count, rate, weight_decay=0.01, norm=norm, max_norm=max_norm, copies=copies)
        return norm


def train(steps: int = 20, lengths=(70, 1, 129, 56), channels: int = 96, inner: int = 192, device="cuda:0"):
    """Losses of a few steps towards the output of another block, and the block."""
    gen = torch.Generator().manual_seed(1)
    starts = torch.tensor([0, *torch.tensor(lengths).cumsum(0).tolist()], dtype=torch.int32, device=device)
    x = torch.randn((sum(lengths), channels), generator=gen).to(device, torch.bfloat16)
    _, target, _ = SelectiveBlock(channels, inner, device=device, seed=2).forward(x, starts)
    block = SelectiveBlock(channels, inner, device=device, seed=3)
    trainer, losses = Trainer(block), []
    for _ in range(steps):
        _, o, kept = block.forward(x, starts)
        e = o.float() - target.float()
        losses.append((e * e).mean())
        _, dw = block.backward((2 * e).to(torch.bfloat16), kept)
        trainer.step(dw, rate=3e-3)
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
        # a prompt, and three tokens behind it
        prompt = torch.randn(33, channels).to(a.device, torch.bfloat16)
        conv_state, scan_state = block.pool(1)
        starts = torch.tensor([0, 33], dtype=torch.int32, device=a.device)
        y, _, _ = block.forward(prompt, starts, conv_last=conv_state, scan_last=scan_state)
        row = y[-1:]
        for i in range(3):
            row, _ = block.token(row, conv_state, scan_state)
            print("token", i, "finite" if torch.isfinite(row).all() else "not finite")


if __name__ == "__main__":
    main()
