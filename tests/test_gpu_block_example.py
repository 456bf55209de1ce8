"""The example that runs the block operators together: its gradients against
automatic differentiation of the same block in 64 bits, and its training."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import gated_block  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def reference(block, x, z, do):
    w = {k: v.detach().cpu().double().requires_grad_() for k, v in block.w.items()}
    x, z = (t.detach().cpu().double().requires_grad_() for t in (x, z))
    rms = lambda v, g: v / (v.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt() * g  # noqa: E731
    F = torch.nn.functional
    a = rms(x, w["pre"])
    C = x.shape[-1]
    h = F.silu(F.linear(a, w["gate"].view(-1, C), w["gate_bias"])) * F.linear(a, w["up"].view(-1, C), w["up_bias"])
    f = F.linear(h, w["down"].view(C, -1))
    f = (f - f.mean(-1, keepdim=True)) / (f.var(-1, unbiased=False, keepdim=True) + 1e-6).sqrt() * w["post"] + w["post_bias"]
    y = x + w["scale"] * torch.sigmoid(z)[:, None, None, :] * f
    o = rms(y, w["next"])
    g = torch.autograd.grad((o * do.cpu().double()).sum(), [x, z, *w.values()])
    return y, o, g[0], g[1], dict(zip(w, g[2:]))


@pytest.mark.parametrize("dtype,tol", [(torch.float32, 1e-4), (torch.bfloat16, 0.03)])
def test_block_against_autograd(dtype, tol):
    # six operators one after another, each rounding its outputs once: in the
    # 2-norm a few half steps of the type (fp32: its sums' roundings)
    gen = torch.Generator().manual_seed(5)
    t = lambda *s: torch.randn(s, generator=gen).to(DEV, dtype)  # noqa: E731
    block = gated_block.GatedBlock(40, 96, dtype=dtype)
    x, z, do = t(3, 5, 4, 40), t(3, 40), t(3, 5, 4, 40)
    y, o, kept = block.forward(x, z)
    dx, dz, dw = block.backward(do, kept)
    torch.cuda.synchronize()
    ry, ro, rx, rz, rw = reference(block, x, z, do)
    pairs = [("y", y, ry), ("o", o, ro), ("dx", dx, rx), ("dz", dz, rz)] + [(k, dw[k], rw[k]) for k in rw]
    for name, got, want in pairs:
        err = ((got.cpu().double() - want).norm() / want.norm()).item()
        print(f"  {name}: {err:.2e}", flush=True)
        assert err <= tol, (name, err)


def test_training_lowers_the_loss():
    _, losses = gated_block.train(steps=12)
    assert all(v == v for v in losses) and losses[-1] < losses[0], losses
