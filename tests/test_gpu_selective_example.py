"""The example that runs the operators along a sequence and the optimizer step
together: its gradients against automatic differentiation of the same block in 64
bits, its form for tokens against the one for prompts, and its training."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import selective_block  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
LENGTHS = (5, 0, 33, 1, 18)


def starts_of(lengths):
    return torch.tensor([0, *torch.tensor(lengths).cumsum(0).tolist()], dtype=torch.int32, device=DEV)


def reference(block, x, do):
    w = {k: v.detach().cpu().double().requires_grad_() for k, v in block.w.items()}
    x = x.detach().cpu().double().requires_grad_()
    rms = lambda v, g: v / (v.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt() * g  # noqa: E731
    silu, E, R, N = torch.nn.functional.silu, block.inner, block.rank, block.states
    uz = rms(x, w["pre"]) @ w["in"].t()
    hs, at = [], 0
    for n in LENGTHS:
        u, z = uz[at:at + n, :E], uz[at:at + n, E:]
        at += n
        line = torch.cat([torch.zeros(3, E, dtype=torch.float64), u])
        v = silu(torch.stack([(line[t:t + 4] * w["conv"].t()).sum(0) for t in range(n)]) + w["conv_bias"]) if n else u
        p = v @ w["x"].t()
        d = torch.log1p(torch.exp(p[:, :R] @ w["step"].t() + w["step_bias"]))
        h, A = torch.zeros(E, N, dtype=torch.float64), -torch.exp(w["A_log"])
        for t in range(n):
            h = torch.exp(d[t][:, None] * A) * h + (d[t] * v[t])[:, None] * p[t, R:R + N]
            hs.append(((h * p[t, R + N:]).sum(1) + w["D"] * v[t]) * silu(z[t]))
    y = x + torch.stack(hs) @ w["out"].t()
    o = rms(y, w["next"])
    g = torch.autograd.grad((o * do.cpu().double()).sum(), [x, *w.values()])
    return y, o, g[0], dict(zip(w, g[1:]))


@pytest.mark.parametrize("dtype,tol", [(torch.float32, 1e-4), (torch.bfloat16, 0.05)])
def test_block_against_autograd(dtype, tol):
    # a chain of nine operators, each rounding its outputs once: in the 2-norm a few
    # half steps of the type, in bf16 (2^-8 each) through the scan's products of three
    gen = torch.Generator().manual_seed(5)
    t = lambda *s: torch.randn(s, generator=gen).to(DEV, dtype)  # noqa: E731
    block = selective_block.SelectiveBlock(40, 72, dtype=dtype)
    x, do = t(sum(LENGTHS), 40), t(sum(LENGTHS), 40)
    y, o, kept = block.forward(x, starts_of(LENGTHS))
    dx, dw = block.backward(do, kept)
    torch.cuda.synchronize()
    ry, ro, rx, rw = reference(block, x, do)
    assert set(dw) == set(rw)
    for name, got, want in [("y", y, ry), ("o", o, ro), ("dx", dx, rx)] + [(k, dw[k], rw[k]) for k in rw]:
        assert got.shape == want.shape, name
        err = ((got.cpu().double() - want).norm() / want.norm()).item()
        print(f"  {name}: {err:.2e}", flush=True)
        assert err <= tol, (name, err)


def test_tokens_go_on_from_a_prompt():
    gen = torch.Generator().manual_seed(6)
    block = selective_block.SelectiveBlock(40, 72, dtype=torch.float32)
    x = torch.randn(3, 30, 40, generator=gen).to(DEV)
    whole, _, _ = block.forward(x.view(90, 40), starts_of((30, 30, 30)))
    conv, scan = block.pool(3)
    first, _, _ = block.forward(x[:, :20].reshape(60, 40), starts_of((20, 20, 20)), conv_last=conv, scan_last=scan)
    parts = [first.view(3, 20, 40)]
    for t in range(20, 30):
        parts.append(block.token(x[:, t].contiguous(), conv, scan)[0].unsqueeze(1))
    got, want = torch.cat(parts, 1), whole.view(3, 30, 40)
    # the same sums in other orders, in fp32
    assert ((got - want).norm() / want.norm()).item() <= 1e-5


def test_training_runs():
    block, losses = selective_block.train(steps=6)
    assert all(v == v for v in losses)
    assert all(torch.isfinite(v).all() for v in block.w.values())


def test_a_step_moves_every_weight_by_its_gradient():
    """The first AdamW step of each weight is the rate against its gradient's sign."""
    block = selective_block.SelectiveBlock(40, 72)
    x = torch.randn(57, 40, generator=torch.Generator().manual_seed(7)).to(DEV, torch.bfloat16)
    y, o, kept = block.forward(x, starts_of(LENGTHS))
    _, dw = block.backward(torch.ones_like(o), kept)
    trainer = selective_block.Trainer(block, bits=32)
    before = [p.clone() for p in trainer.params]
    trainer.step(dw, rate=1e-3, max_norm=1e9)
    for k, p, b in zip(trainer.names, trainer.params, before):
        g = dw[k].float()
        want = b * (1 - 1e-5) - 1e-3 * g / (g.abs() + 1e-8)
        assert torch.allclose(p, want, rtol=1e-5, atol=1e-7), k
        assert torch.equal(block.w[k], p.to(block.w[k].dtype)), k
