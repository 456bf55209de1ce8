"""The running bounds of both forms of gelu (CPU): values and derivatives are torch's,
and the kernels' arithmetic in fp32 stays inside, while a bound that a wrong
polynomial would pass does not exist."""
import math

import pytest
import torch

from running_bounds import U32, B, act


@pytest.mark.parametrize("kind", ["gelu", "gelu_tanh"])
def test_values_and_derivatives(kind):
    t = torch.linspace(-9, 9, 4001, dtype=torch.float64).requires_grad_()
    want = torch.nn.functional.gelu(t, approximate="tanh" if kind == "gelu_tanh" else "none")
    slope, = torch.autograd.grad(want.sum(), t)
    v, d = act(B(t), kind)
    assert torch.allclose(v.v, want.detach(), rtol=1e-10, atol=1e-13) and torch.allclose(d.v, slope, rtol=1e-10, atol=1e-13)
    # a few thousand units of the largest part at most
    assert (v.e <= 400 * v.v.abs() + 50).all() and (d.e <= 400).all()


@pytest.mark.parametrize("kind", ["gelu", "gelu_tanh"])
def test_fp32_arithmetic_stays_inside(kind):
    t = torch.cat([torch.linspace(-13, 13, 20011), torch.randn(20000, generator=torch.Generator().manual_seed(1))])
    assert t.dtype == torch.float32
    if kind == "gelu":
        e = torch.exp(-0.5 * t * t)
        tail = 0.5 * torch.special.erfcx(t.abs() * math.sqrt(0.5)) * e
        p = torch.where(t < 0, tail, 1 - tail)
        v, d = t.clamp(min=0) - t.abs() * tail, p + t * 0.39894228040143268 * e
    else:
        k = 0.79788456080286536
        p = 1 / (1 + torch.exp(-2 * k * (t + 0.044715 * t * t * t)))
        v, d = t * p, p + t * p * (1 - p) * (2 * k) * (1 + 3 * 0.044715 * t * t)
    for got, want in zip((v, d), act(B(t), kind)):
        off = (got.double() - want.v).abs()
        assert (off <= U32 * want.e + 2.0 ** -126).all()
        assert ((got.double() * (1 + 1e-4) - want.v).abs() > U32 * want.e).float().mean() > 0.4
