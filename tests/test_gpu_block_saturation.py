"""Activations and their derivatives over the whole range of their arguments: near
0, in the tails, saturated, up to the largest finite values, infinities and NaN,
through the gate of a block norm and through the gated layer's forms.

Tolerances.  The hardware's exponential and reciprocal are good to a unit in the
last place, but an exponential's argument E moves it by its own roundings: at most
six of them (cube, sum, two constants, products), so a tail's relative error is at
most (6 E + 16) 2^-24 with E = |t|, t^2 / 2 (gelu) or 2 sqrt(2 / pi) |t + 0.044715
t^3| (gelu_tanh); a logistic value below the smallest normal is 0, which moves a
value by |t| times that.  A derivative is a sum of terms no larger than
1 + |t|, 16 roundings of them while the activation is not saturated (|t| < 200); where it is, 0 or 1.
Then the output's own rounding, and in the gated layer's gradient that of dg and
du as operands in bf16.
"""
import math

import pytest
import torch

import block_reference as br
import convolution_implicit_gemm_conv2d_amd as cm

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF16, F32 = torch.bfloat16, torch.float32
SIZES = [0.0, 1e-30, 1e-8, 0.1, 0.3, 0.59, 0.61, 1.0, 2.0, 3.0, 4.0, 5.5, 7.0, 9.0, 11.0, 13.0, 13.6, 14.0, 20.0, 40.0, 64.0, 80.0, 87.0, 88.5,
         89.0, 100.0, 104.0, 128.0, 199.0, 1e4, 1e10, 1e13, 1e18, 3e19, 1e25, 1e32, 3e38]


def arguments(dtype):
    v = torch.tensor(SIZES + [-s for s in SIZES], dtype=torch.float64).to(dtype)
    return torch.cat([v, v[torch.randperm(len(v), generator=torch.Generator().manual_seed(1))]])


def act64(t, kind):
    """Value and derivative from definitions that keep the tails."""
    zero, one = torch.zeros_like(t), torch.ones_like(t)
    if kind == "none":
        return t, one
    if kind == "relu":
        return torch.where(t > 0, t, zero), torch.where(t > 0, one, zero)
    if kind == "tanh":
        return torch.tanh(t), torch.cosh(t.clamp(-300, 300)) ** -2
    if kind == "gelu":
        phi = 0.5 * torch.erfc(-t / math.sqrt(2))
        return t * phi, phi + t * torch.exp(-0.5 * t * t) / math.sqrt(2 * math.pi)
    c = math.sqrt(2 / math.pi)
    w, slope = {"gelu_tanh": (2 * c * (t + 0.044715 * t ** 3), 2 * c * (1 + 0.134145 * t * t))}.get(kind, (t, one))
    p, q = torch.sigmoid(w), torch.sigmoid(-w)
    if kind == "sigmoid":
        return p, p * q
    return t * p, p + t * p * q * torch.where(p * q == 0, one, slope)


def tolerances(t, kind, v, d, dtype):
    a = t.abs()
    tiny = torch.finfo(F32).tiny
    e = {"gelu": 0.5 * a * a, "gelu_tanh": 2 * math.sqrt(2 / math.pi) * (a + 0.044715 * a ** 3)}.get(kind, a)
    e = torch.where(v.abs() < a / 2, e, 0 * e).clamp(max=120)  # on the side of the tail
    if kind in ("sigmoid", "tanh"):
        e = a.clamp(max=120)
    value = (6 * e + 16) * br.U32 * v.abs() + (1 + a.clamp(max=200)) * tiny
    if kind == "tanh":
        value = value + 4 * br.U32 * (a > 0.5)
    slope = 16 * br.U32 * torch.where(a < 200, 1 + a, 0 * a) + tiny
    half = br.half_step(dtype)
    return value + half * (v.abs() + value) + tiny, slope + half * (d.abs() + slope) + tiny


def close(name, got, want, tol, t):
    g = got.detach().cpu().double()
    bad = ~((g - want).abs() <= tol)
    assert not bad.any(), (name, [(a, b, c) for a, b, c in zip(t[bad].tolist(), g[bad].tolist(), want[bad].tolist())][:8])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kind", list(cm.ACTIVATIONS))
@pytest.mark.parametrize("C", [40, 148, 600, 9000, 5])  # lanes, a wave, a workgroup, sums apart, short rows
def test_gate(C, kind, dtype):
    v = arguments(dtype)
    rows = -(-len(v) // C) + 1
    z = torch.cat([v] * (-(-rows * C // len(v))))[:rows * C].view(rows, C)
    t = z.double()
    want_v, want_d = act64(t, kind)
    tol_v, tol_d = tolerances(t, kind, want_v, want_d, dtype)
    x, f = torch.zeros_like(z).to(DEV), torch.ones_like(z).to(DEV)
    y, _ = cm.block_norm(x, f, gate=z.to(DEV), pre="none", gate_activation=kind)
    g = cm.block_norm_grad(f, None, x, f, gate=z.to(DEV), pre="none", gate_activation=kind)
    torch.cuda.synchronize()
    close("value", y, want_v, tol_v, t)
    close("branch", g["branch"], want_v, tol_v, t)
    close("derivative", g["gate"], want_d, tol_d, t)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kind", list(cm.ACTIVATIONS))
@pytest.mark.parametrize("rows", [60, 148, 20000])  # few rows, small tiles, larger ones
def test_gated_layer(rows, kind, dtype):
    # g is the argument and u is 1, exactly: dx is (act', act, 0, ...)
    v = arguments(dtype)
    v = torch.cat([v] * (-(-rows // len(v))))[:rows]
    C, F = 16, 40
    x = torch.zeros(rows, C, dtype=dtype)
    x[:, 0], x[:, 1] = v, 1
    wg, wu = torch.zeros(F, C, dtype=dtype), torch.zeros(F, C, dtype=dtype)
    wg[:, 0], wu[:, 1] = 1, 1
    dh = torch.zeros(rows, F, dtype=dtype)
    dh[:, 7] = 1
    t = v.double()
    want_v, want_d = act64(t, kind)
    tol_v, tol_d = tolerances(t, kind, want_v, want_d, dtype)
    a = [s.to(DEV) for s in (x, wg, wu)]
    saved = torch.empty(rows, 2 * F, device=DEV)
    h = cm.gated_feed_forward(*a, activation=kind, saved=saved)
    outs = [cm.gated_feed_forward_grad(dh.to(DEV), *a, activation=kind, saved=s)[0] for s in (None, saved)]
    torch.cuda.synchronize()
    for f in (0, 7, F - 1):
        close("h", h[:, f], want_v, tol_v, t)
        assert torch.equal(saved[:, f].cpu().double(), t)
    half = br.half_step(dtype)
    for dx in outs:  # one rounding more, as operands
        close("dg", dx[:, 0], want_d, 2 * tol_d + half * want_d.abs(), t)
        close("du", dx[:, 1], want_v, 2 * tol_v + half * want_v.abs(), t)
        assert (dx[:, 2:] == 0).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kind", list(cm.ACTIVATIONS))
def test_infinities_and_nan(kind, dtype):
    # the formula's limit, or NaN where the formula has infinity times 0
    inf = float("inf")
    z = torch.tensor([inf, -inf, float("nan"), 1.0] * 10, dtype=dtype).view(1, 40)
    x, f = torch.zeros_like(z).to(DEV), torch.ones_like(z).to(DEV)
    y, _ = cm.block_norm(x, f, gate=z.to(DEV), pre="none", gate_activation=kind)
    d = cm.block_norm_grad(f, None, x, f, gate=z.to(DEV), pre="none", gate_activation=kind)["gate"]
    up = {"sigmoid": 1.0, "tanh": 1.0}.get(kind, inf)
    down = {"none": -inf, "tanh": -1.0}.get(kind, 0.0)
    slope = {"none": (1.0, 1.0), "sigmoid": (0.0, 0.0), "tanh": (0.0, 0.0)}.get(kind, (1.0, 0.0))
    exact = kind in ("none", "sigmoid", "tanh", "relu")
    for name, got, limits in (("value", y.cpu(), (up, down)), ("derivative", d.cpu(), slope)):
        for i, want in enumerate(limits):
            v = got[0, i::4]
            assert ((v == want) | (torch.isnan(v) & (not exact))).all(), (name, i, v)
        assert torch.isfinite(got[0, 3::4]).all()
    assert torch.isnan(y[0, 2::4]).all()
