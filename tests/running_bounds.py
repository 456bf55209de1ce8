"""Values in 64 bits that carry a bound on the error of the same arithmetic in
fp32: a running analysis.  Each operation adds one rounding of its result (half
a step of fp32, 2^-24 relative), sums of n terms n - 1 roundings of the sum of
magnitudes, in whatever order; inputs' errors pass through by the derivative.
Errors are in units of 2^-24; second-order terms are covered by a hundredth."""
import math

import torch

U32 = 2.0 ** -24


class B:
    """A value and the bound of its error."""

    def __init__(self, v, e=None):
        self.v = v.detach().cpu().double() if isinstance(v, torch.Tensor) else torch.tensor(float(v), dtype=torch.float64)
        self.e = torch.zeros_like(self.v) if e is None else e

    def __add__(self, o):
        o = o if isinstance(o, B) else B(o)
        v = self.v + o.v
        return B(v, self.e + o.e + v.abs())

    def __mul__(self, o):
        o = o if isinstance(o, B) else B(o)
        v = self.v * o.v
        return B(v, self.e * o.v.abs() + o.e * self.v.abs() + v.abs())

    def __neg__(self):
        return B(-self.v, self.e)

    def __getitem__(self, i):
        return B(self.v[i], self.e[i])

    def sum(self, dim):
        n = self.v.shape[dim]
        return B(self.v.sum(dim), self.e.sum(dim) + max(n - 1, 0) * self.v.abs().sum(dim))

    def exp(self):
        """By the hardware's base-2 exponential (two units: one of the last place)
        of a product with a rounded constant."""
        v = self.v.exp()
        return B(v, v * (self.e + 2 * self.v.abs() + 2))

    def select(self, mask):
        return B(self.v * mask, self.e * mask)


def cat(parts, dim=0):
    return B(torch.cat([p.v for p in parts], dim), torch.cat([p.e for p in parts], dim))


def stack(parts, dim=0):
    return B(torch.stack([p.v for p in parts], dim), torch.stack([p.e for p in parts], dim))


def softplus(a):
    """log(1 + exp(a)) and its derivative.  exp(-|a|) is off by 2 |a| + 2 units
    relative, its quotient with 2 + exp(-|a|) by four more (sum, reciprocal,
    product), the series by four more."""
    v = torch.nn.functional.softplus(a.v, threshold=1e9)
    s = torch.sigmoid(a.v)
    tail = torch.log1p(torch.exp(-a.v.abs()))
    e = a.e * s + tail * (2 * a.v.abs() + 10) + v
    # the derivative's own slope is s (1 - s)
    return B(v, e), B(s, a.e * s * (1 - s) + s * (2 * a.v.abs() + 6))


def act(a, kind):
    """An activation and its derivative: exponentials as above, a reciprocal and
    a few products (12 units beside the exponential's)."""
    x = a.v
    if kind == "none":
        return a, B(torch.ones_like(x))
    if kind == "relu":
        return B(x.clamp(min=0), a.e * (x > 0)), B((x > 0).double())
    if kind in ("gelu", "gelu_tanh"):
        return gelu(a, kind)
    p = torch.sigmoid(x)
    if kind == "sigmoid":
        v, d, dd = p, p * (1 - p), p
    elif kind == "silu":
        v, d, dd = x * p, p + x * p * (1 - p), torch.ones_like(x)
    elif kind == "tanh":
        v = torch.tanh(x)
        d, dd = 1 - v * v, torch.ones_like(x)
    else:
        raise ValueError(kind)
    n = 2 * x.abs() + 12
    return B(v, a.e * d.abs() + n * v.abs()), B(d, a.e * dd + n * (d.abs() + dd))


def gelu(a, kind):
    """Both forms of it, and their derivatives.

    The normal distribution's tail is exp(-t^2 / 2) times a fitted polynomial in a
    reciprocal: the exponent's three roundings move the exponential by 3 t^2 / 2 units
    relative, itself two more; fit (2), reciprocal (2), eight multiply-adds (their terms
    cancel to a third at worst) and products: 40 in all.  t Phi(t) is max(t, 0) less |t|
    times the tail.

    The tanh form is t times the logistic function of w = 2 k (t + c t^3): six
    roundings of w, the exponential's two |w| / 2 and two more, sum and reciprocal
    come to (1 - p) 8 |w| + 4 units relative.

    Exponentials and reciprocals below 2^-126 are zeros: off by that much, times what
    they are multiplied by."""
    t = a.v
    least = 2.0 ** -126 / U32 * (1 + t.abs())
    if kind == "gelu":
        tail = torch.erfc(t.abs() * math.sqrt(0.5)) / 2
        p, dense = torch.where(t < 0, tail, 1 - tail), torch.exp(-t * t / 2) / math.sqrt(2 * math.pi)
        n = 1.5 * t * t + 40
        v, d = t * p, p + t * dense
        ev = t.abs() * tail * n + v.abs() + t.abs() * tail + least
        ed = tail * n + (t * dense).abs() * n + 2 * (p + (t * dense).abs()) + least
    else:
        k, c = math.sqrt(2 / math.pi), 0.044715
        w = 2 * k * (t + c * t ** 3)
        p, slope = torch.sigmoid(w), 2 * k * (1 + 3 * c * t * t)
        n = torch.sigmoid(-w) * 8 * w.abs() + 4
        second = t * p * torch.sigmoid(-w) * slope
        v, d = t * p, p + second
        ev = v.abs() * (n + 2) + least
        # 1 - p is off by what p is, and a rounding
        ed = p * n + (t * p * slope).abs() * (p * n + 1) * (w.abs() < 25) + second.abs() * (n + 8) + p + second.abs() + least * (1 + slope)
    # both second derivatives stay below 1
    return B(v, a.e * d.abs() + ev), B(d, a.e + ed)


def within(name, got, want, also=0.0):
    """|got - want| <= half a step of the type of ``got`` relative to the value,
    the bound of the arithmetic before it, and the smallest normal number."""
    g, r = got.detach().cpu().double(), want.v
    assert g.shape == r.shape, (name, g.shape, r.shape)
    assert torch.isfinite(g).all(), f"{name}: not finite"
    tol = torch.finfo(got.dtype).eps / 2 * (r.abs() + U32 * want.e) + 1.01 * U32 * want.e + torch.finfo(got.dtype).tiny + also
    if g.numel():
        worst = ((g - r).abs() / tol).max().item()
        print(f"  {name}: {worst:.3f} of its tolerance (largest {math.sqrt((r * r).mean().item()):.2g} rms)", flush=True)
        assert worst <= 1.0, f"{name}: {worst:.3g} times its tolerance"
