"""Plain 64-bit forms of the operators around a convolution, written from
their definitions, with a magnitude beside each value: what a sum of its terms
without their signs comes to, so that a tolerance can count roundings.

``within`` holds a computed tensor to a reference: half a step of its type
relative to the value (the one rounding of the output), plus ``n`` roundings
of 2^-24 relative to the magnitude (the fp32 arithmetic before it).
"""
import math

import torch

U32 = 2.0 ** -24
EPS = 1e-6


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def within(name, got, ref, mag, n, also=0.0):
    """|got - ref| <= half a step of |ref| + n 2^-24 mag + also, element by
    element; NaN and infinities must agree.  Half a step of the smallest
    normal covers results below it."""
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    g, r = got.detach().cpu().double(), ref.detach().cpu().double()
    fine = torch.isfinite(r)
    assert torch.equal(torch.isnan(g), torch.isnan(r)), f"{name}: NaN in other places"
    assert torch.equal(g[~fine & ~torch.isnan(r)], r[~fine & ~torch.isnan(r)]), f"{name}: infinities differ"
    m = mag.detach().cpu().double().expand_as(r)
    tol = half_step(got.dtype) * r.abs() + n * U32 * (m + r.abs()) + also + torch.finfo(got.dtype).tiny
    over = ((g - r).abs() / tol)[fine]
    if over.numel():
        worst = over.max().item()
        print(f"  {name}: {worst:.3f} of its tolerance", flush=True)
        assert worst <= 1.0, f"{name}: {worst:.3g} times its tolerance"


def act(v, kind):
    """Value and derivative."""
    one = torch.ones_like(v)
    if kind == "none":
        return v, one
    if kind == "relu":
        return torch.where(v > 0, v, 0 * one), (v > 0).double()
    if kind in ("sigmoid", "silu"):
        p = torch.sigmoid(v)
        return (p, p * (1 - p)) if kind == "sigmoid" else (v * p, p + v * p * (1 - p))
    if kind == "tanh":
        return torch.tanh(v), 1 - torch.tanh(v) ** 2
    if kind == "gelu":
        phi = 0.5 * (1 + torch.erf(v / math.sqrt(2)))
        return v * phi, phi + v * torch.exp(-v * v / 2) / math.sqrt(2 * math.pi)
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (v + 0.044715 * v ** 3))
    return 0.5 * v * (1 + t), 0.5 * (1 + t) + 0.5 * v * (1 - t * t) * c * (1 + 0.134145 * v * v)


def _standard(v, m, kind, eps):
    """Normalised rows, 1/scale and magnitude from values and their magnitude."""
    if kind == "none":
        return v, torch.ones_like(v[..., :1]), m
    mu = v.mean(-1, keepdim=True) if kind == "layer" else torch.zeros_like(v[..., :1])
    r = 1 / torch.sqrt(((v - mu) ** 2).mean(-1, keepdim=True) + eps)
    vh = (v - mu) * r
    # a relative error of the row's scale follows from the values' own
    big = (m + m.mean(-1, keepdim=True)) * r
    return vh, r, big * (1 + vh.abs().amax(-1, keepdim=True))


def _back(q, qm, vh, vm, r, kind):
    """Gradient through a norm and its magnitude."""
    if kind == "none":
        return q, qm
    d = q - vh * (q * vh).mean(-1, keepdim=True)
    if kind == "layer":
        d = d - q.mean(-1, keepdim=True)
    m = qm + vm * (qm * vm).mean(-1, keepdim=True) + qm.mean(-1, keepdim=True)
    return d * r, m * r * (1 + vm.amax(-1, keepdim=True))


def block_norm(x, f=None, z=None, s=None, w_post=None, b_post=None, w_pre=None, b_pre=None, post="none", pre="rms",
               gate_act="none", eps=EPS, dy=None, da=None):
    """Everything in 64 bits from [rows, C] tensors; the gate is given row by
    row.  Returns {name: (value, magnitude)}, gradients too with dy or da."""
    to = lambda t: None if t is None else t.detach().cpu().double()  # noqa: E731
    x, f, z, s, w_post, b_post, w_pre, b_pre, dy, da = map(to, (x, f, z, s, w_post, b_post, w_pre, b_pre, dy, da))
    C = x.shape[-1]
    one = torch.ones(C, dtype=torch.float64)
    s_ = one if s is None else s
    wp, wq = (one if w_post is None else w_post), (one if w_pre is None else w_pre)
    bp, bq = (0 * one if b_post is None else b_post), (0 * one if b_pre is None else b_pre)
    out = {}
    y, ym = x, x.abs()
    if f is not None:
        fh, rf, fm = _standard(f, f.abs(), post, eps)
        n, nm = fh * wp + bp, fm * wp.abs() + bp.abs()
        zv, zd = act(z, gate_act) if z is not None else (one, 0 * one)
        g = s_ * zv
        y, ym = x + g * n, x.abs() + g.abs() * nm
        out["y"] = (y, ym)
    if pre != "none":
        yh, ry, yhm = _standard(y, ym, pre, eps)
        out["a"] = (yh * wq + bq, yhm * wq.abs() + bq.abs())
    if dy is None and da is None:
        return out
    d = torch.zeros_like(x) if dy is None else dy
    dm = d.abs()
    if da is not None:
        q = da * wq
        t, tm = _back(q, q.abs(), yh, yhm, ry, pre)
        d, dm = d + t, dm + tm
        out["dw_pre"] = ((da * yh).sum(0), (da.abs() * yhm).sum(0))
        out["db_pre"] = (da.sum(0), da.abs().sum(0))
    out["dx"] = (d, dm)
    if f is None:
        return out
    P, Pm = d * n, dm * nm
    # the derivative of a saturated activation is a difference of its terms
    zm = zd.abs() + 1.0
    out["dz"] = (P * s_ * zd, Pm * s_.abs() * zm)
    out["ds"] = ((P * zv).sum(0), (Pm * zv.abs()).sum(0))
    dn, dnm = d * g, dm * g.abs()
    out["dw_post"] = ((dn * fh).sum(0), (dnm * fm).sum(0))
    out["db_post"] = (dn.sum(0), dnm.sum(0))
    out["df"] = _back(dn * wp, dnm * wp.abs(), fh, fm, rf, post)
    return out


def gated(x, wg, wu, bg=None, bu=None, kind="silu", dh=None):
    """Forward and, with dh, gradient in 64 bits: {name: (value, magnitude)}."""
    to = lambda t: None if t is None else t.detach().cpu().double()  # noqa: E731
    x, wg, wu, bg, bu, dh = map(to, (x, wg, wu, bg, bu, dh))
    g, u = x @ wg.t(), x @ wu.t()
    gm, um = x.abs() @ wg.abs().t(), x.abs() @ wu.abs().t()
    if bg is not None:
        g, u, gm, um = g + bg, u + bu, gm + bg.abs(), um + bu.abs()
    v, d = act(g, kind)
    # |act'| <= 1.13 for every activation here, and |act| <= |t| or 1
    vm = 1.13 * gm + v.abs()
    out = {"g": (g, gm), "u": (u, um), "h": (v * u, vm * um)}
    if dh is None:
        return out
    dg, du = dh * u * d, dh * v
    # |act''| <= 1.13: an error of g moves act' by as much
    dgm, dum = dh.abs() * um * (d.abs() + 1.13 * gm + 1), dh.abs() * vm
    out["dg"], out["du"] = (dg, dgm), (du, dum)
    out["dx"] = (dg @ wg + du @ wu, dgm @ wg.abs() + dum @ wu.abs())
    out["dwg"], out["dwu"] = (dg.t() @ x, dgm.t() @ x.abs()), (du.t() @ x, dum.t() @ x.abs())
    out["dbg"], out["dbu"] = (dg.sum(0), dgm.sum(0)), (du.sum(0), dum.sum(0))
    # what one more rounding of dg and du (as operands of the products) moves
    dga, dua = dg.abs(), du.abs()
    out["rounded"] = {"dx": dga @ wg.abs() + dua @ wu.abs(), "dwg": dga.t() @ x.abs(), "dwu": dua.t() @ x.abs(),
                      "dbg": dga.sum(0), "dbu": dua.sum(0)}
    return out
