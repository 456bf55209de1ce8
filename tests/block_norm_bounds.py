"""How far the block norms' kernels may be from the 64-bit values: a running
analysis of their fp32 arithmetic, to first order, with the values at hand.

Each quantity is a pair (v, e): its value in 64 bits and a bound of its absolute
error in units of 2^-24.  An operation's result is off by what its operands bring
with it and by |v| for its own rounding; a sum of terms one after another, over a
chain of s additions, by s times the sum of their magnitudes.  No magnitude is
taken over a row's largest values, so that a gradient of zeros, or one that lacks
a row's term, is far outside.

A row's sum is a chain of at most 16 channels of a lane (C / 512 in a long row's
walk), 6 steps of a wave and 8 for 16 waves.  A column's is a chain over the rows
of a piece, at most 2 rows / 200 + 10, 7 over a workgroup and, for at most 1024
pieces, 80 for the pieces' partials.
"""
import torch

import block_reference as br

EPS = br.EPS


def exact(t):
    return t, torch.zeros_like(t)


def mul(a, b):
    v = a[0] * b[0]
    return v, a[1] * b[0].abs() + a[0].abs() * b[1] + v.abs()


def add(a, b):
    v = a[0] + b[0]
    return v, a[1] + b[1] + v.abs()


def sub(a, b):
    return add(a, (-b[0], b[1]))


def row_mean(a, chain):
    v, m = a[0].mean(-1, keepdim=True), a[0].abs().mean(-1, keepdim=True)
    return v, a[1].mean(-1, keepdim=True) + (chain + 2) * m


def column_sum(a, chain):
    return a[0].sum(-2), a[1].sum(-2) + chain * a[0].abs().sum(-2)


def activation(z, kind):
    """The activation and its derivative: no more than 16 roundings of values that
    |act|, |act'| and the argument bound."""
    v, d = br.act(z, kind)
    e = 0.0 if kind == "none" else 16 * (1 + z.abs())
    return (v, torch.zeros_like(v) + e), (d, torch.zeros_like(d) + e)


def standard(a, kind, eps, chain):
    """Normalised rows and the reciprocal of their scale."""
    if kind == "layer":
        a = sub(a, row_mean(a, chain))
    v, e = row_mean(mul(a, a), chain)
    v, e = v + eps, e + v + eps
    r = v ** -0.5
    r = r, r * (0.5 * e / v + 4)
    return mul(a, r), r


def back(q, vh, r, kind, chain):
    """Gradient through a norm."""
    t = sub(q, row_mean(q, chain)) if kind == "layer" else q
    return mul(sub(t, mul(vh, row_mean(mul(q, vh), chain))), r)


def gradients(dy, da, x, f=None, z=None, s=None, w_post=None, b_post=None, w_pre=None, b_pre=None, post="none", pre="rms",
              gate_act="none", eps=EPS):
    """{name: (value, error)} from [rows, C] tensors; `z` is [images, C] (or has a
    row for each), its gradient summed over each image's rows."""
    to = lambda t: None if t is None else exact(t.detach().cpu().double())  # noqa: E731
    x, f, s, w_post, b_post, w_pre, dy, da = map(to, (x, f, s, w_post, b_post, w_pre, dy, da))
    rows, C = x[0].shape
    one = exact(torch.ones(C, dtype=torch.float64))
    row, column = 30 + C // 512, 2 * rows // 200 + 10 + 7 + 80
    wp, wq, s = w_post or one, w_pre or one, s or one
    out, y = {}, x
    if f is not None:
        fh, rf = standard(f, post, eps, row) if post != "none" else (f, None)
        n = mul(fh, wp)
        n = add(n, b_post) if b_post is not None else n
        zv, zd = one, None
        if z is not None:
            z = z.detach().cpu().double()
            zv, zd = activation(z.repeat_interleave(rows // z.shape[0], 0), gate_act)
        g = mul(s, zv)
        y = add(x, mul(g, n))
    d = dy if dy is not None else exact(torch.zeros_like(x[0]))
    if da is not None:
        yh, ry = standard(y, pre, eps, row)
        d = add(d, back(mul(da, wq), yh, ry, pre, row))
        out["pre_weight"] = column_sum(mul(da, yh), column)
        out["pre_bias"] = column_sum(da, column)
    out["x"] = d
    if f is None:
        return out
    P = mul(d, n)
    if z is not None:
        dz = mul(P, mul(s, zd))
        if z.shape[0] < rows:
            k = z.shape[0]
            dz = column_sum(tuple(t.reshape(k, rows // k, C) for t in dz), column)
        out["gate"] = dz
    out["scale"] = column_sum(mul(P, zv), column)
    dn = mul(d, g)
    out["post_weight"] = column_sum(mul(dn, fh), column)
    out["post_bias"] = column_sum(dn, column)
    p = mul(dn, wp)
    out["branch"] = back(p, fh, rf, post, row) if post != "none" else p
    return out


def off(got, want):
    """The largest error as a share of its tolerance: half a step of the type
    relative to the value, and the fp32 arithmetic's bound, with a tenth for what
    the first order leaves out."""
    v, e = want
    g = got.detach().cpu().double().reshape(v.shape)
    tol = br.half_step(got.dtype) * (v.abs() + 1.1 * br.U32 * e) + 1.1 * br.U32 * e + torch.finfo(got.dtype).tiny
    return ((g - v).abs() / tol).max().item()
