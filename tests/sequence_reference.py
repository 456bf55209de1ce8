"""The operators along a sequence row by row, in 64 bits with running bounds,
written from their definitions.  Sequences are lists of (first row, end)."""
import torch

from running_bounds import B, act, cat, softplus, stack


def spans_of(rows, seqs=None, starts=None):
    if starts is None:
        one = rows // seqs
        return [(i * one, (i + 1) * one) for i in range(seqs)]
    return list(zip(starts[:-1], starts[1:]))


def causal(x, w, b, kind, spans, initial=None, dy=None, dlast=None):
    """x [rows, C], w [C, K], initial [S, K - 1, C]: {name: B}, rows of no sequence zero."""
    rows, C = x.shape
    K = w.shape[1]
    xb, wb = B(x), B(w)
    bias = B(b) if b is not None else B(torch.zeros(C))
    r, y, dx, di, last = {}, [], [], [], []
    zero = lambda n: B(torch.zeros(n, C))  # noqa: E731
    dw, db = [], []
    at = 0
    for s, (f, e) in enumerate(spans):
        line = cat([B(initial[s]) if initial is not None else zero(K - 1), xb[f:e]])
        last.append(line[line.v.shape[0] - (K - 1):])
        n = e - f
        win = stack([line[k:k + n] for k in range(K)], 2)  # [n, C, K]
        terms = cat([win * wb, B(bias.v.expand(n, C))[..., None]], 2)
        pre = terms.sum(2)
        v, d = act(pre, kind)
        y += [zero(f - at), v]
        if dy is not None:
            dp = B(dy[f:e]) * d
            parts = []
            for j in range(n + K - 1):  # position j - (K - 1) of the sequence
                ts = [(j - k, k) for k in range(K) if 0 <= j - k < n]
                p = [dp[t] * wb[:, k] for t, k in ts]
                if dlast is not None and j >= n:
                    p.append(B(dlast[s][j - n]))
                parts.append(stack(p).sum(0) if p else B(torch.zeros(C)))
            g = stack(parts)
            di.append(g[:K - 1])
            dx += [zero(f - at), g[K - 1:]]
            dw.append(dp[..., None] * win)
            db.append(dp)
        at = e
    r["y"] = cat(y + [zero(rows - at)])
    r["last"] = stack(last)
    if dy is not None:
        r["x"] = cat(dx + [zero(rows - at)])
        r["weight"], r["bias"], r["initial"] = cat(dw).sum(0), cat(db).sum(0), stack(di)
    return r


def scan(x, delta, A, Bm, C, D, z, bias, plus, kind, spans, initial=None, dy=None, dlast=None):
    """x, delta, z [rows, C], Bm and C [rows, G, N], A [C, N]: {name: B}."""
    rows, ch = x.shape
    N, G = A.shape[1], Bm.shape[1]
    per = ch // G
    xb, Ab = B(x), B(A)
    raw = B(delta) + (B(bias) if bias is not None else B(torch.zeros(ch)))
    d, slope = softplus(raw) if plus else (raw, B(torch.ones(rows, ch)))
    wide = lambda t: B(t).v.repeat_interleave(per, 1)  # noqa: E731
    Bw, Cw = B(wide(Bm)), B(wide(C))
    arg = d[..., None] * Ab
    a = arg.exp()
    dx = d * xb
    b = dx[..., None] * Bw
    skip = B(D) if D is not None else B(torch.zeros(ch))
    zv, zd = act(B(z), kind) if z is not None else (None, None)
    none = B(torch.zeros(ch, N))
    hs, before, last, real = [none] * rows, [none] * rows, [], torch.zeros(rows, 1, dtype=torch.float64)
    for s, (f, e) in enumerate(spans):
        h = B(initial[s]) if initial is not None else none
        for t in range(f, e):
            before[t] = h
            h = a[t] * h + b[t]
            hs[t] = h
        last.append(h)
        real[f:e] = 1
    hs, before = (stack(v) if rows else B(torch.zeros(0, ch, N)) for v in (hs, before))
    core = cat([hs * Cw, (skip * xb)[..., None]], 2).sum(2)
    r = {"y": (core * zv if zv is not None else core).select(real), "last": stack(last)}
    if dy is None:
        return r
    g = B(dy).select(real)
    if zv is not None:
        r["z"] = g * core * zd
        g = g * zv
    from_y = g[..., None] * Cw
    G_, di = [none] * rows, []
    for s, (f, e) in enumerate(spans):
        carry = B(dlast[s]) if dlast is not None else none
        for t in range(e - 1, f - 1, -1):
            G_[t] = from_y[t] + carry
            carry = G_[t] * a[t]
        di.append(carry)
    G_ = stack(G_) if rows else B(torch.zeros(0, ch, N))
    q = G_ * a * before
    r["A"] = (d[..., None] * q).sum(0)
    w = (G_ * Bw).sum(2)
    dd = ((q * Ab).sum(2) + w * xb) * slope
    r["delta"], r["delta_bias"] = dd.select(real), dd.select(real).sum(0)
    r["x"] = (w * d + skip * g).select(real)
    r["D"] = (g * xb).sum(0)
    fold = lambda t: B(t.v.view(rows, G, per, N), t.e.view(rows, G, per, N)).sum(2)  # noqa: E731
    r["B"], r["C"] = fold((G_ * dx[..., None]).select(real[..., None])), fold(hs * g[..., None])
    r["initial"] = stack(di)
    return r
