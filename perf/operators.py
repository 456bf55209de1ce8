"""Cases that measure the block operators: the gated feed-forward layer, the
norms around a block, and the global gradient norm with clipping.

``run`` computes one pass: with ``own`` false in elementary torch operations
in 32 bits, with ``own`` true through the package.  ``exact`` gives the same
outputs in 64 bits from the definitions.
"""
from __future__ import annotations

import math
import random

import torch

own = False

BF16, F32 = "bf16", "fp32"
TYPES = {BF16: torch.bfloat16, F32: torch.float32}
ACTS = ("none", "sigmoid", "silu", "gelu", "gelu_tanh", "relu", "tanh")
EPS = 1e-6
CLIP_EPS = 1e-6


def listed():
    return [
        # One token through a gated layer: serving, a stream of two weights.
        dict(name="gated_token", op="gated", rows=1, channels=2048, hidden=8192, dtype=BF16, act="silu",
             bias=False, train=False, keep=False),
        # A small ragged batch of requests, a hidden width that fits no tile.
        dict(name="gated_batch37", op="gated", rows=37, channels=1000, hidden=2730, dtype=BF16, act="gelu_tanh",
             bias=True, train=False, keep=False),
        # The pixels of 32 maps of 56x56 at 256 channels: a gated 1x1 layer's inference.
        dict(name="gated_image", op="gated", rows=32 * 56 * 56, channels=256, hidden=1024, dtype=BF16, act="gelu",
             bias=True, train=False, keep=False),
        # The same layer's training step at 28x28, pre-activations computed again in the backward pass.
        dict(name="gated_train_image", op="gated", rows=32 * 28 * 28, channels=256, hidden=1024, dtype=BF16,
             act="silu", bias=True, train=True, keep=False),
        # A wide layer's training step over a long batch of tokens, pre-activations kept.
        dict(name="gated_train_tokens", op="gated", rows=8192, channels=4096, hidden=8192, dtype=BF16, act="silu",
             bias=False, train=True, keep=True),
        # An fp32 training step, no size a multiple of a tile or a vector.
        dict(name="gated_train_fp32", op="gated", rows=1001, channels=190, hidden=517, dtype=F32, act="sigmoid",
             bias=True, train=True, keep=False),
        # One token between two blocks: latency.
        dict(name="norm_token", op="norm", rows=1, channels=4096, dtype=BF16, pre="rms", post="rms", gate="none",
             act="none", scale=False, train=False),
        # 32 maps of 56x56 between two blocks, one gate an image, a residual scale a channel.
        dict(name="norm_image", op="norm", rows=32 * 56 * 56, channels=256, dtype=BF16, pre="layer", post="layer",
             gate="image", images=32, act="sigmoid", scale=True, train=False),
        # A long batch of tokens, gated element by element: the training step.
        dict(name="norm_train_tokens", op="norm", rows=16384, channels=4096, dtype=BF16, pre="rms", post="rms",
             gate="full", act="silu", scale=True, train=True),
        # An fp32 training step with odd sizes and one gate an image.
        dict(name="norm_train_fp32", op="norm", rows=1239, channels=1001, dtype=F32, pre="layer", post="layer",
             gate="image", images=7, act="sigmoid", scale=True, train=True),
        # The gradients of a few convolution layers: launches count.
        dict(name="clip_layers", op="clip", tensors=12, total=700_001, spread=6.0, dtype="mixed", max_norm=1.0),
        # The gradients of a whole model, a few large and many small.
        dict(name="clip_model", op="clip", tensors=290, total=300_000_003, spread=9.0, dtype="mixed", max_norm=1.0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(("gated", "gated", "norm", "norm", "clip"))
    if op == "gated":
        while True:
            rows, channels, hidden = _log(rng, 1, 100_352), _log(rng, 16, 4096), _log(rng, 16, 8192)
            if rng.random() < 0.6:
                channels, hidden = -(-channels // 8) * 8, -(-hidden // 8) * 8
            train = rng.random() < 0.5
            dtype = F32 if rng.random() < 0.25 else BF16
            cost = rows * channels * hidden * (1 if dtype == BF16 else 16)
            if cost <= 8192 * 4096 * 8192 and rows * hidden <= 32 * 56 * 56 * 1024:
                return dict(op=op, rows=rows, channels=channels, hidden=hidden, dtype=dtype, act=rng.choice(ACTS[1:]),
                            bias=rng.random() < 0.5, train=train, keep=train and rng.random() < 0.5)
    if op == "norm":
        while True:
            rows, channels = _log(rng, 1, 200_000), _log(rng, 8, 16_384)
            if rng.random() < 0.6:
                channels = -(-channels // 8) * 8
            if rows * channels <= 16384 * 4096:
                break
        gate = rng.choice(("none", "image", "full"))
        images = 1
        if gate == "image":
            images = _log(rng, 1, min(rows, 64))
            rows = rows // images * images
        return dict(op=op, rows=rows, channels=channels, dtype=rng.choice((BF16, BF16, F32)),
                    pre=rng.choice(("rms", "layer")), post=rng.choice(("none", "rms", "layer")), gate=gate,
                    images=images, act=rng.choice(("none", "sigmoid", "silu", "tanh")), scale=rng.random() < 0.5,
                    train=rng.random() < 0.5)
    tensors = _log(rng, 1, 600)
    return dict(op=op, tensors=tensors, total=max(tensors, _log(rng, 1000, 300_000_000)), spread=rng.uniform(1.0, 10.0),
                dtype=rng.choice((BF16, F32, "mixed")), max_norm=1.0)


# ------------------------------------------------------------------ inputs --

def _sizes(case):
    """Element counts of a list of gradients: log-uniform, at least one each."""
    n, total = case["tensors"], case["total"]
    r = random.Random(n * 1_000_003 + total)
    w = [math.exp(r.uniform(0.0, case["spread"])) for _ in range(n)]
    left = total - n
    s = sum(w)
    sizes = [1 + int(left * v / s) for v in w]
    sizes[0] += total - sum(sizes)
    return sizes


def _clip_types(case):
    kinds = {BF16: (torch.bfloat16,), F32: (torch.float32,), "mixed": (torch.bfloat16, torch.float32, torch.bfloat16)}
    k = kinds[case["dtype"]]
    return [k[i % len(k)] for i in range(case["tensors"])]


class _Maker:
    def __init__(self, seed, dtype):
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        self.dtype = dtype

    def __call__(self, *shape, std=1.0, mean=0.0, dtype=None):
        t = torch.empty(shape, device="cuda").normal_(mean, std, generator=self.gen)
        return t.to(dtype or self.dtype)


def prepare(case, seed):
    s = {"case": case}
    if case["op"] == "gated":
        m, c, f = case["rows"], case["channels"], case["hidden"]
        make = _Maker(seed, TYPES[case["dtype"]])
        s["x"] = make(m, c)
        s["wg"], s["wu"] = make(f, c, std=c ** -0.5), make(f, c, std=c ** -0.5)
        s["bg"], s["bu"] = (make(f, std=0.1), make(f, std=0.1)) if case["bias"] else (None, None)
        if case["train"]:
            s["dh"] = make(m, f)
        return s
    if case["op"] == "norm":
        m, c = case["rows"], case["channels"]
        make = _Maker(seed, TYPES[case["dtype"]])
        # x is the residual stream (wide), f a block's output (with an offset a channel).
        s["x"], s["f"] = make(m, c, std=2.0), make(m, c, std=0.5, mean=0.1)
        s["w_pre"] = make(c, std=0.1, mean=1.0)
        s["b_pre"] = make(c, std=0.1) if case["pre"] == "layer" else None
        s["w_post"] = make(c, std=0.1, mean=1.0) if case["post"] != "none" else None
        s["b_post"] = make(c, std=0.1) if case["post"] == "layer" else None
        s["s"] = make(c, std=0.05, mean=0.2) if case["scale"] else None
        s["z"] = {"none": None, "image": (case.get("images", 1), c), "full": (m, c)}[case["gate"]]
        if s["z"] is not None:
            s["z"] = make(*s["z"])
        if case["gate"] == "image":  # rows of one image share its gate
            s["x"], s["f"] = (t.view(case["images"], -1, c) for t in (s["x"], s["f"]))
        if case["train"]:
            s["dy"], s["da"] = make(*s["x"].shape), make(*s["x"].shape)
        return s
    make = _Maker(seed, torch.float32)
    s["grads"] = [make(n, std=0.01, dtype=t) for n, t in zip(_sizes(case), _clip_types(case))]
    # The optimizer's gradient buffers: one flat buffer a type, each tensor
    # from a multiple of 256 bytes on.
    s["flat"], s["out"] = _flat(case)
    return s


def _flat(case, dtype=None):
    sizes, types = _sizes(case), _clip_types(case)
    ends, starts = {}, []
    for n, t in zip(sizes, types):
        starts.append(ends.get(t, 0))
        ends[t] = starts[-1] + -(-n // 128) * 128
    flat = {t: torch.zeros(n, dtype=dtype or t, device="cuda") for t, n in ends.items()}
    out = [flat[t][i:i + n] for n, t, i in zip(sizes, types, starts)]
    return flat, out


# -------------------------------------------------------------- plain form --

def _act(v, kind):
    """Value and derivative of an activation."""
    if kind == "none":
        return v, torch.ones_like(v)
    if kind == "relu":
        on = (v > 0).to(v.dtype)
        return v * on, on
    if kind == "sigmoid":
        p = 1 / (1 + torch.exp(-v))
        return p, p * (1 - p)
    if kind == "silu":
        p = 1 / (1 + torch.exp(-v))
        return v * p, p * (1 + v * (1 - p))
    if kind == "tanh":
        t = torch.tanh(v)
        return t, 1 - t * t
    if kind == "gelu":
        p = 0.5 * (1 + torch.erf(v * math.sqrt(0.5)))
        return v * p, p + v * torch.exp(-0.5 * v * v) / math.sqrt(2 * math.pi)
    k = math.sqrt(2 / math.pi)
    t = torch.tanh(k * (v + 0.044715 * v * v * v))
    return 0.5 * v * (1 + t), 0.5 * (1 + t) + 0.5 * v * (1 - t * t) * k * (1 + 3 * 0.044715 * v * v)


def _plain_gated(s):
    case, out = s["case"], s["x"].dtype
    x, wg, wu = s["x"].float(), s["wg"].float(), s["wu"].float()
    g, u = x @ wg.t(), x @ wu.t()
    if case["bias"]:
        g, u = g + s["bg"].float(), u + s["bu"].float()
    v, d = _act(g, case["act"])
    h = (v * u).to(out)
    if not case["train"]:
        return {"h": h}
    dh = s["dh"].float()
    dg, du = dh * u * d, dh * v
    r = {"h": h, "dx": (dg @ wg + du @ wu).to(out), "dwg": (dg.t() @ x).to(out), "dwu": (du.t() @ x).to(out)}
    if case["bias"]:
        r["dbg"], r["dbu"] = dg.sum(0).to(out), du.sum(0).to(out)
    return r


def _normed(v, kind):
    """The normalised rows and the reciprocal of their scale."""
    if kind == "layer":
        v = v - v.mean(-1, keepdim=True)
    r = 1 / torch.sqrt((v * v).mean(-1, keepdim=True) + EPS)
    return v * r, r


def _normed_grad(q, vh, r, kind):
    t = q - vh * (q * vh).mean(-1, keepdim=True)
    if kind == "layer":
        t = t - q.mean(-1, keepdim=True)
    return t * r


def _plain_norm(s):
    case, out = s["case"], s["x"].dtype
    c = case["channels"]
    x, f = s["x"].float(), s["f"].float()
    if case["post"] != "none":
        fh, rf = _normed(f, case["post"])
        n = fh * s["w_post"].float()
        if s["b_post"] is not None:
            n = n + s["b_post"].float()
    else:
        n = f
    scale = s["s"].float() if s["s"] is not None else torch.ones(c, device=x.device)
    z = None
    if s["z"] is not None:
        z = s["z"].float()
        z = z[:, None, :] if case["gate"] == "image" else z
        zv, zd = _act(z, case["act"])
        factor = scale * zv
    else:
        factor = scale
    y = x + factor * n
    yh, ry = _normed(y, case["pre"])
    a = yh * s["w_pre"].float()
    if s["b_pre"] is not None:
        a = a + s["b_pre"].float()
    r = {"y": y.to(out), "a": a.to(out)}
    if not case["train"]:
        return r
    rows = tuple(range(x.dim() - 1))
    dy, da = s["dy"].float(), s["da"].float()
    d = dy + _normed_grad(da * s["w_pre"].float(), yh, ry, case["pre"])
    r["dx"] = d.to(out)
    r["dw_pre"] = (da * yh).sum(rows).to(out)
    if s["b_pre"] is not None:
        r["db_pre"] = da.sum(rows).to(out)
    p = d * n
    if z is not None:
        dz = p * scale * zd
        r["dz"] = (dz.sum(1) if case["gate"] == "image" else dz).to(out)
    if s["s"] is not None:
        r["ds"] = (p * zv if z is not None else p).sum(rows).to(out)
    dn = d * factor
    if case["post"] != "none":
        r["dw_post"] = (dn * fh).sum(rows).to(out)
        if s["b_post"] is not None:
            r["db_post"] = dn.sum(rows).to(out)
        dn = _normed_grad(dn * s["w_post"].float(), fh, rf, case["post"])
    r["df"] = dn.to(out)
    return r


def _plain_clip(s):
    total = torch.stack([g.float().square().sum(dtype=torch.float64) for g in s["grads"]]).sum()
    norm = total.sqrt().float()
    c = (s["case"]["max_norm"] / (norm + CLIP_EPS)).clamp(max=1.0)
    [o.copy_(g.float() * c) for g, o in zip(s["grads"], s["out"])]
    return _clipped(norm, s["flat"])


def _clipped(norm, flat):
    """The norm and the buffers of the clipped gradients."""
    return {"norm": norm, **{str(t): v for t, v in flat.items()}}


# --------------------------------------------------------------- one pass --

def run(state):
    case = state["case"]
    if not own:
        return {"gated": _plain_gated, "norm": _plain_norm, "clip": _plain_clip}[case["op"]](state)
    import convolution_implicit_gemm_conv2d_amd as cm

    s = state
    if case["op"] == "gated":
        kept = None
        if case["keep"]:
            kept = torch.empty(case["rows"], 2 * case["hidden"], dtype=torch.float32, device=s["x"].device)
        h = cm.gated_feed_forward(s["x"], s["wg"], s["wu"], s["bg"], s["bu"], activation=case["act"], saved=kept)
        if not case["train"]:
            return {"h": h}
        dx, dwg, dwu, dbg, dbu = cm.gated_feed_forward_grad(s["dh"], s["x"], s["wg"], s["wu"], s["bg"], s["bu"],
                                                            activation=case["act"], saved=kept)
        r = {"h": h, "dx": dx, "dwg": dwg, "dwu": dwu}
        if case["bias"]:
            r["dbg"], r["dbu"] = dbg, dbu
        return r
    if case["op"] == "norm":
        how = dict(gate=s["z"], scale=s["s"], post_weight=s["w_post"], post_bias=s["b_post"], pre_weight=s["w_pre"],
                   pre_bias=s["b_pre"], post=case["post"], pre=case["pre"], gate_activation=case["act"], eps=EPS)
        y, a = cm.block_norm(s["x"], s["f"], **how)
        r = {"y": y, "a": a}
        if not case["train"]:
            return r
        d = cm.block_norm_grad(s["dy"], s["da"], s["x"], s["f"], **how)
        names = dict(dx="x", df="branch", dz="gate", ds="scale", dw_post="post_weight", db_post="post_bias",
                     dw_pre="pre_weight", db_pre="pre_bias")
        r.update({k: d[v] for k, v in names.items() if d[v] is not None})
        return r
    norm = cm.clip_gradients(s["grads"], case["max_norm"], out=s["out"], eps=CLIP_EPS)
    return _clipped(norm, s["flat"])


def work(case):
    e = 2 if case.get("dtype") == BF16 else 4
    if case["op"] == "gated":
        m, c, f = case["rows"], case["channels"], case["hidden"]
        values, flops = m * c + 2 * f * c + m * f, 4 * m * f * c
        if case["train"]:
            values, flops = values + m * f + m * c + 2 * f * c, flops + 8 * m * f * c
        return {"bytes": e * values, "flops": flops}
    if case["op"] == "norm":
        n = case["rows"] * case["channels"]
        full = 1 if case["gate"] == "full" else 0
        values, flops = 4 + full, 20
        if case["train"]:  # dy, da read; dx, df (and dz) written
            values, flops = values + 4 + full, 70
        return {"bytes": e * n * values, "flops": flops * n}
    total = sum(n * (2 if t == torch.bfloat16 else 4) for n, t in zip(_sizes(case), _clip_types(case)))
    return {"bytes": 2 * total, "flops": 3 * case["total"]}


# ----------------------------------------------------------------- 64 bits --

def _act64(v, kind):
    fn = {"none": lambda t: t, "sigmoid": torch.sigmoid, "silu": torch.nn.functional.silu, "relu": torch.relu,
          "tanh": torch.tanh, "gelu": torch.nn.functional.gelu,
          "gelu_tanh": lambda t: torch.nn.functional.gelu(t, approximate="tanh")}
    return fn[kind](v)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "clip":
        norm = math.sqrt(sum(float(torch.dot(g.double(), g.double())) for g in s["grads"]))
        c = min(1.0, case["max_norm"] / (norm + CLIP_EPS))
        flat, out = _flat(case, torch.float64)
        [o.copy_(g.double() * c) for g, o in zip(s["grads"], out)]
        return _clipped(torch.tensor(norm, dtype=torch.float64, device="cuda"), flat)
    leaf = {k: t.double().requires_grad_(case["train"]) for k, t in s.items()
            if isinstance(t, torch.Tensor) and k not in ("dh", "dy", "da")}
    if case["op"] == "gated":
        g = torch.nn.functional.linear(leaf["x"], leaf["wg"], leaf.get("bg"))
        u = torch.nn.functional.linear(leaf["x"], leaf["wu"], leaf.get("bu"))
        r = {"h": _act64(g, case["act"]) * u}
        loss = [(r["h"], s["dh"])] if case["train"] else []
    else:
        def norm(v, kind, w, b):
            if kind == "none":
                return v
            mean = v.mean(-1, keepdim=True) if kind == "layer" else 0.0
            var = ((v - mean) ** 2).mean(-1, keepdim=True)
            v = (v - mean) / (var + EPS) ** 0.5 * w
            return v if b is None else v + b

        n = norm(leaf["f"], case["post"], leaf.get("w_post"), leaf.get("b_post"))
        if "s" in leaf:
            n = n * leaf["s"]
        if "z" in leaf:
            z = _act64(leaf["z"], case["act"])
            n = n * (z.unsqueeze(1) if case["gate"] == "image" else z)
        y = leaf["x"] + n
        a = norm(y, case["pre"], leaf["w_pre"], leaf.get("b_pre"))
        r = {"y": y, "a": a}
        loss = [(y, s["dy"]), (a, s["da"])] if case["train"] else []
    if loss:
        names = list(leaf)
        got = torch.autograd.grad([o for o, _ in loss], [leaf[k] for k in names], [d.double() for _, d in loss])
        r.update({"d" + k: v for k, v in zip(names, got)})
    return {k: v.detach() for k, v in r.items()}
