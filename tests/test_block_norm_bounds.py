"""The bounds that the block norms' gradients are held to (CPU): they hold the
64-bit values rounded once and the same formulas in 32 bits, and they refuse zeros
and sums that lack one row."""
import pytest
import torch

import block_norm_bounds as bounds
import block_reference as br

BF16, F32 = torch.bfloat16, torch.float32


def make(seed, rows, C, dtype, post, pre, gate, images):
    gen = torch.Generator().manual_seed(seed)

    def t(*shape, std=1.0, mean=0.0):
        return (torch.randn(shape, generator=gen) * std + mean).to(dtype)

    d = dict(x=t(rows, C, std=2.0), f=t(rows, C, std=0.5, mean=0.3), s=t(C, std=0.3, mean=0.5),
             w_post=t(C, mean=1.0, std=0.2) if post != "none" else None, b_post=t(C, std=0.2) if post == "layer" else None,
             w_pre=t(C, mean=1.0, std=0.2), b_pre=t(C, std=0.2) if pre == "layer" else None,
             z={"none": None, "full": (rows, C), "image": (images, C)}[gate])
    if d["z"] is not None:
        d["z"] = t(*d["z"])
    return d, t(rows, C), t(rows, C)


def in_32_bits(d, dy, da, post, pre, kind, images):
    """Gradients by automatic differentiation of the same formulas in fp32."""
    leaf = {k: v.float().requires_grad_() for k, v in d.items() if v is not None}
    rows = d["x"].shape[0]

    def norm(v, kind, w, b):
        if kind == "none":
            return v
        v = v - v.mean(-1, keepdim=True) if kind == "layer" else v
        v = v / (v.pow(2).mean(-1, keepdim=True) + bounds.EPS).sqrt() * w
        return v if b is None else v + b

    n = norm(leaf["f"], post, leaf.get("w_post"), leaf.get("b_post")) * leaf["s"]
    if "z" in leaf:
        v = {"sigmoid": torch.sigmoid, "silu": torch.nn.functional.silu}[kind](leaf["z"])
        n = n * v.repeat_interleave(rows // v.shape[0], 0)
    y = leaf["x"] + n
    a = norm(y, pre, leaf["w_pre"], leaf.get("b_pre"))
    names = dict(x="x", f="branch", z="gate", s="scale", w_post="post_weight", b_post="post_bias", w_pre="pre_weight", b_pre="pre_bias")
    g = torch.autograd.grad((y * dy.float()).sum() + (a * da.float()).sum(), list(leaf.values()))
    return {names[k]: v for k, v in zip(leaf, g)}


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,images,C,post,pre,gate,kind", [
    (4203, 3, 200, "rms", "rms", "none", "none"), (4203, 3, 520, "layer", "rms", "image", "silu"),
    (530, 5, 8192, "layer", "layer", "full", "sigmoid"), (12, 3, 1000, "layer", "layer", "image", "sigmoid"),
    (2103, 3, 1500, "none", "layer", "full", "silu"), (300, 1, 5, "rms", "layer", "image", "silu")])
def test_bounds_refuse_what_is_wrong(rows, images, C, post, pre, gate, kind, dtype):
    d, dy, da = make(rows + C, rows, C, dtype, post, pre, gate, images)
    how = dict(post=post, pre=pre, gate_act=kind)
    ref = bounds.gradients(dy, da, **d, **how)
    plain = br.block_norm(d["x"], d["f"], None if d["z"] is None else d["z"].repeat_interleave(rows // d["z"].shape[0], 0), d["s"],
                          d["w_post"], d["b_post"], d["w_pre"], d["b_pre"], post, pre, kind, dy=dy, da=da)
    same = in_32_bits(d, dy, da, post, pre, kind, images)
    short = {"x": "dx", "branch": "df", "scale": "ds", "post_weight": "dw_post", "post_bias": "db_post", "pre_weight": "dw_pre",
             "pre_bias": "db_pre"}
    for name, want in ref.items():
        value = want[0]
        if name in short:  # the two 64-bit forms agree
            assert torch.allclose(value, plain[short[name]][0], rtol=1e-9, atol=1e-9), name
        assert bounds.off(value.to(dtype), want) <= 1.0, name
        if name in same:
            assert bounds.off(same[name].to(dtype), want) <= 1.0, (name, bounds.off(same[name].to(dtype), want))
        assert bounds.off(torch.zeros_like(value).to(dtype), want) > 1.5, name
    # a row's part of a sum: the gradient without it is the sum of the others'
    z = None if d["z"] is None else d["z"].repeat_interleave(rows // d["z"].shape[0], 0)
    each = bounds.gradients(dy, da, **{**d, "z": z}, **how)["gate"][0] if gate == "image" else None
    for lost in (0, rows - 1):
        keep = torch.arange(rows) != lost
        part = {**d, "x": d["x"][keep], "f": d["f"][keep], "z": None if z is None else z[keep]}
        rest = bounds.gradients(dy[keep], da[keep], **part, **how)
        for name in ("scale", "post_weight", "post_bias", "pre_weight", "pre_bias"):
            assert bounds.off(rest[name][0].to(dtype), ref[name]) > 1.5, (name, lost)
        if gate == "image":
            without = ref["gate"][0].clone()
            without[lost // (rows // images)] -= each[lost]
            assert bounds.off(without.to(dtype), ref["gate"]) > 1.5, ("gate", lost)
