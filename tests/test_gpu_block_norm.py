"""The norms around a block against their 64-bit forms: widths from one
channel to rows longer than the registers hold, odd ones, both types, every
norm, gates of each shape, rows of zeros, few and many rows.

Roundings counted: a lane adds at most 16 channels (a long row's lane at most
C/512), a wave 6 steps, a workgroup 8 waves, and at most 40 more operations
lie between an input and an output; column sums add at most rows + 300 terms
one after another.
"""
import pytest
import torch

import block_reference as br
import convolution_implicit_gemm_conv2d_amd as cm

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF16, F32 = torch.bfloat16, torch.float32


def make(seed, rows, C, dtype, post, pre, gate, scale, images, train=True):
    gen = torch.Generator().manual_seed(seed)

    def t(*shape, std=1.0, mean=0.0):
        return (torch.randn(shape, generator=gen) * std + mean).to(dtype)

    shape = (images, rows // images, C) if gate == "image" else (rows, C)
    d = dict(x=t(*shape, std=2.0), branch=t(*shape, std=0.5, mean=0.3), scale=t(C, std=0.3, mean=0.5) if scale else None,
             post_weight=t(C, mean=1.0, std=0.2) if post != "none" else None,
             post_bias=t(C, std=0.2) if post == "layer" else None,
             pre_weight=t(C, mean=1.0, std=0.2) if pre != "none" else None,
             pre_bias=t(C, std=0.2) if pre == "layer" else None,
             gate={"none": None, "full": (rows, C), "image": (images, C), "row": (C,)}[gate])
    if d["gate"] is not None:
        d["gate"] = t(*d["gate"])
    return d, t(*shape), t(*shape)


def dev(d):
    return {k: v.to(DEV) if isinstance(v, torch.Tensor) else v for k, v in d.items()}


def check(d, dy, da, post, pre, act, eps=br.EPS, kw=None):
    kw = kw or dev(d)
    C = d["x"].shape[-1]
    rows = d["x"].numel() // C
    flat = lambda t: None if t is None else t.reshape(-1, C)  # noqa: E731
    z = d["gate"]
    zr = None if z is None else flat(z).repeat_interleave(max(rows // max(flat(z).shape[0], 1), 1), 0)
    how = dict(post=post, pre=pre, gate_activation=act, eps=eps)
    y, a = cm.block_norm(**kw, **how)
    dyd, dad = (None if t is None else t.to(DEV) for t in (dy, da))
    g = cm.block_norm_grad(dyd, dad, **kw, **how) if dy is not None or da is not None else None
    torch.cuda.synchronize()
    ref = br.block_norm(flat(d["x"]), flat(d["branch"]), zr, d["scale"], d["post_weight"], d["post_bias"],
                        d["pre_weight"], d["pre_bias"], post, pre, act, eps, flat(dy), flat(da))
    n = 70 + C // 512
    cols = n + rows + 300
    if d["branch"] is not None:
        br.within("y", flat(y), *ref["y"], n)
    if pre != "none":
        br.within("a", flat(a), *ref["a"], n)
    if g is None:
        return
    br.within("dx", flat(g["x"]), *ref["dx"], n)
    if d["branch"] is not None:
        br.within("df", flat(g["branch"]), *ref["df"], n)
    names = dict(scale="ds", post_weight="dw_post", post_bias="db_post", pre_weight="dw_pre", pre_bias="db_pre")
    for k, name in names.items():
        if d[k] is not None and name in ref:
            br.within(name, g[k], *ref[name], cols)
    if z is not None:
        share = lambda t: t.reshape(flat(z).shape[0], -1, C).sum(1)  # noqa: E731
        br.within("dz", flat(g["gate"]), share(ref["dz"][0]), share(ref["dz"][1]), cols)


KINDS = [("rms", "rms", "none", "none", False), ("layer", "layer", "image", "sigmoid", True),
         ("rms", "layer", "full", "silu", True), ("none", "rms", "row", "tanh", True),
         ("layer", "none", "full", "gelu", False), ("rms", "rms", "image", "gelu_tanh", False),
         ("none", "layer", "none", "none", True), ("rms", "rms", "full", "relu", True)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("C", [1, 7, 64, 257, 512, 1000, 1024, 1025, 4096, 8191, 8192, 9001])
def test_widths(C, dtype):
    for i, (post, pre, gate, act, scale) in enumerate(KINDS):
        if i % 4 != C % 4 and C > 64:
            continue
        print(f"C={C} {dtype} post={post} pre={pre} gate={gate} act={act}", flush=True)
        d, dy, da = make(C + i, 12, C, dtype, post, pre, gate, scale, images=3)
        check(d, dy, da if pre != "none" else None, post, pre, act)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,images,C", [(1, 1, 96), (3, 3, 40), (700, 7, 96), (2600, 2, 33), (5000, 2500, 16),
                                           (130, 1, 1288)])
def test_rows(kind, rows, images, C):
    post, pre, gate, act, scale = kind
    d, dy, da = make(rows, rows, C, BF16 if rows % 2 else F32, post, pre, gate, scale, images)
    check(d, dy, da if pre != "none" else None, post, pre, act)


def test_norm_alone_and_one_gradient():
    d, dy, da = make(5, 33, 200, F32, "none", "layer", "none", False, 1)
    d["branch"] = None
    check(d, dy, da, "none", "layer", "none")
    check(d, None, da, "none", "layer", "none")
    d, dy, da = make(6, 33, 200, F32, "rms", "rms", "full", True, 1)
    check(d, dy, None, "rms", "rms", "silu")
    check(d, None, da, "rms", "rms", "silu")


@pytest.mark.parametrize("post,pre", [("rms", "rms"), ("layer", "layer")])
def test_constant_rows(post, pre):
    # a row of zeros, and one whose deviations are all zero: the scale is eps alone
    d, dy, da = make(7, 6, 72, F32, post, pre, "none", False, 1)
    d["x"][1], d["branch"][1] = 0.0, 0.0
    d["x"][2], d["branch"][2] = 1.5, 0.25
    check(d, dy, da, post, pre, "none", eps=1e-3)


def test_no_rows():
    d, dy, da = make(8, 0, 24, F32, "layer", "layer", "none", True, 1)
    kw = dev(d)
    y, a = cm.block_norm(**kw, post="layer", pre="layer")
    assert y.shape == a.shape == (0, 24)
    g = cm.block_norm_grad(dy.to(DEV), da.to(DEV), **kw, post="layer", pre="layer")
    for k in ("scale", "post_weight", "post_bias", "pre_weight", "pre_bias"):
        assert torch.equal(g[k].cpu(), torch.zeros(24)), k


def test_not_finite_stays_in_its_row():
    d, dy, da = make(9, 8, 130, F32, "layer", "rms", "full", True, 1)
    d["branch"][3, 5] = float("nan")
    d["x"][6, 129] = float("inf")
    y, a = (t.cpu() for t in cm.block_norm(**dev(d), post="layer", pre="rms", gate_activation="sigmoid"))
    rows = torch.tensor([0, 1, 2, 4, 5, 7])
    assert torch.isnan(y[3]).all() and torch.isnan(a[3]).all() and torch.isnan(a[6, 129])
    assert torch.isfinite(y[rows]).all() and torch.isfinite(a[rows]).all()


def test_unaligned_rows_and_guards():
    # views at odd offsets of a larger buffer: nothing around them is written
    C, rows = 203, 9
    d, dy, da = make(10, rows, C, BF16, "rms", "rms", "none", True, 1)
    kw = dev(d)

    def moved(t):
        b = torch.full((t.numel() + 7,), -7.0, dtype=t.dtype, device=DEV)
        b[3:3 + t.numel()] = t.reshape(-1)
        return b, b[3:3 + t.numel()].view(t.shape)

    for k in ("x", "branch", "scale", "pre_weight", "post_weight"):
        kw[k] = moved(kw[k])[1]
    check(d, dy, da, "rms", "rms", "none", kw=kw)
    by, y = moved(torch.zeros(rows, C, dtype=BF16))
    ba, a = moved(torch.zeros(rows, C, dtype=BF16))
    cm.conv_block_norm_fwd(kw["x"], kw["branch"], None, kw["scale"], kw["post_weight"], None, kw["pre_weight"], None, y,
                           a, rows, C, 1, 1, 1, 0, 1e-6, cm.CONV_BF16)
    want = cm.block_norm(**kw, post="rms", pre="rms")
    torch.cuda.synchronize()
    for b, v, w in ((by, y, want[0]), (ba, a, want[1])):
        assert torch.equal(v, w)
        assert (b[:3] == -7).all() and (b[3 + rows * C:] == -7).all()


def test_same_on_every_run_and_on_another_stream():
    d, dy, da = make(11, 3000, 256, BF16, "layer", "layer", "image", True, 6)
    kw = dev(d)
    how = dict(post="layer", pre="layer", gate_activation="sigmoid")
    dyd, dad = dy.to(DEV), da.to(DEV)
    first = cm.block_norm_grad(dyd, dad, **kw, **how)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in (None, s, s.cuda_stream):
        again = cm.block_norm_grad(dyd, dad, **kw, **how, stream=stream)
        torch.cuda.synchronize()
        for k, v in first.items():
            assert torch.equal(v, again[k]), k


def test_graph_replays():
    d, dy, da = make(12, 500, 384, BF16, "rms", "rms", "image", True, 5)
    kw, how = dev(d), dict(post="rms", pre="rms", gate_activation="sigmoid")
    dyd, dad = dy.to(DEV), da.to(DEV)
    y, a = cm.block_norm(**kw, **how)
    g = cm.block_norm_grad(dyd, dad, **kw, **how)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y2, a2 = cm.block_norm(**kw, **how)
        g2 = cm.block_norm_grad(dyd, dad, **kw, **how)
    for _ in range(3):
        cm.block_norm(**kw, **how)
        for t in (y2, a2, *[v for v in g2.values() if v is not None]):
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, y2) and torch.equal(a, a2)
        for k, v in g.items():
            assert v is None or torch.equal(v, g2[k]), k
