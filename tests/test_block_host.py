"""Host-side checks of the operators around a convolution (CPU): the 64-bit
forms against automatic differentiation and against differences, and every
refusal.  No call here reaches a GPU."""
import itertools

import pytest
import torch

import block_reference as br
import convolution_implicit_gemm_conv2d_amd as cm
from convolution_implicit_gemm_conv2d_amd import _lib

FAKE = 0x1000  # never dereferenced: every call below fails validation first
ACTS = list(cm.ACTIVATIONS)


@pytest.mark.parametrize("kind", ACTS)
def test_activation_derivatives(kind):
    v = torch.linspace(-6, 6, 97, dtype=torch.float64) + 0.01
    h = 1e-6
    d = (br.act(v + h, kind)[0] - br.act(v - h, kind)[0]) / (2 * h)
    assert torch.allclose(br.act(v, kind)[1], d, atol=1e-8)


@pytest.mark.parametrize("post,pre", itertools.product(["none", "rms", "layer"], repeat=2))
def test_norm_reference_against_autograd_and_differences(post, pre):
    gen = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(s, generator=gen, dtype=torch.float64)  # noqa: E731
    t = {k: r(5, 9).requires_grad_() for k in ("x", "f", "z")}
    t |= {k: r(9).requires_grad_() for k in ("s", "w_post", "b_post", "w_pre", "b_pre")}
    dy, da = r(5, 9), r(5, 9)

    def loss(v):
        def norm(q, kind, w, b):
            if kind == "none":
                return q * w + b  # the reference applies given weights even so
            q = q - q.mean(-1, keepdim=True) if kind == "layer" else q
            return q / (q.pow(2).mean(-1, keepdim=True) + br.EPS).sqrt() * w + b

        y = v["x"] + v["s"] * torch.sigmoid(v["z"]) * norm(v["f"], post, v["w_post"], v["b_post"])
        out = (y * dy).sum()
        return out + (norm(y, pre, v["w_pre"], v["b_pre"]) * da).sum() if pre != "none" else out

    ref = br.block_norm(t["x"], t["f"], t["z"], t["s"], t["w_post"], t["b_post"], t["w_pre"], t["b_pre"], post, pre,
                        "sigmoid", br.EPS, dy, da if pre != "none" else None)
    got = torch.autograd.grad(loss(t), list(t.values()), allow_unused=True)
    for (k, v), g in zip(t.items(), got):
        name = "d" + k
        if name not in ref:
            assert g is None
            continue
        value = ref[name][0]
        assert torch.allclose(value, g, atol=1e-10), name
        step = torch.zeros_like(v)
        step.view(-1)[3] = 1e-6
        up, down = ({**t, k: v + sign * step} for sign in (1, -1))
        assert abs((loss(up) - loss(down)).item() / 2e-6 - value.reshape(-1)[3].item()) < 1e-6, name


@pytest.mark.parametrize("kind", ACTS)
def test_gated_reference_against_autograd(kind):
    gen = torch.Generator().manual_seed(2)
    r = lambda *s: torch.randn(s, generator=gen, dtype=torch.float64).requires_grad_()  # noqa: E731
    x, wg, wu, bg, bu, dh = r(4, 6), r(5, 6), r(5, 6), r(5), r(5), r(4, 5)
    F = torch.nn.functional
    fn = {"none": lambda v: v, "sigmoid": torch.sigmoid, "silu": F.silu, "gelu": F.gelu, "relu": torch.relu,
          "gelu_tanh": lambda v: F.gelu(v, approximate="tanh"), "tanh": torch.tanh}[kind]
    h = fn(F.linear(x, wg, bg)) * F.linear(x, wu, bu)
    ref = br.gated(x, wg, wu, bg, bu, kind, dh)
    assert torch.allclose(ref["h"][0], h, atol=1e-12)
    for name, g in zip(("dx", "dwg", "dwu", "dbg", "dbu"), torch.autograd.grad(h, (x, wg, wu, bg, bu), dh)):
        assert torch.allclose(ref[name][0], g, atol=1e-12), name


# ------------------------------------------------------------- C refusals --

def norm_fwd(x=FAKE, branch=FAKE, gate=None, scale=None, post_w=None, post_b=None, pre_w=None, pre_b=None, y=FAKE, a=FAKE,
             rows=4, C=8, gate_rows=1, post=1, pre=1, act=0, eps=1e-6, dtype=1):
    return _lib.load().conv_block_norm_fwd(x, branch, gate, scale, post_w, post_b, pre_w, pre_b, y, a, rows, C, gate_rows,
                                           post, pre, act, eps, dtype, None)


NORM_BAD = [
    dict(dtype=2), dict(dtype=-1), dict(act=7), dict(act=-1), dict(post=3), dict(pre=-1), dict(rows=-1), dict(C=0),
    dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(x=None), dict(y=None, a=None),
    dict(branch=None), dict(branch=None, post=0, scale=FAKE), dict(branch=None, post=0, gate=FAKE),
    dict(gate=FAKE, gate_rows=0), dict(gate=FAKE, gate_rows=3), dict(pre=0), dict(post=0, post_w=FAKE),
    dict(post_b=FAKE), dict(pre_b=FAKE), dict(pre=0, a=None, pre_w=FAKE), dict(x=FAKE + 1), dict(a=FAKE + 2, dtype=0),
]


@pytest.mark.parametrize("bad", NORM_BAD)
def test_norm_refusals(bad):
    assert norm_fwd(**bad) == cm.CONV_ERR_INVALID_ARG
    assert "conv_block_norm_fwd" in cm.conv_last_error()


def test_norm_overflow_and_empty():
    assert norm_fwd(C=(1 << 20) + 1) == cm.CONV_ERR_OVERFLOW
    assert norm_fwd(rows=1 << 31) == cm.CONV_ERR_OVERFLOW
    assert norm_fwd(rows=0) == cm.CONV_OK  # nothing to launch


def norm_bwd(dy=FAKE, da=FAKE, x=FAKE, branch=FAKE, gate=None, scale=None, post_w=None, post_b=None, pre_w=None, pre_b=None,
             grads=(FAKE, FAKE) + (None,) * 6, ws=FAKE, ws_bytes=1 << 40, rows=4, C=8, gate_rows=1, post=1, pre=1, act=0,
             eps=1e-6, dtype=1):
    return _lib.load().conv_block_norm_bwd(dy, da, x, branch, gate, scale, post_w, post_b, pre_w, pre_b, *grads, ws,
                                           ws_bytes, rows, C, gate_rows, post, pre, act, eps, dtype, None)


@pytest.mark.parametrize("bad", [
    dict(dy=None, da=None), dict(pre=0), dict(branch=None, post=0), dict(ws=None), dict(ws=FAKE + 8), dict(ws_bytes=10),
    dict(grads=(FAKE, FAKE, FAKE) + (None,) * 5), dict(grads=(None,) * 5 + (FAKE,) + (None,) * 2),
    dict(grads=(None,) * 7 + (FAKE,)), dict(post=0, grads=(None,) * 4 + (FAKE,) + (None,) * 3), dict(dy=FAKE + 1),
    *[b for b in NORM_BAD if not {"y", "a"} & set(b)]])
def test_norm_grad_refusals(bad):
    assert norm_bwd(**bad) == cm.CONV_ERR_INVALID_ARG


def gated_fwd(x=FAKE, wg=FAKE, wu=FAKE, bg=None, bu=None, h=FAKE, saved=None, rows=4, C=8, F=8, act=2, dtype=1):
    return _lib.load().conv_gated_fwd(x, wg, wu, bg, bu, h, saved, rows, C, F, act, dtype, None)


GATED_BAD = [dict(x=None), dict(wg=None), dict(wu=None), dict(bg=FAKE), dict(bu=FAKE), dict(rows=-1), dict(C=0),
             dict(F=0), dict(act=7), dict(act=-1), dict(dtype=2), dict(saved=FAKE + 2), dict(x=FAKE + 1),
             dict(wu=FAKE + 2, dtype=0)]


@pytest.mark.parametrize("bad", GATED_BAD + [dict(h=None)])
def test_gated_refusals(bad):
    assert gated_fwd(**bad) == cm.CONV_ERR_INVALID_ARG


def gated_bwd(dh=FAKE, x=FAKE, wg=FAKE, wu=FAKE, bg=None, bu=None, saved=None, grads=(FAKE,) * 3 + (None,) * 2, ws=FAKE,
              ws_bytes=1 << 40, rows=4, C=8, F=8, act=2, dtype=1):
    return _lib.load().conv_gated_bwd(dh, x, wg, wu, bg, bu, saved, *grads, ws, ws_bytes, rows, C, F, act, dtype, None)


@pytest.mark.parametrize("bad", GATED_BAD + [dict(dh=None), dict(ws=None), dict(ws=FAKE + 4), dict(ws_bytes=1)])
def test_gated_grad_refusals(bad):
    assert gated_bwd(**bad) == cm.CONV_ERR_INVALID_ARG


def test_gated_overflow_and_empty():
    assert gated_fwd(rows=1 << 31) == cm.CONV_ERR_OVERFLOW
    assert gated_fwd(F=(1 << 20) + 1) == cm.CONV_ERR_OVERFLOW
    assert gated_fwd(rows=0, x=None, h=None) == cm.CONV_OK


def test_list_refusals():
    n, one = 1, [FAKE]
    ok = dict(grads=one, outs=one, counts=[8], dtypes=[0], n=n, max_norm=1.0, eps=0.0, norm=FAKE, workspace=FAKE,
              workspace_bytes=1 << 30, stream=0)
    for bad in (dict(n=-1), dict(dtypes=[2]), dict(grads=[0]), dict(outs=[0]), dict(grads=[FAKE + 2]),
                dict(outs=[FAKE + 1], dtypes=[1]), dict(max_norm=-1.0), dict(max_norm=float("nan")), dict(eps=-1.0),
                dict(eps=float("inf")), dict(workspace=None), dict(workspace=FAKE + 8), dict(workspace_bytes=8),
                dict(norm=FAKE + 2)):
        with pytest.raises(cm.ConvError) as e:
            cm.conv_grad_clip(**{**ok, **bad})
        assert e.value.status == cm.CONV_ERR_INVALID_ARG, bad
    with pytest.raises(cm.ConvError) as e:
        cm.conv_grad_clip(**{**ok, "counts": [1 << 46]})
    assert e.value.status == cm.CONV_ERR_OVERFLOW
    with pytest.raises(cm.ConvError):
        cm.conv_grad_norm(one, [8], [0], 1, None, FAKE, 1 << 30, 0)


def test_workspace_sizes():
    assert cm.conv_grad_workspace_size(0) >= 8 and cm.conv_grad_workspace_size(1000) >= 8 * 8 * 256
    assert cm.conv_block_norm_bwd_workspace_size(0, 8, 0) == 0
    assert cm.conv_block_norm_bwd_workspace_size(64, 8, 16) > 0
    with pytest.raises(cm.ConvError):
        cm.conv_block_norm_bwd_workspace_size(64, 8, 7)
    for args in ((-1, 8, 8, 1), (4, 0, 8, 1), (4, 8, 8, 3)):
        with pytest.raises(cm.ConvError):
            cm.conv_gated_bwd_workspace_size(*args)
    lib = _lib.load()
    assert lib.conv_grad_workspace_size(1, None) == cm.CONV_ERR_INVALID_ARG
    assert lib.conv_gated_bwd_workspace_size(1, 1, 1, 1, None) == cm.CONV_ERR_INVALID_ARG
    assert lib.conv_block_norm_bwd_workspace_size(1, 1, 0, None) == cm.CONV_ERR_INVALID_ARG


# -------------------------------------------------------- Python refusals --

def test_tensor_level_refusals():
    x, w = torch.zeros(4, 8), torch.zeros(6, 8)
    bad = [
        lambda: cm.gated_feed_forward(x, w, w),  # not on a GPU
        lambda: cm.gated_feed_forward(x.half(), w, w),
        lambda: cm.gated_feed_forward(x, w, w, activation="swish"),
        lambda: cm.gated_feed_forward(x, torch.zeros(6, 7), w),
        lambda: cm.gated_feed_forward(x, w, torch.zeros(5, 8)),
        lambda: cm.gated_feed_forward(x, w, w, torch.zeros(6)),
        lambda: cm.gated_feed_forward(x, w, w, torch.zeros(5), torch.zeros(5)),
        lambda: cm.gated_feed_forward(x, w.bfloat16(), w),
        lambda: cm.gated_feed_forward(x, w, w, saved=torch.zeros(4, 6)),
        lambda: cm.gated_feed_forward(x, w, w, out=torch.zeros(4, 7)),
        lambda: cm.gated_feed_forward_grad(torch.zeros(4, 8), x, w, w),
        lambda: cm.block_norm(x, torch.zeros(4, 7)),
        lambda: cm.block_norm(x, x, gate=torch.zeros(3, 8)),
        lambda: cm.block_norm(x, x, scale=torch.zeros(7)),
        lambda: cm.block_norm(x, x, post="batch"),
        lambda: cm.block_norm(x, pre="none"),
        lambda: cm.block_norm(x, x),
        lambda: cm.block_norm_grad(torch.zeros(3, 8), None, x, x),
        lambda: cm.gradient_norm([]),
        lambda: cm.gradient_norm([x]),
        lambda: cm.gradient_norm([x.double()]),
        lambda: cm.clip_gradients([], 1.0),
        lambda: cm.clip_gradients([x], 1.0, out=[]),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            print(i)


@pytest.mark.parametrize("dtype", [0, 1])
def test_gated_workspace_without_rows(dtype):
    assert cm.conv_gated_bwd_workspace_size(0, 16, 24, dtype) >= 0


def test_gated_forward_workspace():
    assert cm.conv_gated_fwd_workspace_size(4096, 256, 1024, 1) == 0  # whole units
    need = cm.conv_gated_fwd_workspace_size(4096, 255, 2048, 1)
    assert need >= (4096 + 2 * 2048) * 256 * 2
    lib = _lib.load()
    assert lib.conv_gated_fwd_workspace_size(1, 1, 1, 1, None) == cm.CONV_ERR_INVALID_ARG
    for ws, size in ((None, need), (FAKE + 8, need), (FAKE, need - 1)):
        assert lib.conv_gated_fwd_ex(FAKE, FAKE, FAKE, None, None, FAKE, None, ws, size, 4096, 255, 2048, 2, 1,
                                     None) == cm.CONV_ERR_INVALID_ARG
    for bad in GATED_BAD:
        a = {**dict(x=FAKE, wg=FAKE, wu=FAKE, bg=None, bu=None, saved=None, rows=4, C=8, F=8, act=2, dtype=1), **bad}
        assert lib.conv_gated_fwd_ex(a["x"], a["wg"], a["wu"], a["bg"], a["bu"], FAKE, a["saved"], None, 0, a["rows"], a["C"],
                                     a["F"], a["act"], a["dtype"], None) == cm.CONV_ERR_INVALID_ARG
