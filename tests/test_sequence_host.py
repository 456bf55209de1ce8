"""Host-side checks of the operators along a sequence and of the optimizer step
(CPU): the 64-bit forms against automatic differentiation and against
differences, and every refusal.  No call here reaches a GPU."""
import pytest
import torch

import convolution_implicit_gemm_conv2d_amd as cm
import sequence_reference as sr
from convolution_implicit_gemm_conv2d_amd import _lib
from running_bounds import U32, B, act, softplus

FAKE = 0x10000000  # never dereferenced: every call below fails validation first


def apart(i):
    """Addresses that do not overlap for the sizes used here."""
    return FAKE * (i + 1)


def leaf(*shape, gen, std=1.0):
    return (torch.randn(shape, generator=gen, dtype=torch.float64) * std).requires_grad_()


def differences(loss, t, at, want):
    step = torch.zeros_like(t)
    step.view(-1)[at] = 1e-6
    with torch.no_grad():
        d = (loss(t + step) - loss(t - step)).item() / 2e-6
    assert abs(d - want.reshape(-1)[at].item()) < 1e-6


@pytest.mark.parametrize("kind", ["none", "silu", "sigmoid", "tanh", "relu"])
def test_causal_reference(kind):
    gen = torch.Generator().manual_seed(1)
    spans, K = [(1, 8), (8, 8), (8, 10)], 4
    x, w, b, initial = leaf(11, 3, gen=gen), leaf(3, K, gen=gen), leaf(3, gen=gen), leaf(3, K - 1, 3, gen=gen)
    dy, dlast = torch.randn(11, 3, generator=gen, dtype=torch.float64), torch.randn(3, K - 1, 3, generator=gen, dtype=torch.float64)
    fn = {"none": lambda v: v, "silu": torch.nn.functional.silu, "sigmoid": torch.sigmoid, "tanh": torch.tanh, "relu": torch.relu}[kind]

    def loss(x=x, w=w, b=b, initial=initial):
        out = 0
        for s, (f, e) in enumerate(spans):
            line = torch.cat([initial[s], x[f:e]])
            for t in range(e - f):
                out = out + (fn((line[t:t + K] * w.t()).sum(0) + b) * dy[f + t]).sum()
            out = out + (line[e - f:] * dlast[s]).sum()
        return out

    ref = sr.causal(x, w, b, kind, spans, initial, dy, dlast)
    names = ("x", "weight", "bias", "initial")
    for name, g in zip(names, torch.autograd.grad(loss(), (x, w, b, initial))):
        assert torch.allclose(ref[name].v, g, atol=1e-12), name
    differences(lambda t: loss(x=t), x, 7, ref["x"].v)
    differences(lambda t: loss(initial=t), initial, 4, ref["initial"].v)


@pytest.mark.parametrize("plus,kind", [(True, "silu"), (False, "sigmoid"), (True, "none")])
def test_scan_reference(plus, kind):
    gen = torch.Generator().manual_seed(2)
    spans, C, N, G = [(0, 5), (5, 5), (5, 9)], 6, 3, 2
    x, delta, z = (leaf(10, C, gen=gen) for _ in range(3))
    Bm, Cm = (leaf(10, G, N, gen=gen) for _ in range(2))
    A, D, bias, initial = leaf(C, N, gen=gen, std=0.3), leaf(C, gen=gen), leaf(C, gen=gen), leaf(3, C, N, gen=gen)
    dy, dlast = torch.randn(10, C, generator=gen, dtype=torch.float64), torch.randn(3, C, N, generator=gen, dtype=torch.float64)
    fn = {"silu": torch.nn.functional.silu, "sigmoid": torch.sigmoid, "none": lambda v: v}[kind]
    leaves = dict(x=x, delta=delta, A=A, B=Bm, C=Cm, D=D, z=z, delta_bias=bias, initial=initial)

    def loss(**k):
        k = {**leaves, **k}
        out = 0
        for s, (f, e) in enumerate(spans):
            h = k["initial"][s]
            for t in range(f, e):
                d = k["delta"][t] + k["delta_bias"]
                d = torch.log1p(d.exp()) if plus else d
                b, c = (k[n][t].repeat_interleave(C // G, 0) for n in "BC")
                h = (d[:, None] * k["A"]).exp() * h + (d * k["x"][t])[:, None] * b
                out = out + (((h * c).sum(1) + k["D"] * k["x"][t]) * fn(k["z"][t]) * dy[t]).sum()
            out = out + (h * dlast[s]).sum()
        return out

    ref = sr.scan(x, delta, A, Bm, Cm, D, z, bias, plus, kind, spans, initial, dy, dlast)
    for (name, t), g in zip(leaves.items(), torch.autograd.grad(loss(), list(leaves.values()))):
        assert torch.allclose(ref[name].v, g, atol=1e-12), name
        differences(lambda v: loss(**{name: v}), t, t.numel() // 3, ref[name].v)  # noqa: B023


def test_bounds_hold_for_fp32_and_are_not_loose():
    """The same arithmetic in fp32 stays inside, an error of a few roundings does not."""
    gen = torch.Generator().manual_seed(3)
    v = torch.randn(4000, generator=gen)
    for got, want in ((torch.nn.functional.softplus(v), softplus(B(v))[0]), (torch.nn.functional.silu(v), act(B(v), "silu")[0]),
                      ((v * v + v), B(v) * B(v) + B(v)), ((v[:3999].view(3, -1) ** 2).sum(1), (B(v[:3999].view(3, -1)) * B(v[:3999].view(3, -1))).sum(1))):
        off = (got.double() - want.v).abs()
        assert (off <= U32 * want.e + U32 * want.v.abs()).all()
        assert (want.e <= 4100 * want.v.abs() + 40).all()


# ------------------------------------------------------------ C refusals --

def causal(x=apart(0), w=apart(1), bias=None, starts=None, initial=None, y=apart(2), last=None, rows=8, seqs=2, C=8, K=4, xs=8, act=2, clear=0, dtype=1):
    return _lib.load().conv_causal_fwd(x, w, bias, starts, initial, y, last, rows, seqs, C, K, xs, act, clear, dtype, None)


CAUSAL_BAD = [dict(x=None), dict(w=None), dict(rows=-1), dict(rows=9), dict(seqs=-1), dict(seqs=0), dict(C=0), dict(K=1), dict(K=9), dict(xs=7), dict(act=7),
              dict(act=-1), dict(dtype=2), dict(x=FAKE + 1), dict(w=FAKE + 2, dtype=0), dict(starts=apart(5) + 2), dict(initial=apart(5) + 1)]


@pytest.mark.parametrize("bad", CAUSAL_BAD + [dict(y=None), dict(y=apart(0) + 16), dict(last=apart(2)), dict(initial=apart(5), last=apart(5) + 16),
                                              dict(xs=16, y=apart(0) + 16)])
def test_causal_refusals(bad):
    assert causal(**bad) == cm.CONV_ERR_INVALID_ARG
    assert "conv_causal_fwd" in cm.conv_last_error()


def test_sizes_too_large():
    assert causal(C=(1 << 20) + 1, xs=1 << 21) == cm.CONV_ERR_OVERFLOW
    assert causal(rows=1 << 31) == cm.CONV_ERR_OVERFLOW
    assert causal(xs=1 << 24) == cm.CONV_ERR_OVERFLOW
    assert causal(rows=0, seqs=0, x=None, y=None) == cm.CONV_OK  # nothing to launch


def causal_bwd(dy=apart(0), x=apart(1), w=apart(2), starts=None, initial=None, grads=(apart(3), apart(4), apart(5), None), ws=apart(6), ws_bytes=1 << 20,
               rows=8, seqs=2, C=8, K=4, xs=8, act=2, dtype=1):
    return _lib.load().conv_causal_bwd(dy, None, x, w, None, starts, initial, *grads, ws, ws_bytes, rows, seqs, C, K, xs, act, 0, dtype, None)


@pytest.mark.parametrize("bad", CAUSAL_BAD + [dict(dy=None), dict(ws=None), dict(ws=apart(6) + 8), dict(ws_bytes=8), dict(grads=(apart(3), apart(3), None, None)),
                                              dict(grads=(apart(0), None, None, None)), dict(ws=apart(3))])
def test_causal_grad_refusals(bad):
    assert causal_bwd(**bad) == cm.CONV_ERR_INVALID_ARG


def scan(x=apart(0), delta=apart(1), A=apart(2), b=apart(3), c=apart(4), D=None, z=None, bias=None, starts=None, initial=None, y=apart(5), last=None,
         saved=None, ws=apart(6), ws_bytes=1 << 24, rows=8, seqs=2, C=8, N=4, G=1, xs=8, ds=8, zs=8, bs=4, cs=4, act=2, dtype=1):
    return _lib.load().conv_scan_fwd(x, delta, A, b, c, D, z, bias, starts, initial, y, last, saved, ws, ws_bytes, rows, seqs, C, N, G, xs, ds, zs, bs, cs, 1,
                                    act, 0, dtype, None)


SCAN_BAD = [dict(x=None), dict(delta=None), dict(A=None), dict(b=None), dict(c=None), dict(rows=-1), dict(rows=9), dict(seqs=0), dict(C=0), dict(N=0), dict(N=65),
            dict(G=0), dict(G=3), dict(xs=7), dict(ds=7), dict(z=apart(9), zs=7), dict(bs=3), dict(cs=3), dict(G=2, bs=7), dict(act=7), dict(dtype=2),
            dict(x=FAKE + 1), dict(A=apart(2) + 2), dict(D=apart(9) + 1), dict(starts=apart(9) + 2)]


@pytest.mark.parametrize("bad", SCAN_BAD + [dict(y=None), dict(y=apart(0)), dict(last=apart(5)), dict(saved=apart(1)), dict(rows=4096, seqs=1, ws=None),
                                            dict(rows=4096, seqs=1, ws_bytes=16), dict(initial=apart(9), last=apart(9))])
def test_scan_refusals(bad):
    assert scan(**bad) == cm.CONV_ERR_INVALID_ARG
    assert "conv_scan_fwd" in cm.conv_last_error()


def scan_bwd(x=apart(0), delta=apart(1), A=apart(2), b=apart(3), c=apart(4), D=None, z=None, dy=apart(5), starts=None, grads=(apart(10),) + (None,) * 8,
             ws=apart(6), ws_bytes=1 << 24, rows=8, seqs=2, C=8, N=4, G=1, xs=8, ds=8, zs=8, bs=4, cs=4, act=2, dtype=1):
    return _lib.load().conv_scan_bwd(dy, None, x, delta, A, b, c, D, z, None, starts, None, None, *grads, ws, ws_bytes, rows, seqs, C, N, G, xs, ds, zs, bs, cs,
                                    1, act, 0, dtype, None)


@pytest.mark.parametrize("bad", SCAN_BAD + [dict(dy=None), dict(ws=None), dict(ws=apart(6) + 4), dict(ws_bytes=64), dict(grads=(None,) * 6 + (apart(10),) + (None,) * 2),
                                            dict(grads=(apart(10), apart(10)) + (None,) * 7), dict(grads=(apart(5),) + (None,) * 8), dict(ws=apart(10))])
def test_scan_grad_refusals(bad):
    assert scan_bwd(**bad) == cm.CONV_ERR_INVALID_ARG


def test_step_refusals():
    lib = _lib.load()

    def conv(x=apart(0), w=apart(1), state=apart(2), slots=None, y=apart(3), rows=4, count=4, C=8, K=4, xs=8, act=0, dtype=0):
        return lib.conv_causal_step(x, w, None, state, slots, y, rows, count, C, K, xs, act, 0, dtype, None)

    def step(x=apart(0), delta=apart(1), A=apart(2), b=apart(3), c=apart(4), state=apart(5), slots=None, y=apart(6), rows=4, count=4, C=8, N=4, G=1, bs=4, act=0,
             dtype=0):
        return lib.conv_scan_step(x, delta, A, b, c, None, None, None, state, slots, y, rows, count, C, N, G, 8, 8, 8, bs, 4, 1, act, 0, dtype, None)

    for bad in (dict(x=None), dict(w=None), dict(state=None), dict(y=None), dict(count=3), dict(count=-1), dict(K=1), dict(xs=4), dict(slots=apart(7) + 2),
                dict(y=apart(2)), dict(state=apart(0)), dict(dtype=5)):
        assert conv(**bad) == cm.CONV_ERR_INVALID_ARG, bad
    for bad in (dict(x=None), dict(A=None), dict(state=None), dict(y=None), dict(count=3), dict(N=65), dict(G=3), dict(bs=2), dict(slots=apart(7) + 1),
                dict(y=apart(5)), dict(state=apart(2)), dict(act=9)):
        assert step(**bad) == cm.CONV_ERR_INVALID_ARG, bad
    assert conv(rows=0, x=None, y=None) == cm.CONV_OK and step(rows=0, x=None, y=None) == cm.CONV_OK


ADAM = dict(params=[apart(0)], grads=[apart(1)], m=[apart(2)], v=[apart(3)], m_scales=None, v_scales=None, copies=None, counts=[256], param_dtypes=[0],
            grad_dtypes=[0], copy_dtypes=None, n=1, bits=32, lr=0.1, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.0, step=1, norm=None, stream=0)


@pytest.mark.parametrize("bad", [
    dict(n=-1), dict(bits=16), dict(bits=8), dict(params=[0]), dict(grads=[0]), dict(m=[0]), dict(v=[0]), dict(params=[apart(0) + 2]), dict(grads=[apart(1) + 1], grad_dtypes=[1]),
    dict(m=[apart(2) + 2]), dict(param_dtypes=[2]), dict(grad_dtypes=[-1]), dict(copies=[apart(4)]), dict(copies=[apart(4)], copy_dtypes=[3]),
    dict(copies=[apart(4) + 1], copy_dtypes=[1]), dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=float("nan")), dict(beta2=1 - 1e-12), dict(eps=0.0), dict(eps=-1.0),
    dict(eps=1e-40), dict(lr=float("inf")), dict(lr=float("nan")), dict(weight_decay=-0.1), dict(step=0), dict(max_norm=-1.0), dict(norm_eps=-1.0),
    dict(norm=apart(5) + 2), dict(lr_dev=apart(5) + 2), dict(step_dev=apart(5) + 4), dict(grads=[apart(0)]), dict(m=[apart(3) + 1020]), dict(copies=[apart(1)], copy_dtypes=[0]),
    dict(norm=apart(0)), dict(bits=8, m_scales=[apart(6)], v_scales=[apart(6) + 4]), dict(bits=8, m_scales=[0], v_scales=[apart(6)])])
def test_adamw_refusals(bad):
    with pytest.raises(cm.ConvError) as e:
        cm.conv_adamw(**{**ADAM, **bad})
    assert e.value.status == cm.CONV_ERR_INVALID_ARG


def test_adamw_list_refusals():
    with pytest.raises(cm.ConvError) as e:
        cm.conv_adamw(**{**ADAM, "counts": [1 << 38]})
    assert e.value.status == cm.CONV_ERR_OVERFLOW
    two = {k: [v[0], v[0] + FAKE * 40] if k in ("params", "grads", "m", "v") else v * 2 if k in ("counts", "param_dtypes", "grad_dtypes") else v for k, v in ADAM.items()}
    two["n"] = 2
    for k in ("params", "m", "v"):
        with pytest.raises(cm.ConvError):
            cm.conv_adamw(**{**two, k: [two[k][0]] * 2})  # the same tensor twice
    cm.conv_adamw(**{**ADAM, "counts": [0], "params": [0]})  # nothing to launch
    cm.conv_adamw(**{**ADAM, "n": 0})
    ok = dict(m=[apart(0)], v=[apart(1)], m_scales=[apart(2)], v_scales=[apart(3)], m_out=[apart(4)], v_out=[apart(5)], counts=[256], n=1, stream=0)
    for bad in (dict(n=-1), dict(m=[0]), dict(m_scales=[apart(2) + 1]), dict(m_out=[apart(5) + 512]), dict(v_out=[apart(0)]), dict(m_out=[apart(4) + 2])):
        with pytest.raises(cm.ConvError):
            cm.conv_adamw_moments(**{**ok, **bad})


def test_workspace_sizes():
    assert cm.conv_scan_saved_size(33, 10, 16) == 3 * 10 * 16 * 4 and cm.conv_scan_saved_size(0, 10, 16) == 0
    assert cm.conv_scan_fwd_workspace_size(4096, 64, 4096, 16, 1, False) == 0  # enough sequences
    assert cm.conv_scan_fwd_workspace_size(4096, 1, 64, 16, 1, False) > 0
    assert cm.conv_scan_bwd_workspace_size(4096, 1, 64, 16, 1, True, False) - cm.conv_scan_bwd_workspace_size(4096, 1, 64, 16, 1, True, True) >= 256 * 64 * 16 * 4
    assert cm.conv_causal_bwd_workspace_size(0, 8, 4, 1) == 0 and cm.conv_causal_bwd_workspace_size(100, 8, 4, 1) > 0
    lib = _lib.load()
    assert lib.conv_scan_saved_size(1, 1, 1, None) == cm.CONV_ERR_INVALID_ARG
    assert lib.conv_scan_fwd_workspace_size(1, 1, 1, 1, 1, 0, None) == cm.CONV_ERR_INVALID_ARG
    assert lib.conv_causal_bwd_workspace_size(1, 1, 4, 1, None) == cm.CONV_ERR_INVALID_ARG
    for args in ((8, 3, 4, 4, 1, False), (8, 2, 4, 65, 1, False), (8, 2, 4, 4, 3, False), (-1, 1, 4, 4, 1, False)):
        with pytest.raises(cm.ConvError):
            cm.conv_scan_fwd_workspace_size(*args)


# -------------------------------------------------------- Python refusals --

def test_tensor_level_refusals():
    t = torch.zeros
    x, w, A, b = t(4, 8), t(8, 4), t(8, 3), t(4, 3)
    i32 = torch.int32
    p = [t(5)]
    bad = [
        lambda: cm.causal_conv(x, w),  # not on a GPU
        lambda: cm.causal_conv(x.half(), w.half()),
        lambda: cm.causal_conv(x, w, activation="swish"),
        lambda: cm.causal_conv(x, t(7, 4)),
        lambda: cm.causal_conv(x, t(8, 9)),
        lambda: cm.causal_conv(x, t(8, 1)),
        lambda: cm.causal_conv(x, t(8, 2, 2)),
        lambda: cm.causal_conv(x, w, t(7)),
        lambda: cm.causal_conv(x, w.bfloat16()),
        lambda: cm.causal_conv(t(8, 4).t(), t(4, 8).t()),
        lambda: cm.causal_conv(t(2, 2, 2, 8), w),
        lambda: cm.causal_conv(x[:1].expand(4, 8), w),
        lambda: cm.causal_conv(x, w, initial=t(1, 4, 8)),
        lambda: cm.causal_conv(x, w, last=t(2, 3, 8)),
        lambda: cm.causal_conv(x, w, out=t(4, 7)),
        lambda: cm.causal_conv(x, w, starts=t(3)),
        lambda: cm.causal_conv(x, w, starts=t(1, dtype=i32)),
        lambda: cm.causal_conv(t(1, 4, 8), w, starts=t(3, dtype=i32)),
        lambda: cm.causal_conv_grad(t(4, 7), x, w),
        lambda: cm.causal_conv_grad(x, x, w, dlast=t(1, 2, 8)),
        lambda: cm.causal_conv_step(x, w, t(3, 3, 8)),
        lambda: cm.causal_conv_step(x, w, t(4, 2, 8)),
        lambda: cm.causal_conv_step(x, w, t(4, 3, 8), slots=t(4)),
        lambda: cm.causal_conv_step(x, w, t(4, 3, 8), slots=t(3, dtype=i32)),
        lambda: cm.selective_scan(x, x, A, b, b),  # not on a GPU
        lambda: cm.selective_scan(x, t(4, 7), A, b, b),
        lambda: cm.selective_scan(x, x.bfloat16(), A, b, b),
        lambda: cm.selective_scan(x, x, t(8, 65), t(4, 65), t(4, 65)),
        lambda: cm.selective_scan(x, x, t(7, 3), b, b),
        lambda: cm.selective_scan(x, x, A.bfloat16(), b, b),
        lambda: cm.selective_scan(x, x, A, t(4, 2), b),
        lambda: cm.selective_scan(x, x, A, t(4, 3, 3), t(4, 3, 3)),
        lambda: cm.selective_scan(x, x, A, b, t(4, 2, 3)),
        lambda: cm.selective_scan(x, x, A, b, b, D=t(7)),
        lambda: cm.selective_scan(x, x, A, b, b, z=t(3, 8)),
        lambda: cm.selective_scan(x, x, A, b, b, delta_bias=t(8).bfloat16()),
        lambda: cm.selective_scan(x, x, A, b, b, gate_activation="swish"),
        lambda: cm.selective_scan(x, x, A, b, b, initial=t(1, 8, 4)),
        lambda: cm.selective_scan(x, x, A, b, b, saved=t(5)),
        lambda: cm.selective_scan(x, x, A, b, t(3, 4).t()),
        lambda: cm.selective_scan_grad(t(3, 8), x, x, A, b, b),
        lambda: cm.selective_scan_grad(x, x, x, A, b, b, dlast=t(2, 8, 3)),
        lambda: cm.selective_step(x, x, A, b, b, t(3, 8, 3)),
        lambda: cm.selective_step(x, x, A, b, b, t(4, 8, 3).bfloat16()),
        lambda: cm.selective_step(x, x, A, b, b, t(4, 8, 3), slots=t(5, dtype=i32)),
        lambda: cm.adamw_step([], [], {"m": [], "v": []}, 1, 0.1),
        lambda: cm.adamw_step(p, p, cm.adamw_state(p), 1, 0.1),  # not on a GPU
        lambda: cm.adamw_state(p, 16),
        lambda: cm.adamw_moments(cm.adamw_state(p)),
        lambda: cm.adamw_moments(cm.adamw_state(p, 8)),  # not on a GPU
    ]
    host = {0, 24, 46, 49}  # calls that only lack a GPU
    for i, call in enumerate(bad):
        print(i, flush=True)
        with pytest.raises(ValueError) as e:
            call()
        assert ("GPU" in str(e.value)) == (i in host), e.value
