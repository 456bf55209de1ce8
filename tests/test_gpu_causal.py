"""The short causal convolution, its gradient and its token form against their
64-bit values with running bounds."""
import pytest
import torch

import convolution_implicit_gemm_conv2d_amd as cm
import sequence_reference as sr
from running_bounds import within

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF16, F32 = torch.bfloat16, torch.float32


def rand(*shape, seed, dtype, std=1.0):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * std).to(dtype)


def dev(t):
    return None if t is None else t.to(DEV)


def wider(t, extra):
    """The same values as a part of a wider tensor."""
    if not extra:
        return t.to(DEV)
    w = torch.full((*t.shape[:-1], t.shape[-1] + extra), float("nan"), dtype=t.dtype, device=DEV)
    w[..., 1:1 + t.shape[-1]] = t.to(DEV)
    return w[..., 1:1 + t.shape[-1]]


# lengths of packed sequences, rows in front and behind; or (S, L)
PACKED = [([1], 0, 0), ([5, 0, 1, 40, 2], 0, 3), ([0, 0, 7], 2, 1), ([0], 0, 4), ([33, 130, 1, 1, 64, 3], 1, 0)]
DENSE = [(1, 1), (3, 2), (2, 17), (5, 64), (1, 300)]


def starts_of(lengths, front):
    s = [front]
    for n in lengths:
        s.append(s[-1] + n)
    return s


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", PACKED + DENSE, ids=str)
@pytest.mark.parametrize("C,K,kind,extra", [(1, 2, "none", 0), (3, 4, "silu", 2), (4, 3, "sigmoid", 0), (37, 4, "silu", 5), (64, 8, "relu", 0), (130, 5, "tanh", 0),
                                            (1024, 4, "silu", 1024), (9, 6, "silu", 0), (12, 7, "none", 3)])
def test_forward_and_gradient(dtype, shape, C, K, kind, extra):
    packed = isinstance(shape[0], list)
    starts = starts_of(shape[0], shape[1]) if packed else None
    rows, seqs = (starts[-1] + shape[2], len(shape[0])) if packed else (shape[0] * shape[1], shape[0])
    spans = sr.spans_of(rows, seqs, starts)
    x, w, b = rand(rows, C, seed=1, dtype=dtype), rand(C, K, seed=2, dtype=dtype, std=K ** -0.5), rand(C, seed=3, dtype=dtype)
    initial, dy, dlast = rand(seqs, K - 1, C, seed=4, dtype=dtype), rand(rows, C, seed=5, dtype=dtype), rand(seqs, K - 1, C, seed=6, dtype=dtype)
    st = torch.tensor(starts, dtype=torch.int32, device=DEV) if packed else None
    lead = (rows, C) if packed else (seqs, shape[1], C)
    xd = wider(x.view(lead), extra)
    for bias, first, behind in ((b, initial, dlast), (None, None, None)):
        how = dict(activation=kind, starts=st, initial=dev(first))
        last = torch.full((seqs, K - 1, C), float("nan"), dtype=dtype, device=DEV)
        y = cm.causal_conv(xd, w.to(DEV), dev(bias), last=last, **how)
        g = cm.causal_conv_grad(dy.to(DEV).view(lead), xd, w.to(DEV), dev(bias), dlast=dev(behind), **how)
        torch.cuda.synchronize()
        ref = sr.causal(x, w, bias, kind, spans, first, dy, behind)
        within("y", y.view(rows, C), ref["y"])
        assert torch.equal(last.cpu().double(), ref["last"].v)
        within("dx", g["x"].view(rows, C), ref["x"])
        within("dw", g["weight"], ref["weight"])
        assert (g["bias"] is None) == (bias is None) and (g["initial"] is None) == (first is None)
        if bias is not None:
            within("db", g["bias"], ref["bias"])
            within("dinitial", g["initial"], ref["initial"])


def test_outputs_of_the_caller_keep_rows_of_no_sequence():
    x, w = rand(20, 24, seed=1, dtype=F32).to(DEV), rand(24, 4, seed=2, dtype=F32).to(DEV)
    st = torch.tensor([3, 9, 9, 15], dtype=torch.int32, device=DEV)
    out = torch.full((20, 24), 7.0, device=DEV)
    y = cm.causal_conv(x, w, starts=st, out=out)
    z = cm.causal_conv(x, w, starts=st)
    assert y.data_ptr() == out.data_ptr()
    assert (out[:3] == 7).all() and (out[15:] == 7).all() and (z[:3] == 0).all() and (z[15:] == 0).all()
    assert torch.equal(out[3:15], z[3:15])


def test_a_sequence_in_parts_and_a_depthwise_weight():
    x, w, b = (t.to(DEV) for t in (rand(1, 50, 40, seed=1, dtype=BF16), rand(40, 4, seed=2, dtype=BF16), rand(40, seed=3, dtype=BF16)))
    whole = cm.causal_conv(x, w.view(40, 4, 1), b, activation="silu")
    state, parts = None, []
    for a, e in ((0, 1), (1, 3), (3, 30), (30, 50)):
        last = torch.empty(1, 3, 40, dtype=BF16, device=DEV)
        parts.append(cm.causal_conv(x[:, a:e], w.view(40, 1, 4), b, activation="silu", initial=state, last=last))
        state = last
    assert torch.equal(torch.cat(parts, 1), whole)
    # the same as the library's own depthwise conv1d, cut to its causal part
    y = cm.conv1d(x, w.view(40, 4, 1), b, padding=3, groups=40, layout="NLC")[:, :50]
    assert torch.allclose(cm.causal_conv(x, w, b).float(), y.float(), rtol=2 ** -7, atol=2 ** -20)


def test_infinities_stay_in_their_window():
    x = torch.zeros(1, 40, 8, device=DEV)
    x[0, 10] = float("inf")
    x[0, 20] = float("nan")
    y = cm.causal_conv(x, torch.ones(8, 5, device=DEV))[0, :, 0]
    assert torch.isinf(y[10:15]).all() and torch.isnan(y[20:25]).all()
    rest = torch.cat([y[:10], y[15:20], y[25:]])
    assert (rest == 0).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,C,K,extra", [(1, 1, 2, 0), (3, 37, 4, 3), (64, 300, 8, 0), (17, 513, 3, 0)])
def test_tokens(dtype, rows, C, K, extra):
    pool = rows + 3
    x, w, b = rand(rows, C, seed=1, dtype=dtype), rand(C, K, seed=2, dtype=dtype), rand(C, seed=3, dtype=dtype)
    state = rand(pool, K - 1, C, seed=4, dtype=dtype)
    slots = torch.randperm(pool, generator=torch.Generator().manual_seed(5))[:rows].to(torch.int32)
    sd = state.to(DEV)
    y = cm.causal_conv_step(wider(x, extra), w.to(DEV), sd, b.to(DEV), activation="silu", slots=slots.to(DEV))
    first = state[slots.long()]
    ref = sr.causal(x, w, b, "silu", [(i, i + 1) for i in range(rows)], first)
    within("y", y, ref["y"])
    after = state.clone()
    after[slots.long()] = ref["last"].v.to(dtype)
    assert torch.equal(sd.cpu(), after)
    sd = first.to(DEV)
    again = cm.causal_conv_step(wider(x, extra), w.to(DEV), sd, b.to(DEV), activation="silu")
    assert torch.equal(again, y) and torch.equal(sd.cpu(), ref["last"].v.to(dtype))


def test_rows_of_one_slot_follow_each_other_and_padding_is_left():
    x, w = rand(7, 300, seed=1, dtype=F32).to(DEV), rand(300, 4, seed=2, dtype=F32).to(DEV)
    state = rand(2, 3, 300, seed=3, dtype=F32).to(DEV)
    slots = torch.tensor([1, -1, 0, 1, 5, 1, 0], dtype=torch.int32, device=DEV)
    one, two = (cm.causal_conv(x[list(r)].unsqueeze(0), w, initial=state[i:i + 1].clone())[0] for i, r in ((0, (2, 6)), (1, (0, 3, 5))))
    out = torch.full_like(x, 7.0)
    cm.causal_conv_step(x, w, state, slots=slots, out=out)
    assert torch.equal(out[[2, 6]], one) and torch.equal(out[[0, 3, 5]], two)
    assert (out[[1, 4]] == 7).all()
    assert torch.equal(state[1], x[[0, 3, 5]]) and torch.equal(state[0, 1:], x[[2, 6]])
    assert (cm.causal_conv_step(x, w, state, slots=slots)[[1, 4]] == 0).all()


def test_streams_graphs_and_runs():
    x, w, b = (t.to(DEV) for t in (rand(600, 72, seed=1, dtype=BF16), rand(72, 4, seed=2, dtype=BF16), rand(72, seed=3, dtype=BF16)))
    st = torch.tensor([0, 100, 101, 590], dtype=torch.int32, device=DEV)
    how = dict(activation="silu", starts=st)
    y, g = cm.causal_conv(x, w, b, **how), cm.causal_conv_grad(x, x, w, b, **how)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        y2, g2 = cm.causal_conv(x, w, b, stream=stream, **how), cm.causal_conv_grad(x, x, w, b, stream=stream, **how)
        torch.cuda.synchronize()
        assert torch.equal(y, y2) and all(torch.equal(g[k], g2[k]) for k in ("x", "weight", "bias"))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y2, g2 = cm.causal_conv(x, w, b, **how), cm.causal_conv_grad(x, x, w, b, **how)
    for _ in range(3):
        y2.zero_()
        [g2[k].zero_() for k in ("x", "weight", "bias")]
        cm.causal_conv_grad(x[:50], x[:50], w, b)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, y2) and all(torch.equal(g[k], g2[k]) for k in ("x", "weight", "bias"))
