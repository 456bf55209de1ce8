"""The selective scan, its gradient and its token form against their 64-bit
values with running bounds."""
import pytest
import torch

import convolution_implicit_gemm_conv2d_amd as cm
import sequence_reference as sr
from running_bounds import within

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF16, F32 = torch.bfloat16, torch.float32


class Inputs:
    """Tensors of a call, on the host; steps between about 0.001 and 1."""

    def __init__(self, rows, C, N, G, dtype, seqs, seed=0, plus=True):
        gen = torch.Generator().manual_seed(seed)
        r = lambda *s, std=1.0, t=dtype: (torch.randn(s, generator=gen) * std).to(t)  # noqa: E731
        self.x, self.z, self.dy = r(rows, C), r(rows, C), r(rows, C)
        self.delta = r(rows, C, std=0.5) if plus else r(rows, C, std=0.3).abs()
        self.bias = (torch.rand(C, generator=gen) * 7 - 6) if plus else None
        self.A = -(torch.rand(C, N, generator=gen) * N + 0.1)
        self.B, self.C, self.D = r(rows, G, N), r(rows, G, N), r(C, t=F32)
        self.initial, self.dlast = r(seqs, C, N, t=F32), r(seqs, C, N, t=F32)


def dev(t):
    return None if t is None else t.to(DEV)


def wider(t, extra):
    if not extra:
        return t.to(DEV)
    flat = t.reshape(t.shape[0], -1)
    w = torch.full((flat.shape[0], flat.shape[1] + extra), float("nan"), dtype=t.dtype, device=DEV)
    w[:, 1:1 + flat.shape[1]] = flat.to(DEV)
    return w[:, 1:1 + flat.shape[1]].unflatten(1, t.shape[1:])


def starts_of(lengths, front):
    s = [front]
    for n in lengths:
        s.append(s[-1] + n)
    return s


def check(i, spans, lead, starts, extra=0, kind="silu", plus=True, full=True, keep=True):
    rows, C = i.x.shape
    seqs = len(spans)
    st = None if starts is None else torch.tensor(starts, dtype=torch.int32, device=DEV)
    z, D, bias, initial, dlast = (t if full else None for t in (i.z, i.D, i.bias, i.initial, i.dlast))
    if plus and not full:
        bias = None
    view = lambda t: t.unflatten(0, lead[:-1]) if len(lead) == 3 else t  # noqa: E731
    ins = [view(wider(t, extra)) for t in (i.x, i.delta)] + [i.A.to(DEV)] + [view(wider(t, extra)) for t in (i.B, i.C)]
    how = dict(D=dev(D), z=None if z is None else view(wider(z, extra)), delta_bias=dev(bias), softplus=plus, gate_activation=kind, starts=st, initial=dev(initial))
    last = torch.full((seqs, C, i.A.shape[1]), float("nan"), device=DEV)
    saved = cm.selective_scan_saved(ins[0], ins[2]) if keep else None
    y = cm.selective_scan(*ins, last=last, saved=saved, **how)
    g = cm.selective_scan_grad(view(i.dy.to(DEV)), *ins, dlast=dev(dlast), saved=saved, **how)
    torch.cuda.synchronize()
    ref = sr.scan(i.x, i.delta, i.A, i.B, i.C, D, z, bias, plus, kind, spans, initial, i.dy, dlast)
    within("y", y.reshape(rows, C), ref["y"])
    within("last", last, ref["last"])
    for k, v in g.items():
        if v is None:
            assert not full or k == "delta_bias"
            continue
        within("d" + k, v.reshape(ref[k].v.shape), ref[k])
    return y, last, g


# channels, states, groups
WIDTHS = [(1, 1, 1), (5, 3, 1), (16, 4, 2), (63, 5, 1), (64, 16, 1), (65, 8, 5), (40, 16, 4), (20, 17, 1), (33, 24, 3), (12, 32, 2), (10, 33, 1), (18, 48, 2),
          (6, 64, 1)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("C,N,G", WIDTHS)
@pytest.mark.parametrize("S,L", [(1, 1), (3, 2), (2, 16), (2, 37)])
def test_prompts(dtype, C, N, G, S, L):
    i = Inputs(S * L, C, N, G, dtype, S)
    check(i, sr.spans_of(S * L, S), (S, L, C), None)
    check(i, sr.spans_of(S * L, S), (S, L, C), None, full=False, keep=False)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("C,N,G,extra", [(70, 16, 2, 0), (9, 6, 1, 3), (24, 24, 3, 1), (8, 40, 1, 0)])
@pytest.mark.parametrize("lengths,front,behind", [([1], 0, 0), ([5, 0, 1, 40, 2], 0, 3), ([0, 0, 7], 2, 1), ([0], 0, 4), ([0, 33, 0], 1, 0),
                                                  ([16, 16, 0, 32], 0, 16), ([63, 130, 1, 0, 66, 3], 0, 0)])
def test_packed_sequences(dtype, C, N, G, extra, lengths, front, behind):
    starts = starts_of(lengths, front)
    rows = starts[-1] + behind
    i = Inputs(rows, C, N, G, dtype, len(lengths))
    for keep in (True, False):
        y, _, g = check(i, sr.spans_of(rows, starts=starts), (rows, C), starts, extra=extra, keep=keep)
        for t in (y, g["x"], g["delta"], g["z"], g["B"], g["C"]):
            assert (t[:front] == 0).all() and (t[starts[-1]:] == 0).all()


@pytest.mark.parametrize("S,L,C,N", [(1, 700, 33, 16), (2, 333, 8, 5), (1, 517, 4, 33)])
def test_long_prompts_in_pieces(S, L, C, N):
    i = Inputs(S * L, C, N, 1, F32, S)
    check(i, sr.spans_of(S * L, S), (S, L, C), None)
    check(i, sr.spans_of(S * L, S), (S, L, C), None, full=False, keep=False)


@pytest.mark.parametrize("kind", ["none", "sigmoid", "relu", "tanh"])
def test_gates_and_plain_steps(kind):
    for plus in (True, False):
        i = Inputs(40, 20, 16, 1, F32, 2, plus=plus)
        check(i, sr.spans_of(40, 2), (2, 20, 20), None, kind=kind, plus=plus)


def test_outputs_of_the_caller_keep_rows_of_no_sequence():
    i = Inputs(40, 24, 16, 1, F32, 3)
    st = torch.tensor([3, 9, 9, 25], dtype=torch.int32, device=DEV)
    ins = [t.to(DEV) for t in (i.x, i.delta, i.A, i.B, i.C)]
    out = torch.full((40, 24), 7.0, device=DEV)
    cm.selective_scan(*ins, starts=st, out=out)
    y = cm.selective_scan(*ins, starts=st)
    assert (out[:3] == 7).all() and (out[25:] == 7).all() and torch.equal(out[3:25], y[3:25])


def test_rows_behind_the_last_sequence_may_hold_anything():
    i = Inputs(64, 24, 16, 1, F32, 2)
    ins = [t.to(DEV).clone() for t in (i.x, i.delta, i.A, i.B, i.C)]
    st = torch.tensor([0, 9, 41], dtype=torch.int32, device=DEV)
    y, g = cm.selective_scan(*ins, starts=st), cm.selective_scan_grad(i.dy.to(DEV), *ins, starts=st)
    for k in (0, 1, 3, 4):
        ins[k][41:] = float("nan")
    dy = i.dy.to(DEV).clone()
    dy[41:] = float("inf")
    y2, g2 = cm.selective_scan(*ins, starts=st), cm.selective_scan_grad(dy, *ins, starts=st)
    assert torch.equal(y, y2)
    for k, v in g.items():
        assert v is None or torch.equal(v, g2[k]), k


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,C,N,G,extra", [(1, 1, 1, 1, 0), (3, 37, 5, 1, 2), (64, 128, 16, 2, 0), (5, 300, 24, 3, 1), (2, 9, 64, 1, 0), (4, 1030, 8, 1, 0)])
def test_tokens(dtype, rows, C, N, G, extra):
    i = Inputs(rows, C, N, G, dtype, rows)
    pool = rows + 3
    state = torch.randn(pool, C, N, generator=torch.Generator().manual_seed(9))
    slots = torch.randperm(pool, generator=torch.Generator().manual_seed(5))[:rows].to(torch.int32)
    sd = state.to(DEV)
    ins = [wider(i.x, extra), wider(i.delta, extra), i.A.to(DEV), wider(i.B, extra), wider(i.C, extra)]
    how = dict(D=i.D.to(DEV), z=wider(i.z, extra), delta_bias=i.bias.to(DEV))
    y = cm.selective_step(*ins, sd, slots=slots.to(DEV), **how)
    first = state[slots.long()]
    ref = sr.scan(i.x, i.delta, i.A, i.B, i.C, i.D, i.z, i.bias, True, "silu", [(t, t + 1) for t in range(rows)], first)
    within("y", y, ref["y"])
    within("state", sd[slots.long().to(DEV)], ref["last"])
    rest = torch.ones(pool, dtype=torch.bool)
    rest[slots.long()] = False
    assert torch.equal(sd.cpu()[rest], state[rest])
    sd2 = first.to(DEV)
    assert torch.equal(cm.selective_step(*ins, sd2, **how), y) and torch.equal(sd2, sd[slots.long().to(DEV)])


def test_rows_of_one_slot_follow_each_other_and_padding_is_left():
    i = Inputs(7, 300, 16, 1, F32, 2)
    slots = torch.tensor([1, -1, 0, 1, 5, 1, 0], dtype=torch.int32, device=DEV)
    ins = [t.to(DEV) for t in (i.x, i.delta, i.A, i.B, i.C)]
    state = i.initial.to(DEV).clone()
    out = torch.full((7, 300), 7.0, device=DEV)
    cm.selective_step(*ins, state, slots=slots, out=out)
    for s, r in ((0, [2, 6]), (1, [0, 3, 5])):
        one = i.initial[s:s + 1].to(DEV).clone()
        for row in r:  # one call after another
            y = cm.selective_step(*[t if k == 2 else t[row:row + 1] for k, t in enumerate(ins)], one)
            assert torch.equal(y[0], out[row])
        assert torch.equal(one[0], state[s])
    assert (out[[1, 4]] == 7).all()


def test_a_prompt_in_parts_goes_on_by_tokens():
    i = Inputs(90, 48, 16, 1, F32, 1)
    ins = [t.to(DEV) for t in (i.x, i.delta, i.A, i.B, i.C)]
    whole, end = cm.selective_scan(*ins, last=(last := torch.empty(1, 48, 16, device=DEV))), last
    state, parts = None, []
    cut = lambda a, e: [t if k == 2 else t[a:e] for k, t in enumerate(ins)]  # noqa: E731
    for a, e in ((0, 33), (33, 34), (34, 80)):
        last = torch.empty(1, 48, 16, device=DEV)
        parts.append(cm.selective_scan(*cut(a, e), initial=state, last=last))
        state = last
    for t in range(80, 90):
        parts.append(cm.selective_step(*cut(t, t + 1), state))
    # two orders of the same sums: within the bounds of both
    ref = sr.scan(i.x, i.delta, i.A, i.B, i.C, None, None, None, True, "silu", [(0, 90)])
    within("whole", whole, ref["y"])
    within("parts", torch.cat(parts), ref["y"])
    within("state", state, ref["last"])
    within("end", end, ref["last"])


def test_streams_graphs_and_runs():
    i = Inputs(900, 72, 16, 1, BF16, 3)
    st = torch.tensor([0, 300, 301, 890], dtype=torch.int32, device=DEV)
    ins = [t.to(DEV) for t in (i.x, i.delta, i.A, i.B, i.C)]
    for how in (dict(starts=st, z=i.z.to(DEV)), dict()):
        go = lambda s=None: (cm.selective_scan(*ins, stream=s, **how), cm.selective_scan_grad(i.dy.to(DEV), *ins, stream=s, **how))  # noqa: E731
        y, g = go()
        torch.cuda.synchronize()
        dy = i.dy.to(DEV)
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        for stream in (s, s.cuda_stream):
            y2, g2 = cm.selective_scan(*ins, stream=stream, **how), cm.selective_scan_grad(dy, *ins, stream=stream, **how)
            torch.cuda.synchronize()
            assert torch.equal(y, y2) and all(v is None or torch.equal(v, g2[k]) for k, v in g.items())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y2, g2 = cm.selective_scan(*ins, **how), cm.selective_scan_grad(dy, *ins, **how)
        for _ in range(3):
            y2.zero_()
            [v.zero_() for v in g2.values() if v is not None]
            go()
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, y2) and all(v is None or torch.equal(v, g2[k]) for k, v in g.items())
