"""What a call of the operators along a sequence and of the optimizer step does
beside its results: armed events, versions, inference tensors, strided inputs,
refusals that need a device."""
import pytest
import torch

import convolution_implicit_gemm_conv2d_amd as cm
from test_gpu_block_events import stamped
from test_gpu_block_versions import saved_by_a_graph, written

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def t(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype, device=DEV)


def test_events():
    x, w = t(400, 40), t(40, 4)
    st = torch.tensor([0, 300, 400], dtype=torch.int32, device=DEV)
    ins = (x, x, t(40, 16) - 1, t(400, 16), t(400, 16))
    p = [t(100) for _ in range(60)]  # two launches
    state = cm.adamw_state(p, 8)
    for call in (lambda: cm.causal_conv(x, w), lambda: cm.causal_conv_grad(x, x, w), lambda: cm.causal_conv_step(x, w, t(400, 3, 40)),
                 lambda: cm.selective_scan(*ins), lambda: cm.selective_scan(*ins, starts=st), lambda: cm.selective_scan_grad(x, *ins),
                 lambda: cm.selective_scan_grad(x, *ins, starts=st, saved=cm.selective_scan_saved(x, ins[2]).zero_()),
                 lambda: cm.selective_step(*ins, t(400, 40, 16)), lambda: cm.adamw_step(p, [t(100) for _ in p], state, 1, 0.1),
                 lambda: cm.adamw_moments(state)):
        stamped(call)


def test_what_is_written_counts_a_version():
    x, w, A, b = t(6, 8), t(8, 4), t(8, 3) - 1, t(6, 3)
    for shape, call in (((6, 8), lambda v: cm.causal_conv(x, w, out=v)), ((1, 3, 8), lambda v: cm.causal_conv(x, w, last=v)),
                        ((6, 3, 8), lambda v: cm.causal_conv_step(x, w, v)), ((6, 8), lambda v: cm.causal_conv_step(x, w, t(6, 3, 8), out=v)),
                        ((6, 8), lambda v: cm.selective_scan(x, x, A, b, b, out=v)), ((1, 8, 3), lambda v: cm.selective_scan(x, x, A, b, b, last=v)),
                        ((24,), lambda v: cm.selective_scan(x, x, A, b, b, saved=v)), ((6, 8, 3), lambda v: cm.selective_step(x, x, A, b, b, v)),
                        ((8,), lambda v: cm.adamw_step([v], [t(8)], cm.adamw_state([v]), 1, 0.1)),
                        ((8,), lambda v: cm.adamw_step([t(8)], [t(8)], cm.adamw_state([v]), 1, 0.1, copies=[v]))):
        v, loss = saved_by_a_graph(*shape)
        call(v.detach())
        written(loss)
    v, loss = saved_by_a_graph(6, 8)
    cm.causal_conv(v.detach(), w)
    cm.selective_scan(v.detach(), x, A, b, b)
    loss.backward()  # read alone


def test_inference_tensors_are_taken():
    with torch.inference_mode():
        x, w, A, b, state, scan, p = t(6, 8), t(8, 4), t(8, 3) - 1, t(6, 3), t(6, 3, 8), t(6, 8, 3), t(8)
    cm.causal_conv_step(x, w, state)
    cm.selective_step(x, x, A, b, b, scan)
    cm.adamw_step([p], [t(8)], cm.adamw_state([p]), 1, 0.1)
    torch.cuda.synchronize()


def test_outputs_that_overlap_inputs_are_refused():
    x, w, A, b = t(6, 8), t(8, 4), t(8, 3) - 1, t(6, 3)
    wide = t(6, 16)
    state = t(1, 3, 8)
    for call in (lambda: cm.causal_conv(x, w, out=x), lambda: cm.causal_conv(x, w, initial=state, last=state), lambda: cm.causal_conv(wide[:, 8:], w, out=wide.view(12, 8)[:6]),
                 lambda: cm.selective_scan(x, x.clone(), A, b, b, out=x), lambda: cm.selective_step(x, x.clone(), A, b, b, t(6, 8, 3), out=x),
                 lambda: cm.adamw_step([x], [x], cm.adamw_state([x]), 1, 0.1), lambda: cm.adamw_step([x, x], [wide[:, :8].clone()] * 2, cm.adamw_state([x, x]), 1, 0.1),
                 lambda: cm.adamw_step([x], [t(6, 8)], cm.adamw_state([x]), 1, 0.1, copies=[x])):
        with pytest.raises(cm.ConvError) as e:
            call()
        assert e.value.status == cm.CONV_ERR_INVALID_ARG


def test_lists_that_do_not_fit_are_refused():
    p, g = [t(6, 8)], [t(6, 8)]
    state, eight = cm.adamw_state(p), cm.adamw_state(p, 8)
    for call in (lambda: cm.adamw_step(p, [t(48)[:47]], state, 1, 0.1), lambda: cm.adamw_step(p, g * 2, state, 1, 0.1),
                 lambda: cm.adamw_step(p, g, {"m": state["m"], "v": [t(6, 8, dtype=torch.bfloat16)]}, 1, 0.1),
                 lambda: cm.adamw_step(p, g, {**eight, "m_scale": [t(2)]}, 1, 0.1), lambda: cm.adamw_step(p, g, {**eight, "v": eight["m"]}, 1, 0.1),
                 lambda: cm.adamw_step(p, [t(8, 6).t()], state, 1, 0.1), lambda: cm.adamw_step(p, [t(6, 8).half()], state, 1, 0.1),
                 lambda: cm.adamw_step(p, g, state, t(1), 0.1), lambda: cm.adamw_step(p, g, state, 1, t(2)), lambda: cm.adamw_step(p, g, state, 1, 0.1, norm=t(1).double()),
                 lambda: cm.adamw_step(p, g, state, 1, 0.1, copies=[t(7, 8)]), lambda: cm.adamw_step(p, [None], state, 1, 0.1),
                 lambda: cm.adamw_moments(eight, out={"m": [t(47)], "v": [t(48)]})):
        with pytest.raises(ValueError):
            call()


def test_batches_without_rows():
    w, A = t(8, 4), t(8, 3) - 1
    for x in (t(0, 5, 8), t(3, 0, 8), t(0, 8)):
        S = x.shape[0] if x.dim() == 3 else 1
        b = t(*x.shape[:-1], 3)
        first, h = t(S, 3, 8) + 2, t(S, 8, 3) + 3
        last, end = torch.full_like(first, 7), torch.full_like(h, 7)
        assert cm.causal_conv(x, w, initial=first, last=last).shape == x.shape and torch.equal(first, last)
        assert cm.selective_scan(x, x, A, b, b, initial=h, last=end).shape == x.shape and torch.equal(h, end)
        g = cm.causal_conv_grad(x, x, w, initial=first, dlast=last)
        assert not g["weight"].any() and torch.equal(g["initial"], last)
        g = cm.selective_scan_grad(x, x, x, A, b, b, D=t(8), delta_bias=t(8), initial=h, dlast=end)
        assert not g["A"].any() and not g["D"].any() and not g["delta_bias"].any() and torch.equal(g["initial"], end)
    assert cm.causal_conv_step(t(0, 8), w, t(2, 3, 8)).shape == (0, 8)
    assert cm.selective_step(t(0, 8), t(0, 8), A, t(0, 3), t(0, 3), t(2, 8, 3)).shape == (0, 8)


def test_a_padded_batch_of_tokens_and_many_rows():
    """More rows than a workgroup has lanes, one slot among them many times."""
    rows = 700
    x = torch.randn(rows, 12, generator=torch.Generator().manual_seed(1)).to(DEV)
    slots = torch.arange(rows, dtype=torch.int32)
    slots[5::70] = 5
    slots[9::100] = -1
    state, w = t(rows, 3, 12), torch.ones(12, 4, device=DEV)
    y = cm.causal_conv_step(x, w, state, slots=slots.to(DEV))
    mine = [r for r in range(rows) if slots[r] == 5]
    assert torch.allclose(y[mine], cm.causal_conv(x[mine], w), rtol=1e-6, atol=1e-6)
    assert not y[9::100].any() and torch.equal(state[5], x[mine][-3:])
    alone = [r for r in range(rows) if slots[r] == r and r != 5]
    assert torch.equal(y[alone], x[alone])


@pytest.mark.parametrize("rows", [2, 3, 4, 5, 7, 255, 1023, 1025, 2051])
def test_the_same_slot_twice_wherever_it_stands(rows):
    """Slots are compared four at a time, the last ones one by one, from any address."""
    x = torch.randn(rows, 6, generator=torch.Generator().manual_seed(rows)).to(DEV)
    b, w, A = torch.ones(rows, 2, device=DEV), torch.ones(6, 4, device=DEV), t(6, 2) - 1
    far = {1, min(2, rows - 1), rows // 2, rows - 2, rows - 1}
    for pair in ((i, j) for i in (0, rows // 3) for j in far if j > i):
        i, j = pair
        slots = torch.arange(-1, rows, dtype=torch.int32, device=DEV)[1:]
        slots[j] = i
        state, h = t(rows, 3, 6), t(rows, 6, 2)
        y = cm.causal_conv_step(x, w, state, slots=slots)
        z = cm.selective_step(x, x, A, b, b, h, slots=slots)
        both, of = x[[i, j]], (b[[i, j]], b[[i, j]])
        assert torch.allclose(y[[i, j]], cm.causal_conv(both, w), rtol=1e-6, atol=1e-6)
        # a state and its two products are rounded a few times in 32 bits
        assert torch.allclose(z[[i, j]], cm.selective_scan(both, both, A, *of), rtol=1e-5, atol=1e-5)
        rest = [r for r in range(rows) if r not in pair]
        assert torch.equal(y[rest], x[rest]) and not state[j].any() and not h[j].any()


def test_rate_or_step_alone_on_the_device():
    p0, g = torch.linspace(-1, 1, 500, device=DEV), torch.linspace(2, -1, 500, device=DEV)
    got = []
    for lr, step in ((3e-3, 7), (torch.tensor(3e-3, device=DEV), 7), (3e-3, torch.tensor([7], device=DEV))):
        p = p0.clone()
        state = cm.adamw_state([p])
        cm.adamw_step([p], [g], state, step, lr, weight_decay=0.2)
        got.append(p)
    for p in got[1:]:  # the scalars of both ways are rounded from 64 bits
        assert torch.allclose(p, got[0], rtol=2 ** -21, atol=2 ** -30)


def test_calls_at_once_and_graphs_in_turn():
    """Pieces and partial sums lie in each call's own workspace."""
    gen = torch.Generator().manual_seed(4)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    sets, want = [], []
    for n, L in ((1, 1500), (2, 1100), (3, 700)):
        x, d, b, w = (r(L, 40), r(L, 40), r(L, 16), r(40, 4))
        sets.append([v.to(DEV) for v in (x, d, -torch.rand(40, 16, generator=gen), b, b.flip(0).contiguous())] + [w.to(DEV)])

    def go(x, d, A, b, c, w):
        y = cm.causal_conv(x, w, activation="silu")
        s = cm.selective_scan_saved(x, A)
        z = cm.selective_scan(y, d, A, b, c, saved=s)
        g = cm.selective_scan_grad(z, y, d, A, b, c, saved=s)
        return [y, z, g["x"], g["A"], g["B"], *(cm.causal_conv_grad(g["x"], x, w, activation="silu")[k] for k in ("x", "weight"))]

    want = [go(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = []
    for _ in range(4):
        for s, ins in zip(streams, sets):
            with torch.cuda.stream(s):
                got.append(go(*ins))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(g, want[i % len(sets)]))
    graphs, outs, pool = [], [], None
    for ins in sets:  # one pool of memory, as graphs that run in turn may share
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], pool=pool):
            outs.append(go(*ins))
        pool = pool or graphs[-1].pool()
    for _ in range(3):
        for graph, out, w in zip(graphs, outs, want):
            for t_ in out:
                t_.zero_()
            graph.replay()
            go(*sets[0])
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, w))


def test_many_short_sequences():
    """Packed rows of thousands of sequences come to what a batch of them does."""
    S, L = 3000, 3
    gen = torch.Generator().manual_seed(8)
    x, d, b = (torch.randn(S, L, n, generator=gen).to(DEV) for n in (20, 20, 4))
    A = -torch.rand(20, 4, generator=gen).to(DEV)
    st = torch.arange(0, S * L + 1, L, dtype=torch.int32, device=DEV)
    flat = [v.reshape(S * L, -1) for v in (x, d, b)]
    w = torch.randn(20, 4, generator=gen).to(DEV)
    assert torch.equal(cm.causal_conv(x, w).view(S * L, 20), cm.causal_conv(flat[0], w, starts=st))
    y = cm.selective_scan(x, d, A, b, b).view(S * L, 20)
    z = cm.selective_scan(flat[0], flat[1], A, flat[2], flat[2], starts=st)
    # the groups of lanes that a sum goes over may differ: four states, fp32
    assert torch.allclose(y, z, rtol=1e-5, atol=1e-5)
    a = cm.selective_scan_grad(y.view(S, L, 20), x, d, A, b, b)
    c = cm.selective_scan_grad(y, flat[0], flat[1], A, flat[2], flat[2], starts=st)
    # fp32 sums over 4 states and 20 channels in another order
    for k in ("x", "delta", "B", "C"):
        assert torch.allclose(a[k].view(S * L, -1), c[k], rtol=1e-4, atol=1e-4 * a[k].abs().max().item())
