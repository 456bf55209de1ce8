"""The AdamW step over lists of tensors, against 64 bits; 8-bit states against
the codes that the definition gives in fp32, bit for bit."""
import math

import pytest
import torch

import block_reference as br
import convolution_implicit_gemm_conv2d_amd as cm

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF16, F32 = torch.bfloat16, torch.float32
KINDS = [(F32, F32, None), (BF16, BF16, None), (F32, BF16, BF16), (F32, F32, F32), (BF16, F32, F32)]


def rand(n, seed, std, dtype=F32):
    return (torch.randn(n, generator=torch.Generator().manual_seed(seed)) * std).to(dtype)


def reference(p, g, m, v, step, lr, b1, b2, eps, wd, c):
    """New p, m, v in 64 bits and their magnitudes."""
    p, g, m, v = (t.double() for t in (p, g, m, v))
    g = g * c
    m2, v2 = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g * g
    d = (v2 / (1 - b2 ** step)).sqrt() + eps
    u = lr / (1 - b1 ** step) * m2 / d
    mm = b1 * m.abs() + (1 - b1) * g.abs()
    return p * (1 - lr * wd) - u, m2, v2, p.abs() + lr / (1 - b1 ** step) * mm / d, mm


LISTS = [[1], [0, 5], [7, 8, 9, 127, 128, 129], [2047, 2048, 2049], [3] * 49, [100_003, 1, 65_536, 0, 31], [1000 + i for i in range(100)]]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("sizes", LISTS, ids=[f"{len(s)}x{max(s)}" for s in LISTS])
def test_steps(sizes, bits):
    kinds = [KINDS[i % len(KINDS)] for i in range(len(sizes))]
    ps = [rand(n, i, 0.1, k[0]) for i, (n, k) in enumerate(zip(sizes, kinds))]
    params = [p.to(DEV) for p in ps]
    copies = [None if k[2] is None else torch.full((n,), 7.0, dtype=k[2], device=DEV) for n, k in zip(sizes, kinds)]
    state = cm.adamw_state(params, bits)
    host = [t.clone() for t in ps]
    hm, hv = ([torch.zeros(n) for n in sizes] for _ in range(2))
    lr, b1, b2, eps, wd = 1e-2, 0.9, 0.95, 1e-8, 0.1
    norm = torch.tensor(3.7, device=DEV)
    for step in (1, 2, 3):
        gs = [rand(n, 100 * step + i, 0.01, k[1]) for i, (n, k) in enumerate(zip(sizes, kinds))]
        clip = dict(norm=norm, max_norm=1.0, norm_eps=1e-6) if step == 2 else {}
        c = min(1.0, 1.0 / (norm.item() + 1e-6)) if step == 2 else 1.0
        cm.adamw_step(params, [g.to(DEV) for g in gs], state, step, lr, betas=(b1, b2), eps=eps, weight_decay=wd, copies=copies, **clip)
        values = state if bits == 32 else cm.adamw_moments(state)
        torch.cuda.synchronize()
        for i, g in enumerate(gs):
            p, m, v, pm, mm = reference(host[i], g, hm[i], hv[i], step, lr, b1, b2, eps, wd, c)
            # m: clip, gradient, two products, the sum; v two more; p: those of m and
            # half of v's in its denominator (5), root, factor and eps (4), reciprocal,
            # two products, the sum (5), and the scalars' own roundings (3)
            br.within("p", params[i], p, pm, 24)
            if copies[i] is not None:
                br.within("copy", copies[i], p, pm, 24)
            if bits == 32:
                br.within("m", state["m"][i], m, mm, 5)
                br.within("v", state["v"][i], v, v, 8)
            else:
                # the nearest code: half a step of the line of q, (q + 1/2)^2 to (q + 1)^2
                # or q^2: at most (2 q + 1) / 2 + 1/4 times the scale, q <= sqrt(value / scale) + 1/2
                for name, got, want, power, most in (("m", values["m"][i], m, 1, 127), ("v", values["v"][i], v, 2, 255)):
                    w = want.abs() if power == 1 else want.sqrt()
                    gv = got.cpu().double()
                    gw = gv.abs() if power == 1 else gv.sqrt()
                    blocks = torch.nn.functional.pad(w, (0, -w.numel() % 128)).view(-1, 128)
                    scale = (blocks.amax(1) / most ** 2).repeat_interleave(128)[:w.numel()]
                    q = (w / scale.clamp(min=1e-300)).sqrt()
                    assert ((gw - w).abs() <= scale * (q + 1) * 1.001 + 1e-6 * w).all(), name
                    if power == 1:
                        assert (gv * want >= 0).all()
            host[i] = params[i].cpu()
            hm[i], hv[i] = values["m"][i].cpu().view(-1), values["v"][i].cpu().view(-1)


def codes(m, v):
    """The definition in fp32 on the host: borders counted one by one."""
    n = m.numel()
    pad = lambda t: torch.nn.functional.pad(t, (0, -n % 128)).view(-1, 128)  # noqa: E731
    m, v = pad(m), pad(v)
    tm, tv = m.abs().amax(1, keepdim=True), v.amax(1, keepdim=True)
    root = tv.double().sqrt().float()  # rounded once: the host's fp32 root is off by a place now and then
    km = torch.where(tm < 2.0 ** -100, torch.zeros_like(tm), tm * torch.tensor(1 / 16129, dtype=F32))
    kv = torch.where(tv < 2.0 ** -100, torch.zeros_like(tv), root * torch.tensor(1 / 65025, dtype=F32))
    qm, qv = torch.zeros_like(m), torch.zeros_like(v)
    for c in range(127):
        qm += m.abs() > km * ((c + 0.5) ** 2)
    for c in range(255):
        r = kv * ((c + 0.5) ** 2)
        qv += v > r * r
    qm, qv = torch.where(km > 0, qm, 0 * qm), torch.where(kv > 0, torch.where(v > 0, qv.clamp(min=1), qv), 0 * qv)
    return torch.where(m < 0, -qm, qm).view(-1)[:n].to(torch.int8), km.view(-1), qv.view(-1)[:n].to(torch.uint8), kv.view(-1)


@pytest.mark.parametrize("std", [1e-2, 1.0, 1e8, 1e-12, 1e-17, 1e-25])
def test_codes_are_the_definitions(std):
    n = 70_001
    g = rand(n, 1, std) * torch.exp(rand(n, 2, 3.0))
    g[:300] = 0
    g[1000:1128] = std
    p, state = torch.zeros(n, device=DEV), None
    state = cm.adamw_state([p], 8)
    b1, b2 = 0.9, 0.95
    f = lambda s: torch.tensor(s, dtype=F32)  # noqa: E731
    m, v = torch.zeros(n), torch.zeros(n)
    for step in (1, 2, 3):
        g = g.roll(17)
        cm.adamw_step([p], [g.to(DEV)], state, step, 0.0, betas=(b1, b2))
        m = m * f(b1) + g * f(1 - b1)
        v = v * f(b2) + g * f(1 - b2) * g
        want = codes(m, v)
        for name, t in zip(("m", "m_scale", "v", "v_scale"), want):
            assert torch.equal(state[name][0].cpu(), t), (name, step)
        wide = lambda t: t.repeat_interleave(128)[:n]  # noqa: E731
        qm, km, qv, kv = want
        qm, qv = qm.float(), qv.float()
        m = qm * qm.abs() * wide(km)
        r = qv * qv * wide(kv)
        v = r * r
        got = cm.adamw_moments(state)
        assert torch.equal(got["m"][0].cpu(), m) and torch.equal(got["v"][0].cpu(), v)


@pytest.mark.parametrize("bits", [32, 8])
def test_not_finite_gradients_show(bits):
    p = torch.ones(1000, device=DEV)
    g = torch.full((1000,), 0.1, device=DEV)
    g[3], g[500] = float("nan"), float("inf")
    state = cm.adamw_state([p], bits)
    cm.adamw_step([p], [g], state, 1, 0.1)
    assert torch.isnan(p[[3, 500]]).all() and torch.isfinite(p[[4, 499, 999]]).all()
    values = state if bits == 32 else cm.adamw_moments(state)
    assert torch.isnan(values["m"][0][3]) and not torch.isfinite(values["m"][0][500])
    if bits == 8:  # a block with such a value holds no numbers, nor codes
        assert torch.isnan(values["m"][0][:128]).all() and torch.isnan(values["m"][0][384:512]).all()
        assert (state["m"][0][:128] == 0).all() and (state["m"][0][384:512] == 0).all()
    assert torch.isfinite(values["m"][0][256:384]).all()


def test_memory_orders_views_and_neighbours():
    base = torch.full((5000,), 7.0, device=DEV)
    p = base[3:3 + 2222]
    p.copy_(rand(2222, 1, 1.0))
    keep = p.clone()
    g = rand(2222, 2, 1.0).to(DEV)
    codes_m = torch.full((2300,), 5, dtype=torch.int8, device=DEV)
    state = cm.adamw_state([p], 8)
    state["m"][0] = codes_m[1:1 + 2222]
    state["m"][0].zero_()
    cm.adamw_step([p], [g], state, 1, 1e-2)
    other, plain = [keep.clone()], cm.adamw_state([keep], 8)
    cm.adamw_step(other, [g], plain, 1, 1e-2)
    assert torch.equal(p, other[0]) and torch.equal(state["m"][0], plain["m"][0])
    assert (base[:3] == 7).all() and (base[3 + 2222:] == 7).all() and codes_m[0] == 5 and (codes_m[2223:] == 5).all()
    # a channels-last weight: elements in the order of memory
    w = rand(2 * 3 * 4 * 5, 3, 1.0).view(2, 3, 4, 5).to(DEV).to(memory_format=torch.channels_last)
    gw = rand(2 * 3 * 4 * 5, 4, 1.0).view(2, 3, 4, 5).to(DEV)
    flat, st = [w.contiguous().clone()], cm.adamw_state([w.contiguous()])
    cm.adamw_step(flat, [gw], st, 1, 1e-2)
    st = cm.adamw_state([w])
    assert st["m"][0].stride() == w.stride()
    cm.adamw_step([w], [gw.to(memory_format=torch.channels_last)], st, 1, 1e-2)
    assert torch.equal(w.contiguous(), flat[0])
    with pytest.raises(ValueError):
        cm.adamw_step([w], [gw], st, 2, 1e-2)


def test_rate_and_step_on_the_device_in_a_graph():
    ps = [rand(n, n, 1.0).to(DEV) for n in (300, 5000)]
    gs = [rand(n, n + 1, 1.0).to(DEV) for n in (300, 5000)]
    lr, step = torch.tensor(0.0, device=DEV), torch.tensor(0, device=DEV)
    mine, state = [p.clone() for p in ps], None
    state = cm.adamw_state(mine)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        cm.adamw_step(mine, gs, state, step, lr)
    other, plain = [p.clone() for p in ps], cm.adamw_state(ps)
    for s, rate in ((1, 1e-2), (2, 3e-3), (3, 1e-3)):
        step.fill_(s)
        lr.fill_(rate)
        torch.cuda.synchronize()
        graph.replay()
        cm.adamw_step(other, gs, plain, s, lr.item())
        torch.cuda.synchronize()
        for a, b in zip(mine + state["m"] + state["v"], other + plain["m"] + plain["v"]):
            # the scalars of both ways are rounded from 64 bits
            assert torch.allclose(a, b, rtol=2 ** -21, atol=2 ** -30)


def test_streams_runs_and_versions():
    ps, gs = [rand(9000, 1, 1.0)], [rand(9000, 2, 1.0)]
    s = torch.cuda.Stream()
    got = []
    for stream in (None, s, s.cuda_stream):
        p, g = [t.to(DEV) for t in ps], [t.to(DEV) for t in gs]
        state = cm.adamw_state(p, 8)
        torch.cuda.synchronize()
        cm.adamw_step(p, g, state, 1, 1e-2, stream=stream)
        torch.cuda.synchronize()
        assert p[0]._version > 0 and state["m"][0]._version > 0 and g[0]._version == 0
        got.append([p[0], *(v[0] for v in state.values())])
    for other in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(got[0], other))


def test_after_the_gradients_norm():
    """The norm in hand and the clipped list come to the same step."""
    ps, gs = [rand(n, n, 1.0).to(DEV) for n in (10, 4000)], [rand(n, n + 5, 1.0).to(DEV) for n in (10, 4000)]
    a, b = [p.clone() for p in ps], [p.clone() for p in ps]
    sa, sb = cm.adamw_state(a), cm.adamw_state(b)
    cm.adamw_step(a, gs, sa, 1, 1e-2, norm=cm.gradient_norm(gs), max_norm=0.5)
    clipped = [torch.empty_like(g) for g in gs]
    cm.clip_gradients(gs, 0.5, out=clipped)
    cm.adamw_step(b, clipped, sb, 1, 1e-2)
    assert all(torch.equal(x, y) for x, y in zip(a + sa["m"] + sa["v"], b + sb["m"] + sb["v"]))
    assert math.isfinite(a[0].sum().item())
