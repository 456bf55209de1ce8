"""The global gradient norm and clipping against their 64-bit forms.

Roundings counted: squares and sums are in fp64, so the norm carries one
rounding to fp32 (2^-24 relative); the coefficient three more (sum, quotient,
and the norm's own), a product one, and its type's."""
import math

import pytest
import torch

import block_reference as br
import convolution_implicit_gemm_conv2d_amd as cm

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF16, F32 = torch.bfloat16, torch.float32


def tensors(sizes, seed=0, std=0.01, types=(BF16, F32)):
    gen = torch.Generator().manual_seed(seed)
    return [(torch.randn(n, generator=gen) * std).to(types[i % len(types)]) for i, n in enumerate(sizes)]


def norm64(ts):
    return math.sqrt(sum(float((t.double() ** 2).sum()) for t in ts))


LISTS = [[1], [0, 5], [7, 8, 9], [2047, 2048, 2049], [1] * 127 + [5], [3] * 128, [11] * 129, [100_003, 1, 65_536, 0, 31],
         [1000 + i for i in range(300)], [1_500_001, 40_000, 3]]


@pytest.mark.parametrize("sizes", LISTS, ids=[f"{len(s)}x{max(s)}" for s in LISTS])
def test_norm_and_clip(sizes):
    ts = tensors(sizes, seed=len(sizes))
    want = norm64(ts)
    dev = [t.to(DEV) for t in ts]
    got = cm.gradient_norm(dev)
    assert got.dtype == F32 and got.shape == ()
    for max_norm in (want / 3, want * 3, 0.0):
        out = [torch.full_like(t, -7.0) for t in dev]
        norm = cm.clip_gradients(dev, max_norm, out=out)
        inplace = [t.clone() for t in dev]
        again = cm.clip_gradients(inplace, max_norm)
        torch.cuda.synchronize()
        for v in (got, norm, again):
            assert abs(v.item() - want) <= 2 * br.U32 * want
        c = min(1.0, max_norm / (want + 1e-6))
        for t, o, p in zip(ts, out, inplace):
            br.within("clipped", o, t.double() * c, t.double().abs() * c, 5)
            assert torch.equal(o, p)
        for t, d in zip(ts, dev):
            assert torch.equal(t, d.cpu())  # the gradients themselves stand


def test_unclipped_in_place_keeps_every_bit():
    ts = [t.to(DEV) for t in tensors([5000, 77])]
    keep = [t.clone() for t in ts]
    cm.clip_gradients(ts, 1e9)
    assert all(torch.equal(a, b) for a, b in zip(ts, keep))


def test_squares_beyond_fp32():
    for v in (3e30, 2e-30):
        t = torch.full((1000,), v, device=DEV)
        assert abs(cm.gradient_norm([t]).item() / (v * math.sqrt(1000)) - 1) < 1e-6


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_not_finite(bad):
    a, b = torch.ones(10, device=DEV), torch.ones(10, device=DEV, dtype=BF16)
    a[3] = bad
    out = [torch.empty_like(a), torch.empty_like(b)]
    n = cm.clip_gradients([a, b], 1.0, out=out)
    assert math.isnan(n.item()) if math.isnan(bad) else math.isinf(n.item())
    assert torch.isnan(out[0][3])
    assert torch.isnan(out[1]).all() if math.isnan(bad) else (out[1] == 0).all()


def test_views_at_odd_offsets():
    base = torch.full((5000,), -7.0, device=DEV, dtype=BF16)
    g = tensors([2222], types=(BF16,))[0]
    for at in (1, 3, 8):
        v = base[at:at + 2222]
        base.fill_(-7.0)
        v.copy_(g)
        out = torch.empty(2300, device=DEV, dtype=BF16)
        w = out[at + 1:at + 1 + 2222]
        out.fill_(-7.0)
        cm.clip_gradients([v], 0.1, out=[w])
        c = min(1.0, 0.1 / (norm64([g]) + 1e-6))
        br.within("view", w, g.double() * c, g.double().abs() * c, 5)
        assert (out[:at + 1] == -7).all() and (out[at + 1 + 2222:] == -7).all()
        cm.clip_gradients([v], 0.1)
        assert torch.equal(v, w) and (base[:at] == -7).all() and (base[at + 2222:] == -7).all()


def test_same_on_every_run_streams_and_graph():
    ts = [t.to(DEV) for t in tensors([300_000, 17, 90_001, 5])]
    out = [torch.empty_like(t) for t in ts]
    n = cm.clip_gradients(ts, 0.5, out=out)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in (None, s, s.cuda_stream):
        o = [torch.empty_like(t) for t in ts]
        torch.cuda.synchronize()
        m = cm.clip_gradients(ts, 0.5, out=o, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(n, m) and all(torch.equal(a, b) for a, b in zip(out, o))
    o = [torch.empty_like(t) for t in ts]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m = cm.clip_gradients(ts, 0.5, out=o)
    for _ in range(3):
        cm.clip_gradients(ts, 0.25, out=[torch.empty_like(t) for t in ts])
        [t.zero_() for t in o]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(n, m) and all(torch.equal(a, b) for a, b in zip(out, o))
