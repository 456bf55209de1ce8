"""The gated feed-forward layer against its 64-bit form.

Whole numbers first: with inputs from {-1, 0, 1}, few enough of them not 0,
every product, sum and rounded operand is exact, so each output must be the
exact value rounded once, bit for bit, whatever the tile, the padding and the
order of the sums.  Then ordinary values with every activation.  Roundings
counted there: a sum of K products makes K roundings, an activation and the
products around it at most 40; in bf16, dg and du are rounded once (half a
step of their magnitude in the sums that they enter).
"""
import pytest
import torch

import block_reference as br
import convolution_implicit_gemm_conv2d_amd as cm

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF16, F32 = torch.bfloat16, torch.float32


def whole(gen, shape, share):
    on = torch.rand(shape, generator=gen) < share
    return torch.where(on, torch.randint(0, 2, shape, generator=gen) * 2.0 - 1.0, torch.zeros(()))


def call(x, wg, wu, bg, bu, act, dh, keep):
    d = [None if t is None else t.to(DEV) for t in (x, wg, wu, bg, bu)]
    rows, F = x.numel() // x.shape[-1], wg.shape[0]
    saved = torch.full((rows, 2 * F), float("nan"), device=DEV) if keep else None
    h = cm.gated_feed_forward(*d, activation=act, saved=saved)
    g = cm.gated_feed_forward_grad(dh.to(DEV), *d, activation=act, saved=saved) if dh is not None else None
    torch.cuda.synchronize()
    return h, saved, g


# rows, channels, hidden: single tokens, every group of few rows, widths that
# are no multiple of a vector, a tile or a stage; then sizes that fill the
# device with the largest tiles in each product.
SIZES = [(1, 1, 1), (1, 8, 16), (1, 136, 40), (2, 7, 9), (16, 64, 64), (17, 72, 33), (33, 200, 70), (64, 129, 130),
         (65, 64, 64), (65, 65, 65), (100, 8, 300), (129, 130, 31), (300, 72, 264), (511, 190, 77), (700, 512, 96),
         (1000, 24, 520), (1500, 257, 65)]
LARGE = [(8200, 72, 1032), (8200, 2056, 16), (70, 4104, 2056), (16500, 40, 24), (8200, 75, 1031), (8193, 2049, 17)]


def exact_case(rows, C, F, dtype, keep, act, train=True):
    gen = torch.Generator().manual_seed(rows * 7 + C * 3 + F)
    x = whole(gen, (rows, C), min(1.0, 100 / C)).to(dtype)
    wg, wu = (whole(gen, (F, C), 0.5).to(dtype) for _ in range(2))
    bg, bu = (whole(gen, (F,), 0.7).to(dtype) for _ in range(2))
    dh = whole(gen, (rows, F), min(1.0, 200 / F)).to(dtype) if train else None
    h, saved, g = call(x, wg, wu, bg, bu, act, dh, keep)
    X, G, U, D = (t if t is None else t.to(DEV).double() for t in (x, wg, wu, dh))
    gv, uv = X @ G.t() + bg.to(DEV).double(), X @ U.t() + bu.to(DEV).double()
    assert gv.abs().max() <= 256 and uv.abs().max() <= 256  # exact in bf16
    v, d = br.act(gv, act)
    assert torch.equal(h, (v * uv).to(dtype)), "h"
    if keep:
        assert torch.equal(saved, torch.cat([gv, uv], 1).float()), "saved"
    if not train:
        return
    dg, du = D * uv * d, D * v
    want = ((dg @ G + du @ U), dg.t() @ X, du.t() @ X, dg.sum(0), du.sum(0))
    for name, got, ref in zip(("dx", "dwg", "dwu", "dbg", "dbu"), g, want):
        bad = (got != ref.to(dtype)).nonzero()
        assert bad.numel() == 0, (name, len(bad), bad[0].tolist(), bad[-1].tolist())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_whole_numbers(size, dtype):
    for keep in (False, True):
        for act in ("none", "relu"):
            print(size, dtype, keep, act, flush=True)
            exact_case(*size, dtype, keep, act)


@pytest.mark.parametrize("size", LARGE, ids=str)
def test_whole_numbers_large(size):
    print(size, flush=True)
    exact_case(*size, BF16, False, "relu")


def test_whole_numbers_large_fp32():
    for size in ((2100, 40, 1031), (2100, 1100, 24), (40, 1100, 1031)):
        print(size, flush=True)
        exact_case(*size, F32, False, "relu")


def values(seed, rows, C, F, dtype, bias):
    gen = torch.Generator().manual_seed(seed)
    t = lambda *s, std=1.0: (torch.randn(s, generator=gen) * std).to(dtype)  # noqa: E731
    w = C ** -0.5 * 1.5
    return (t(rows, C), t(F, C, std=w), t(F, C, std=w), t(F, std=0.3) if bias else None, t(F, std=0.3) if bias else None,
            t(rows, F))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kind", list(cm.ACTIVATIONS))
@pytest.mark.parametrize("rows,C,F,bias,keep", [(1, 96, 48, False, False), (45, 129, 70, True, True),
                                                (200, 256, 128, True, False), (333, 100, 190, False, True)])
def test_values(rows, C, F, bias, keep, kind, dtype):
    x, wg, wu, bg, bu, dh = values(rows + C, rows, C, F, dtype, bias)
    h, saved, g = call(x, wg, wu, bg, bu, kind, dh, keep)
    ref = br.gated(x, wg, wu, bg, bu, kind, dh)
    n = C + 40
    br.within("h", h, *ref["h"], n)
    if keep:
        br.within("g", saved[:, :F], *ref["g"], n)
        br.within("u", saved[:, F:], *ref["u"], n)
    for name, got, terms in zip(("dx", "dwg", "dwu", "dbg", "dbu"), g, (2 * F, rows, rows, rows, rows)):
        if got is None:
            continue
        also = br.half_step(BF16) * ref["rounded"][name] if dtype == BF16 and name in ("dx", "dwg", "dwu") else 0.0
        br.within(name, got, *ref[name], n + terms + 40, also)
        if dtype == BF16 and got.numel() >= 1000:
            # roundings of many terms fall to either side: in the 2-norm the
            # operands' roundings add no more than the output's own
            err = (got.cpu().double() - ref[name][0]).norm() / ref[name][0].norm()
            assert err <= 2 * br.half_step(BF16), (name, err.item())


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_gradient_against_differences(dtype):
    # of the kernel's own forward pass, in fp32, along random directions; the
    # step's error falls with its square, the outputs' roundings grow with 1/step
    x, wg, wu, bg, bu, dh = values(3, 20, 24, 40, F32, True)
    if dtype == BF16:
        x, wg, wu, bg, bu, dh = (t.to(BF16).float() for t in (x, wg, wu, bg, bu, dh))
    _, _, g = call(*(t.to(dtype) for t in (x, wg, wu, bg, bu)), "silu", dh.to(dtype), False)
    args = [x, wg, wu, bg, bu]
    gen = torch.Generator().manual_seed(4)
    for i, name in enumerate(("dx", "dwg", "dwu", "dbg", "dbu")):
        way = torch.randn(args[i].shape, generator=gen)
        step = 1e-2
        f = []
        for sign in (1, -1):
            moved = [a + sign * step * way if k == i else a for k, a in enumerate(args)]
            h, _, _ = call(*moved, "silu", None, False)
            f.append((h.cpu().double() * dh.double()).sum().item())
        want = (f[0] - f[1]) / (2 * step)
        got = (g[i].cpu().double() * way.double()).sum().item()
        size = (g[i].cpu().double().abs() * way.double().abs()).sum().item()
        assert abs(got - want) <= 1e-3 * size + (br.half_step(BF16) * size if dtype == BF16 else 0), (name, got, want)


def test_no_rows():
    x, wg, wu, bg, bu, dh = values(5, 0, 16, 24, BF16, True)
    h, _, g = call(x, wg, wu, bg, bu, "silu", dh, False)
    assert h.shape == (0, 24) and g[0].shape == (0, 16)
    for t in g[1:]:
        assert (t == 0).all()


def test_shapes_of_a_convolution():
    # NHWC input and OHWI weights: rows are pixels
    x, wg, wu, _, _, dh = values(6, 2 * 5 * 7, 32, 48, BF16, False)
    flat = cm.gated_feed_forward(x.to(DEV), wg.to(DEV), wu.to(DEV))
    h = cm.gated_feed_forward(x.view(2, 5, 7, 32).to(DEV), wg.view(48, 1, 1, 32).to(DEV), wu.view(48, 1, 1, 32).to(DEV))
    assert h.shape == (2, 5, 7, 48) and torch.equal(h.view(-1, 48), flat)
    g = cm.gated_feed_forward_grad(dh.view(2, 5, 7, 48).to(DEV), x.view(2, 5, 7, 32).to(DEV),
                                   wg.view(48, 1, 1, 32).to(DEV), wu.view(48, 1, 1, 32).to(DEV))
    assert g[0].shape == (2, 5, 7, 32) and g[1].shape == g[2].shape == (48, 1, 1, 32) and g[3] is None


@pytest.mark.parametrize("rows", [1, 40, 300])
def test_not_finite_stays_in_its_row(rows):
    x, wg, wu, bg, bu, _ = values(7, rows, 72, 40, BF16, True)
    x[rows - 1, 3] = float("nan")
    h = cm.gated_feed_forward(*(t.to(DEV) for t in (x, wg, wu, bg, bu))).cpu()
    assert torch.isnan(h[rows - 1]).all() and torch.isfinite(h[:rows - 1]).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,C,F", [(3, 64, 40), (150, 64, 40), (150, 33, 41)])
def test_odd_offsets_and_guards(rows, C, F, dtype):
    x, wg, wu, bg, bu, dh = values(8, rows, C, F, dtype, True)

    def moved(t, fill=None):
        b = torch.full((t.numel() + 9,), -7.0, dtype=t.dtype, device=DEV)
        v = b[3:3 + t.numel()].view(t.shape)
        if fill is None:
            v.copy_(t)
        return b, v

    a = [moved(t)[1] for t in (x, wg, wu, bg, bu)]
    bh, h = moved(torch.zeros(rows, F, dtype=dtype))
    cm.gated_feed_forward(*a, out=h)
    want, _, g = call(x, wg, wu, bg, bu, "silu", dh, False)
    assert torch.equal(h, want) and (bh[:3] == -7).all() and (bh[3 + rows * F:] == -7).all()
    outs = [moved(t) for t in (x, wg, wu, bg, bu)]
    dt = cm.CONV_BF16 if dtype == BF16 else cm.CONV_F32
    need = cm.conv_gated_bwd_workspace_size(rows, C, F, dt)
    ws = torch.full((need + 64,), 123, dtype=torch.uint8, device=DEV)
    cm.conv_gated_bwd(moved(dh)[1], *a, None, *[v for _, v in outs], ws, need, rows, C, F, cm.ACTIVATIONS["silu"], dt)
    torch.cuda.synchronize()
    assert (ws[need:] == 123).all()
    for (b, v), w in zip(outs, g):
        assert torch.equal(v, w)
        assert (b[:3] == -7).all() and (b[3 + v.numel():] == -7).all()


def test_same_on_every_run_and_on_another_stream():
    x, wg, wu, bg, bu, dh = (t.to(DEV) for t in values(9, 3000, 128, 200, BF16, True))
    first = cm.gated_feed_forward_grad(dh, x, wg, wu, bg, bu)
    h = cm.gated_feed_forward(x, wg, wu, bg, bu)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in (None, s, s.cuda_stream):
        again = cm.gated_feed_forward_grad(dh, x, wg, wu, bg, bu, stream=stream)
        h2 = cm.gated_feed_forward(x, wg, wu, bg, bu, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(h, h2) and all(torch.equal(a, b) for a, b in zip(first, again))


def test_graph_replays():
    x, wg, wu, bg, bu, dh = (t.to(DEV) for t in values(10, 700, 128, 200, BF16, True))
    saved = torch.empty(700, 400, device=DEV)
    h = cm.gated_feed_forward(x, wg, wu, bg, bu, saved=saved)
    want = [h, *cm.gated_feed_forward_grad(dh, x, wg, wu, bg, bu, saved=saved),
            *cm.gated_feed_forward_grad(dh, x, wg, wu, bg, bu)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [cm.gated_feed_forward(x, wg, wu, bg, bu, saved=saved),
               *cm.gated_feed_forward_grad(dh, x, wg, wu, bg, bu, saved=saved),
               *cm.gated_feed_forward_grad(dh, x, wg, wu, bg, bu)]
    for _ in range(3):
        cm.gated_feed_forward_grad(dh, x, wg, wu, bg, bu)
        [t.zero_() for t in got]
        saved.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
