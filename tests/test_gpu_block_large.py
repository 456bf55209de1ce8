"""Block operators on tensors past 2^31 elements: rows at both ends and in the
middle against their 64-bit forms, sums over all rows from chunks in 64 bits."""
import pytest
import torch

import block_reference as br
import convolution_implicit_gemm_conv2d_amd as cm

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF16 = torch.bfloat16


def some_rows(rows):
    return torch.cat([torch.arange(0, 40), torch.arange(rows // 2 - 20, rows // 2 + 20), torch.arange(rows - 40, rows)])


def make(gen, *shape, std=1.0, mean=0.0):
    return torch.empty(shape, device=DEV, dtype=BF16).normal_(mean, std, generator=gen)


def test_norms_past_2_31_elements():
    rows, C = 2_200_001, 1000
    gen = torch.Generator(device="cuda").manual_seed(1)
    x, f = make(gen, rows, C, std=2.0), make(gen, rows, C, mean=0.2)
    s, wp, bp, wq = make(gen, C), make(gen, C, mean=1.0, std=0.1), make(gen, C), make(gen, C, mean=1.0, std=0.1)
    how = dict(scale=s, post_weight=wp, post_bias=bp, pre_weight=wq, post="layer", pre="rms")
    y, a = cm.block_norm(x, f, **how)
    pick = some_rows(rows)
    take = lambda t: t[pick.to(DEV)].cpu()  # noqa: E731
    dy = torch.zeros_like(x)
    dy[pick.to(DEV)] = make(gen, len(pick), C)
    ref = br.block_norm(take(x), take(f), None, s, wp, bp, wq, None, "layer", "rms", dy=take(dy))
    br.within("y", take(y), *ref["y"], 80)
    br.within("a", take(a), *ref["a"], 80)
    del y, a
    g = cm.block_norm_grad(dy, None, x, f, **how)  # rows of zeros add nothing to the sums
    torch.cuda.synchronize()
    for name, key in (("dx", "x"), ("df", "branch")):
        br.within(name, take(g[key]), *ref[name], 80)
    for name, key in (("ds", "scale"), ("dw_post", "post_weight"), ("db_post", "post_bias")):
        br.within(name, g[key], *ref[name], 600)


def test_gated_past_2_31_elements():
    rows, C, F = 2_100_000, 16, 1032
    gen = torch.Generator(device="cuda").manual_seed(2)
    x = make(gen, rows, C)
    wg, wu = make(gen, F, C, std=0.25), make(gen, F, C, std=0.25)
    h = cm.gated_feed_forward(x, wg, wu)
    pick = some_rows(rows)
    take = lambda t: t[pick.to(DEV)].cpu()  # noqa: E731
    dh = torch.zeros_like(h)
    dh[pick.to(DEV)] = make(gen, len(pick), F)
    ref = br.gated(take(x), wg, wu, None, None, "silu", take(dh))
    br.within("h", take(h), *ref["h"], C + 40)
    del h
    dx, dwg, dwu, _, _ = cm.gated_feed_forward_grad(dh, x, wg, wu)
    torch.cuda.synchronize()
    half = br.half_step(BF16)
    br.within("dx", take(dx), *ref["dx"], C + 2 * F + 40, half * ref["rounded"]["dx"])
    # rows of zeros add nothing, but count as roundings of the sums that hold them: none of them moves one
    br.within("dwg", dwg, *ref["dwg"], C + 2 * len(pick) + 200, half * ref["rounded"]["dwg"])
    br.within("dwu", dwu, *ref["dwu"], C + 2 * len(pick) + 200, half * ref["rounded"]["dwu"])


def test_clipping_past_2_31_elements():
    n = (1 << 31) + 12_345
    gen = torch.Generator(device="cuda").manual_seed(3)
    t = torch.empty(n, device=DEV, dtype=BF16).normal_(0, 0.01, generator=gen)
    want = sum(float(c.double().square().sum()) for c in t.split(1 << 28)) ** 0.5
    out = torch.empty_like(t)
    norm = cm.clip_gradients([t], 1.0, out=[out])
    torch.cuda.synchronize()
    assert abs(norm.item() - want) <= 2 * br.U32 * want
    c = min(1.0, 1.0 / (want + 1e-6))
    for at in (0, 1 << 30, n - 100_000):
        br.within("clipped", out[at:at + 100_000], t[at:at + 100_000].double() * c, t[at:at + 100_000].double().abs() * c, 5)
