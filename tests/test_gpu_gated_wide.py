"""The gated layer's forms that its other tests' sizes do not reach: the
largest tiles (long sums with enough output tiles to fill the device), few rows
through wide layers, and dx's sum in pieces, ragged in every direction, on
whole numbers (every result exact before its one rounding)."""
import pytest
import torch

import convolution_implicit_gemm_conv2d_amd as cm
from test_gpu_gated import BF16, DEV, F32, call, exact_case, values

pytestmark = pytest.mark.gpu

# rows, channels, hidden: a long sum in the forward product, in dx, in dW
SIZES = [(4097, 1032, 2056), (4097, 4104, 520), (1100, 4104, 2056), (4352, 1024, 2048)]


@pytest.mark.parametrize("keep", [False, True])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_whole_numbers(size, keep):
    print(size, keep, flush=True)
    exact_case(*size, BF16, keep, "relu")
    torch.cuda.empty_cache()


# one row to a few hundred: weights are the stream, dx's sum is cut
FEW = [(1, 264, 1032), (16, 257, 1000), (17, 520, 2050), (33, 64, 4100), (64, 1000, 700), (66, 520, 1032), (130, 257, 3000),
       (200, 1032, 515)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("size", FEW, ids=str)
def test_few_rows(size, dtype):
    print(size, dtype, flush=True)
    exact_case(*size, dtype, False, "relu")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("keep", [False, True])
@pytest.mark.parametrize("rows,C,F", [(5, 40, 20), (70, 72, 33), (130, 33, 7), (300, 64, 1000), (40, 300, 2000)])
def test_workspace_contents_do_not_matter(rows, C, F, keep, dtype):
    # a workspace of NaN: what a call has not written it must not read
    x, wg, wu, bg, bu, dh = values(rows + F, rows, C, F, dtype, True)
    h, saved, want = call(x, wg, wu, bg, bu, "silu", dh, keep)
    a = [t.to(DEV) for t in (x, wg, wu, bg, bu)]
    need = cm.conv_gated_bwd_workspace_size(rows, C, F, cm.CONV_BF16 if dtype == BF16 else cm.CONV_F32)
    ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV)
    got = cm.gated_feed_forward_grad(dh.to(DEV), *a, activation="silu", saved=saved, workspace=ws)
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert torch.isfinite(g).all() and torch.equal(g, w)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("C,post,pre,gate", [(40, "layer", "rms", "image"), (1000, "rms", "layer", "full"), (20, "none", "rms", "none")])
def test_norm_workspace_contents_do_not_matter(C, post, pre, gate, dtype):
    gen = torch.Generator().manual_seed(C)
    t = lambda *s: torch.randn(s, generator=gen).to(dtype).to(DEV)  # noqa: E731
    images, rows = 3, 50
    x, f, dy, da = (t(images, rows, C) for _ in range(4))
    kw = dict(scale=t(C), gate={"none": None, "image": t(images, C), "full": t(images, rows, C)}[gate],
              post_weight=None if post == "none" else t(C), post_bias=t(C) if post == "layer" else None,
              pre_weight=t(C), pre_bias=t(C) if pre == "layer" else None, post=post, pre=pre, gate_activation="sigmoid")
    want = cm.block_norm_grad(dy, da, x, f, **kw)
    gate_rows = {"none": 0, "image": rows, "full": 1}[gate]
    ws = torch.full((cm.conv_block_norm_bwd_workspace_size(images * rows, C, gate_rows),), 255, dtype=torch.uint8, device=DEV)
    got = cm.block_norm_grad(dy, da, x, f, workspace=ws, **kw)
    torch.cuda.synchronize()
    for k, w in want.items():
        assert w is None or (torch.isfinite(got[k]).all() and torch.equal(got[k], w)), k


# rows that are no whole number of 16 bytes: copied first by the gradient, and
# by the forward product from 2^30 products on
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("keep", [False, True])
@pytest.mark.parametrize("size", [(700, 257, 515), (300, 1001, 300), (5000, 33, 600), (2100, 1031, 520), (4100, 1031, 2056)], ids=str)
def test_padded_copies(size, keep, dtype):
    if size[0] * size[1] * size[2] > 1 << 32 and dtype == F32:
        pytest.skip("the wide tiles are bf16's")
    print(size, keep, dtype, flush=True)
    need = cm.conv_gated_fwd_workspace_size(*size, cm.CONV_BF16 if dtype == BF16 else cm.CONV_F32)
    assert (need > 0) == (size[0] * size[1] * size[2] >= 1 << 30)
    exact_case(*size, dtype, keep, "relu")


def test_forward_with_and_without_a_workspace():
    x, wg, wu, bg, bu, _ = (t.to(DEV) for t in values(12, 2100, 1031, 520, BF16, True))
    h = torch.empty(2100, 520, dtype=BF16, device=DEV)
    cm.conv_gated_fwd(x, wg, wu, bg, bu, h, None, 2100, 1031, 520, cm.ACTIVATIONS["silu"], cm.CONV_BF16)
    torch.cuda.synchronize()
    # the same sums in another order: whole stages from the first value on
    got = cm.gated_feed_forward(x, wg, wu, bg, bu)
    assert torch.equal(h, got)
