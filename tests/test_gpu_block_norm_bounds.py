"""The block norms' gradients held to a running analysis of their arithmetic
(block_norm_bounds.py), which refuses zeros and a sum that lacks one row: every
form of the kernels, rows in pieces, long and very short rows, each gate."""
import pytest
import torch

import block_norm_bounds as bounds
import convolution_implicit_gemm_conv2d_amd as cm
from test_gpu_block_norm import BF16, DEV, F32, dev, make

pytestmark = pytest.mark.gpu

FORMS = [("rms", "rms", "full", "silu"), ("layer", "layer", "full", "sigmoid"), ("rms", "rms", "image", "silu"),
         ("layer", "rms", "image", "sigmoid"), ("rms", "layer", "none", "none"), ("none", "layer", "row", "silu"),
         ("layer", "none", "full", "silu"), ("none", "rms", "none", "none")]


def held(rows, images, C, dtype, post, pre, gate, kind, scale):
    print(rows, images, C, dtype, post, pre, gate, kind, flush=True)
    d, dy, da = make(rows + C, rows, C, dtype, post, pre, gate, scale, images)
    da = da if pre != "none" else None
    kw = dev(d)
    got = cm.block_norm_grad(dy.to(DEV), None if da is None else da.to(DEV), **kw, post=post, pre=pre, gate_activation=kind)
    torch.cuda.synchronize()
    flat = lambda t: None if t is None else t.reshape(-1, C)  # noqa: E731
    want = bounds.gradients(flat(dy), flat(da), flat(d["x"]), flat(d["branch"]), flat(d["gate"]), d["scale"], d["post_weight"],
                            d["post_bias"], d["pre_weight"], d["pre_bias"], post, pre, kind)
    for name, g in got.items():
        if g is None:
            assert name not in want or kw[name] is None, name
            continue
        worst = bounds.off(g, want[name])
        print(f"  {name}: {worst:.3f} of its tolerance", flush=True)
        assert worst <= 1.0, (name, worst)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,images,C", [(4203, 3, 60), (4203, 3, 200), (4203, 3, 520), (2103, 3, 1500), (1103, 1, 2048),
                                           (1106, 2, 4096), (603, 3, 4500), (530, 5, 8192)])
def test_pieces(rows, images, C, dtype):
    for i, form in enumerate(FORMS):
        held(rows, images, C, dtype, *form, i % 2 == 0)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,images,C", [(1, 1, 96), (12, 3, 1000), (700, 7, 96), (2600, 2, 33), (3000, 1500, 16), (420, 6, 9001),
                                           (60, 3, 16384), (50, 5, 16391), (24, 2, 20000), (999, 9, 1), (800, 4, 5), (901, 1, 7)])
def test_rows_and_widths(rows, images, C, dtype):
    for i, form in enumerate(FORMS):
        if C == 1 and "layer" in form[:2]:
            continue  # every value is its own mean
        held(rows, images, C, dtype, *form, i % 2 == 1)
