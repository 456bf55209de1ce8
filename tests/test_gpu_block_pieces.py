"""The norms' gradient where its rows are cut into as many pieces as the device
holds workgroups: every form of the kernel (with and without biases, a gate row
shared or not, both types), uneven pieces, and a workspace of exactly the size
that is asked for, with bytes behind it that have to stay.  Then the fp32 gated
layer at widths that 128 x 64 tiles cover with fewer, on whole numbers (every
result exact before its one rounding)."""
import pytest
import torch

import convolution_implicit_gemm_conv2d_amd as cm
from test_gpu_block_norm import BF16, DEV, F32, check, dev, make
from test_gpu_gated import exact_case

pytestmark = pytest.mark.gpu

FORMS = [("rms", "rms", "full"), ("layer", "layer", "full"), ("rms", "rms", "image"), ("layer", "rms", "image"),
         ("rms", "layer", "none")]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,images,C", [(4203, 3, 200), (4203, 3, 520), (2103, 3, 1500), (1103, 1, 2048), (1106, 2, 4096),
                                           (1103, 1, 4500), (530, 5, 8192)])
def test_pieces(rows, images, C, dtype):
    for i, (post, pre, gate) in enumerate(FORMS):
        print(rows, images, C, dtype, post, pre, gate, flush=True)
        d, dy, da = make(rows + i, rows, C, dtype, post, pre, gate, i % 2 == 0, images)
        check(d, dy, da, post, pre, "silu")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,C", [(1, 520), (9, 64), (2050, 40), (2050, 600), (4100, 1000), (1030, 4096), (520, 8192), (64, 9000)])
def test_workspace_is_large_enough(rows, C, dtype):
    gate_rows = {"none": 0, "image": rows, "full": 1}
    for post, pre, gate in FORMS:
        print(rows, C, dtype, post, pre, gate, flush=True)
        d, dy, da = make(rows, rows, C, dtype, post, pre, gate, True, 1)
        kw, how = dev(d), dict(post=post, pre=pre, gate_activation="silu")
        need = cm.conv_block_norm_bwd_workspace_size(rows, C, gate_rows[gate])
        room = torch.full((need + (1 << 20),), 171, dtype=torch.uint8, device=DEV)
        got = cm.block_norm_grad(dy.to(DEV), da.to(DEV), **kw, **how, workspace=room[:need])
        want = cm.block_norm_grad(dy.to(DEV), da.to(DEV), **kw, **how)
        torch.cuda.synchronize()
        assert (room[need:] == 171).all()
        for k, w in want.items():
            assert w is None or torch.equal(got[k], w), k


@pytest.mark.parametrize("keep", [False, True])
@pytest.mark.parametrize("size", [(300, 190, 96), (257, 33, 160), (515, 61, 97), (1001, 190, 517), (700, 64, 32), (1900, 320, 65)], ids=str)
def test_narrow_fp32(size, keep):
    print(size, keep, flush=True)
    exact_case(*size, F32, keep, "relu")
