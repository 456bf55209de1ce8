"""The block norms' gradients of batches without rows: every parameter's is zero,
a shared gate's among them, whatever the memory it is returned in held before."""
import pytest
import torch

import convolution_implicit_gemm_conv2d_amd as cm

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape,gate", [((4, 0, 24), (4, 24)), ((4, 0, 24), (24,)), ((0, 24), (24,)), ((0, 5, 24), (0, 24)),
                                        ((0, 5, 24), (24,)), ((2, 0, 3, 520), (2, 520)), ((3, 0, 7), (3, 7))], ids=str)
def test_gate_of_no_rows(shape, gate, dtype):
    C = shape[-1]
    x, f, dy, da = (torch.zeros(shape, dtype=dtype, device=DEV) for _ in range(4))
    one = torch.ones(C, dtype=dtype, device=DEV)
    z = torch.ones(gate, dtype=dtype, device=DEV)
    kw = dict(gate=z, scale=one, post_weight=one, post_bias=one, pre_weight=one, pre_bias=one, post="layer", pre="layer",
              gate_activation="sigmoid")
    for _ in range(3):
        used = [torch.full(gate, float("nan"), dtype=dtype, device=DEV) for _ in range(16)]
        torch.cuda.synchronize()
        del used  # the allocator hands these out again
        g = cm.block_norm_grad(dy, da, x, f, **kw)
        torch.cuda.synchronize()
        assert g["x"].shape == g["branch"].shape == shape
        for k in ("gate", "scale", "post_weight", "post_bias", "pre_weight", "pre_bias"):
            assert g[k].shape == kw[k].shape and torch.equal(g[k], torch.zeros_like(kw[k])), k
