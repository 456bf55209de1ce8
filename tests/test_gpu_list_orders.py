"""Lists whose tensors lie in memory alike but differ in the stride of a dimension
of one entry, which says nothing of the order."""
import pytest
import torch

import convolution_implicit_gemm_conv2d_amd as cm

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def laid(seed, stride):
    """[4, 1, 5], the last dimension the slowest."""
    t = torch.empty_strided((4, 1, 5), (1, stride, 4), device=DEV)
    return t.copy_(torch.randn(4, 1, 5, generator=torch.Generator().manual_seed(seed)))


@pytest.mark.parametrize("bits", [32, 8])
def test_step(bits):
    p, g, copy = laid(1, 4), laid(2, 1), laid(3, 20)
    flat = [v.permute(2, 1, 0).clone() for v in (p, g)]
    state, plain = cm.adamw_state([p], bits), cm.adamw_state([flat[0]], bits)
    if bits == 32:
        state["m"][0] = laid(4, 7).zero_()
    cm.adamw_step([p], [g], state, 1, 1e-2, copies=[copy])
    cm.adamw_step([flat[0]], [flat[1]], plain, 1, 1e-2)
    assert torch.equal(p.permute(2, 1, 0), flat[0]) and torch.equal(copy, p)
    with pytest.raises(ValueError):
        cm.adamw_step([p], [g.contiguous()], state, 2, 1e-2)


def test_clipping():
    g, out = laid(1, 4), laid(2, 1)
    cm.clip_gradients([g], 0.5, out=[out])
    assert torch.allclose(out, g * (0.5 / g.norm()), rtol=1e-5)
    with pytest.raises(ValueError):
        cm.clip_gradients([g], 0.5, out=[torch.empty(4, 1, 5, device=DEV)])
