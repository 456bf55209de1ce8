"""What the block operators write in a caller's tensors, automatic differentiation
sees: a graph that had saved such a tensor refuses to run backwards."""
import pytest
import torch

import convolution_implicit_gemm_conv2d_amd as cm

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def saved_by_a_graph(*shape, dtype=torch.float32):
    leaf = torch.ones(shape, device=DEV, dtype=dtype, requires_grad=True)
    t = leaf * 2
    return t, (t * t).sum()


def written(loss):
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_clipping_in_place_and_into_out():
    t, loss = saved_by_a_graph(100)
    cm.clip_gradients([t.detach()], 1.0)
    written(loss)
    t, loss = saved_by_a_graph(100)
    g = torch.ones(100, device=DEV)
    cm.clip_gradients([g], 1.0, out=[t.detach()])
    written(loss)
    assert g._version == 0
    t, loss = saved_by_a_graph(100)
    cm.gradient_norm([t.detach()])
    cm.clip_gradients([t.detach()], 1.0, out=[g])
    loss.backward()  # read alone


def test_outputs_of_the_gated_layer():
    x, w = torch.ones(3, 8, device=DEV), torch.ones(16, 8, device=DEV)
    t, loss = saved_by_a_graph(3, 16)
    cm.gated_feed_forward(x, w, w, out=t.detach())
    written(loss)
    t, loss = saved_by_a_graph(3, 32)
    cm.gated_feed_forward(x, w, w, saved=t.detach())
    written(loss)
    t, loss = saved_by_a_graph(3, 16)
    cm.gated_feed_forward_grad(t.detach(), x, w, w)
    loss.backward()
    assert x._version == 0 and w._version == 0


def test_inference_tensors_are_taken():
    with torch.inference_mode():
        g, h = torch.ones(100, device=DEV), torch.empty(3, 16, device=DEV)
        x, w = torch.ones(3, 8, device=DEV), torch.ones(16, 8, device=DEV)
    cm.clip_gradients([g], 1.0)
    cm.gated_feed_forward(x, w, w, out=h)
    torch.cuda.synchronize()
    assert abs(g[0].item() - 0.1) < 1e-6 and torch.isfinite(h).all()
