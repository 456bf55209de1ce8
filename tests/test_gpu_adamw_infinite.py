"""Blocks of 8-bit states whose largest value is infinite or no number: what they stand
for is not finite, and the blocks beside them are untouched.  Lists around the sizes
of tables."""
import pytest
import torch

import convolution_implicit_gemm_conv2d_amd as cm

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.mark.parametrize("bad", [float("inf"), float("nan"), 1e30])
def test_a_block_that_is_not_finite(bad):
    """1e30 is finite, its square is not."""
    g = torch.full((512,), 0.1, device=DEV)
    g[130], g[131] = bad, 0.0
    p = torch.ones(512, device=DEV)
    state = cm.adamw_state([p], 8)
    cm.adamw_step([p], [g], state, 1, 0.1)
    values = cm.adamw_moments(state)
    block = slice(128, 256)
    assert not torch.isfinite(values["v"][0][block]).any() and not torch.isfinite(state["v_scale"][0][1])
    assert torch.isfinite(values["m"][0][block]).all() == (bad == 1e30)
    if bad != 1e30:
        assert (state["m"][0][block] == 0).all() and not torch.isfinite(values["m"][0][block]).any()
    # codes of v: 0, or 1 for a positive value under an infinite scale
    want = torch.zeros(128, dtype=torch.uint8, device=DEV) if bad != bad else (g[block] != 0).to(torch.uint8)
    assert torch.equal(state["v"][0][block], want)
    for t in (values["m"][0], values["v"][0], p):
        assert torch.isfinite(t[:128]).all() and torch.isfinite(t[256:]).all()


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("n", [1, 13, 14, 15, 47, 48, 49, 97])
def test_lists_around_the_sizes_of_tables(n, bits):
    gen = torch.Generator().manual_seed(n)
    ps, gs = ([torch.randn(5 + 130 * (i % 3), generator=gen).to(DEV) for i in range(n)] for _ in range(2))
    one = [torch.cat([torch.nn.functional.pad(t, (0, -t.numel() % 128)) for t in ts]) for ts in (ps, gs)]
    state, flat = cm.adamw_state(ps, bits), cm.adamw_state(one[:1], bits)
    cm.adamw_step(ps, gs, state, 1, 1e-2)
    cm.adamw_step(one[:1], one[1:], flat, 1, 1e-2)
    at = 0
    for i, p in enumerate(ps):
        assert torch.equal(p, one[0][at:at + p.numel()]), i
        assert torch.equal(state["m"][i], flat["m"][0][at:at + p.numel()]), i
        at += -(-p.numel() // 128) * 128
