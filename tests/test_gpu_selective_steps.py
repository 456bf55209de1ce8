"""Several steps of the example's training: the weights that the next forward pass
reads are the parameters, each step's, rounded to their type."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import convolution_implicit_gemm_conv2d_amd as cm  # noqa: E402
import selective_block  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def sizes(t):
    return t.double().square().sum().item()


@pytest.mark.parametrize("bits", [8, 32])
def test_every_step_reaches_the_weights(bits):
    gen = torch.Generator().manual_seed(11)
    starts = torch.tensor([0, 20, 20, 57], dtype=torch.int32, device=DEV)
    block = selective_block.SelectiveBlock(40, 72)
    trainer = selective_block.Trainer(block, bits)
    for step in range(4):
        x, do = (torch.randn(57, 40, generator=gen).to(DEV, torch.bfloat16) for _ in range(2))
        _, _, kept = block.forward(x, starts)
        _, dw = block.backward(do, kept)
        before = [p.clone() for p in trainer.params]
        values = cm.adamw_moments(trainer.state) if bits == 8 else trainer.state
        m, v = ([t.clone() for t in values[k]] for k in ("m", "v"))
        rate = 1e-2
        norm = trainer.step(dw, rate)
        c = min(1.0, 1.0 / (norm.item() + 1e-6))
        assert abs(norm.item() ** 2 / sum(sizes(dw[k]) for k in trainer.names) - 1) < 1e-5
        for k, p, b, mk, vk in zip(trainer.names, trainer.params, before, m, v):
            g = dw[k].double().view(-1) * c
            mk, vk = 0.9 * mk.double().view(-1) + 0.1 * g, 0.999 * vk.double().view(-1) + 0.001 * g * g
            mean, var = mk / (1 - 0.9 ** (step + 1)), vk / (1 - 0.999 ** (step + 1))
            want = b.double().view(-1) * (1 - rate * 0.01) - rate * mean / (var.sqrt() + 1e-8)
            # 24 roundings, as in the steps' own test, of the step with the magnitudes of
            # m's two terms (they may cancel) and of the parameter
            off = (p.double().view(-1) - want).abs()
            scale = rate * ((mk - 0.1 * g).abs() + 0.1 * g.abs()) / (1 - 0.9 ** (step + 1)) / (var.sqrt() + 1e-8)
            assert (off <= 24 * 2.0 ** -24 * (scale + b.double().view(-1).abs()) + 1e-30).all(), (k, step, off.max())
            # what the block computes with next
            assert torch.equal(block.w[k], p.to(block.w[k].dtype)), (k, step)
            assert not torch.equal(p, b), (k, step)
