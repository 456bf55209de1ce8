"""One tensor with more chunks than a grid holds: its tail, cut into a launch of
its own, against the same elements as a small tensor."""
import pytest
import torch

import convolution_implicit_gemm_conv2d_amd as cm

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF16 = torch.bfloat16


def test_a_tensor_of_more_than_a_grid():
    n, tail = (1 << 34) + 128 * 9 + 5, 4096 + 128 * 9 + 5  # the cut lies 1024 elements before 2^34
    if torch.cuda.mem_get_info()[0] < 130 << 30:
        pytest.skip("needs 105 GB of device memory")
    try:
        p, g = (torch.zeros(n, device=DEV, dtype=BF16) for _ in range(2))
        for i, t in enumerate((p, g)):
            t[-tail:] = torch.randn(tail, generator=torch.Generator().manual_seed(i)).to(DEV, BF16)
            t[:300] = torch.randn(300, generator=torch.Generator().manual_seed(i + 7)).to(DEV, BF16)
        ends = [slice(n - tail, n), slice(0, 384)]
        small = [[t[e].clone() for e in ends] for t in (p, g)]
        state, plain = cm.adamw_state([p], 8), cm.adamw_state(small[0], 8)
        for step in (1, 2):
            cm.adamw_step([p], [g], state, step, 1e-2)
            cm.adamw_step(*small, plain, step, 1e-2)
        torch.cuda.synchronize()
        for i, e in enumerate(ends):
            assert torch.equal(p[e], small[0][i])
            for k in ("m", "v"):
                assert torch.equal(state[k][0][e], plain[k][i])
            per = slice(e.start // 128, -(-e.stop // 128))
            for k in ("m_scale", "v_scale"):
                assert torch.equal(state[k][0][per], plain[k][i])
        assert not p[384:4000].any() and not p[-tail - 5000:-tail].any()
    finally:
        p = g = t = state = None
        torch.cuda.empty_cache()
