"""Lists that the optimizer step's Python level takes (CPU): iterators of
parameters, and what it says of lists that it refuses."""
import pytest
import torch

import convolution_implicit_gemm_conv2d_amd as cm


@pytest.mark.parametrize("bits", [32, 8])
def test_states_of_an_iterator_of_parameters(bits):
    layer = torch.nn.Linear(130, 3)
    state = cm.adamw_state(layer.parameters(), bits)
    want = cm.adamw_state(list(layer.parameters()), bits)
    assert {k: [t.shape for t in v] for k, v in state.items()} == {k: [t.shape for t in v] for k, v in want.items()}
    assert all(len(v) == 2 for v in state.values())
