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


def refusal(call):
    with pytest.raises(ValueError) as e:
        call()
    return str(e.value)


def test_refused_lists_are_named():
    p = [torch.zeros(5)]
    assert refusal(lambda: cm.adamw_step([], [], {"m": [], "v": []}, 1, 0.1)) == "the list of parameters is empty"
    assert refusal(lambda: cm.adamw_step([None], p, cm.adamw_state(p), 1, 0.1)) == "an entry of the parameters must be a tensor"
    assert refusal(lambda: cm.adamw_moments({k: [] for k in ("m", "v", "m_scale", "v_scale")})) == "the list of states is empty"
    assert refusal(lambda: cm.gradient_norm([])) == "the list of gradients is empty"
    assert refusal(lambda: cm.clip_gradients(p, 1.0, out=None)).startswith("tensors passed")
    assert refusal(lambda: cm.gradient_norm([3])) == "an entry of the gradients must be a tensor"
