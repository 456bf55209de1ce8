"""The gated layer's largest tiles: long sums with enough output tiles to fill
the device, ragged in every direction, on whole numbers (every result exact
before its one rounding)."""
import pytest
import torch

from test_gpu_gated import BF16, exact_case

pytestmark = pytest.mark.gpu

# rows, channels, hidden: a long sum in the forward product, in dx, in dW
SIZES = [(4097, 1032, 2056), (4097, 4104, 520), (1100, 4104, 2056), (4352, 1024, 2048)]


@pytest.mark.parametrize("keep", [False, True])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_whole_numbers(size, keep):
    print(size, keep, flush=True)
    exact_case(*size, BF16, keep, "relu")
    torch.cuda.empty_cache()
