"""The lanes' layouts that a scan takes for larger batches, at short lengths, against
the 64-bit forms with running bounds; and both forms of gelu as activation and gate."""
import pytest
import torch

import sequence_reference as sr
import test_gpu_causal as causal
import test_gpu_scan as scan

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


# Whole sequences with at least a wave for each SIMD (4096 channels: two sequences of 512
# waves in eight groups of lanes) and less than two (seven of 256 in four), for 5 to 16
# states: one and two of a lane in eight groups.  From eight sequences on, four groups.
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("S,L,N", [(2, 20, 16), (3, 17, 11), (2, 33, 8), (2, 7, 5), (7, 5, 16), (8, 18, 16), (8, 5, 12), (9, 17, 7)])
def test_large_batches(dtype, S, L, N):
    i = scan.Inputs(S * L, 4096, N, 1, dtype, S)
    scan.check(i, sr.spans_of(S * L, S), (S, L, 4096), None)


# Nine to twelve states are three of a lane in four groups: rows of B and C that do not
# divide a wave.
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("N", [9, 10, 11, 12])
@pytest.mark.parametrize("C,G,extra", [(70, 2, 0), (9, 1, 3)])
def test_three_states_of_a_lane(dtype, N, C, G, extra):
    for lengths, front, behind in (([5, 0, 1, 40, 2], 1, 3), ([63, 130, 1, 0, 66, 3], 0, 0)):
        starts = scan.starts_of(lengths, front)
        rows = starts[-1] + behind
        i = scan.Inputs(rows, C, N, G, dtype, len(lengths))
        scan.check(i, sr.spans_of(rows, starts=starts), (rows, C), starts, extra=extra)
    i = scan.Inputs(2 * 37, C, N, G, dtype, 2)
    scan.check(i, sr.spans_of(74, 2), (2, 37, C), None, full=False, keep=False)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("kind", ["gelu", "gelu_tanh"])
def test_gelu(kind, dtype):
    causal.test_forward_and_gradient(dtype, (2, 40), 37, 4, kind, 5)
    causal.test_forward_and_gradient(dtype, ([5, 0, 1, 40, 2], 0, 3), 3, 3, kind, 0)
    i = scan.Inputs(60, 20, 16, 1, dtype, 2)
    i.z = i.z * 4
    scan.check(i, sr.spans_of(60, 2), (2, 30, 20), None, kind=kind)
