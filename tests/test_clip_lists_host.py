"""Lists that clipping refuses because their tensors overlap (CPU): every call here
fails its checks before it reaches a GPU."""
from array import array

import pytest

import convolution_implicit_gemm_conv2d_amd as cm
from convolution_implicit_gemm_conv2d_amd import _lib

FAKE = 0x1000  # never dereferenced


def clip_list(grads, outs, counts, dtypes):
    # a workspace one byte short, so that a list that is accepted goes no further
    n = len(grads)
    lib = _lib.load()
    g, o, c, d = array("Q", grads), array("Q", outs), array("Q", counts), array("i", dtypes)
    at = [v.buffer_info()[0] for v in (g, o, c, d)]
    rc = lib.conv_grad_clip(*at, n, 1.0, 0.0, FAKE, FAKE, cm.conv_grad_workspace_size(n) - 1, None)
    assert rc == cm.CONV_ERR_INVALID_ARG
    return cm.conv_last_error()


@pytest.mark.parametrize("n", [2, 3, 40, 700])
def test_clipping_refuses_tensors_that_overlap(n):
    # two workgroups would scale the same values: results change from run to run
    apart = [FAKE + 4096 * (i * 37 % n) for i in range(n)]
    assert len(set(apart)) == n
    counts, dtypes = [1024] * n, [0] * n
    copies = [v + (1 << 30) for v in apart]
    assert "workspace" in clip_list(apart, apart, counts, dtypes)
    assert "workspace" in clip_list(apart, copies, counts, dtypes)
    assert "workspace" in clip_list([apart[0]] * n, copies, counts, dtypes)  # read twice: fine
    for i, j in ((0, n - 1), (n - 1, 0)):
        twice = list(apart)
        twice[i] = apart[j]
        assert "overlap" in clip_list(twice, twice, counts, dtypes), "one tensor twice, in place"
        twice = list(copies)
        twice[i] = copies[j] + 4092  # one element of the other
        assert "overlap" in clip_list(apart, twice, counts, dtypes), "outputs overlap"
        twice = list(copies)
        twice[i] = apart[j]
        assert "overlap" in clip_list(apart, twice, counts, dtypes), "an output is another gradient"
        twice = list(copies)
        twice[i] = apart[i] + 4
        assert "overlap" in clip_list(apart, twice, counts, dtypes), "an output is its gradient, moved"
        empty = list(counts)
        empty[i] = 0
        twice = list(apart)
        twice[i] = apart[j]
        assert "workspace" in clip_list(twice, twice, empty, dtypes), "no elements, no overlap"
    half = [512 * 4 * i + FAKE for i in range(n)]  # bf16: 1024 elements are 2048 bytes
    assert "workspace" in clip_list(half, half, counts, [1] * n)
    assert "overlap" in clip_list(half, half, counts, dtypes)
