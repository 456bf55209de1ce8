"""The searches for a row's sequence (CPU): the middle of two numbers below 2^31 is
formed without passing it, or a batch of 2^30 packed sequences would read in front of
its offsets."""
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "convolution_implicit_gemm_conv2d_amd", "csrc")


def middles(text):
    """The expressions of ``mid`` in a source's searches from 0 to seqs."""
    found = []
    for body in re.findall(r"int lo = 0, hi = a\.seqs;.*?return lo;", text, re.S):
        found += re.findall(r"const int mid = (.*?);", body)
    return found


def int32(v):
    return (v + (1 << 31)) % (1 << 32) - (1 << 31)


class Int(int):
    """An int of 32 bits."""

    def __add__(self, o):
        return Int(int32(int(self) + int(o)))

    def __sub__(self, o):
        return Int(int32(int(self) - int(o)))

    def __rshift__(self, o):
        return Int(int(self) >> int(o))


@pytest.mark.parametrize("source", ["short_conv.hip", "scan.hpp"])
def test_the_middle_is_one(source):
    with open(os.path.join(CSRC, source)) as f:
        found = middles(f.read())
    assert len(found) == 1
    for expression in found:
        for lo, hi in ((0, 1), (0, 2**31 - 1), (2**30, 2**30 + 5), (2**31 - 2, 2**31 - 1), (3, 2**31 - 1)):
            got = eval(expression, {"lo": Int(lo), "hi": Int(hi)})  # noqa: S307  (a line of this repository)
            assert got == (lo + hi) // 2 and lo <= got < hi, (expression, lo, hi)
