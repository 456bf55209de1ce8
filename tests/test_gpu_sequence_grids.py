"""Batches of more lanes than one dimension of a grid holds (2^32): the last
sequences and rows against the same ones in a small batch."""
import pytest
import torch

import convolution_implicit_gemm_conv2d_amd as cm

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF16 = torch.bfloat16
END = 1000


@pytest.fixture(autouse=True)
def memory():
    yield
    torch.cuda.empty_cache()


def rand(*shape, seed, dtype=BF16):
    return torch.empty(shape, device=DEV, dtype=dtype).normal_(generator=torch.Generator(device=DEV).manual_seed(seed))


def ends(small, *pairs):
    for big, t in pairs:
        assert torch.equal(big[-END:], t[-END:]) and torch.equal(big[:END], t[:END]), small


def cut(t):
    return torch.cat([t[:END], t[-END:]])


def test_short_convolution():
    S = (1 << 32) // 3 + 50_000  # sequences of a row of three channels: a lane for each channel's state alone
    if torch.cuda.mem_get_info()[0] < 70 << 30:
        pytest.skip("needs 55 GB of device memory")
    x, initial, w = rand(S, 1, 3, seed=1), rand(S, 1, 3, seed=2), rand(3, 2, seed=3)
    last = torch.empty_like(x)
    y = cm.causal_conv(x, w, initial=initial, last=last)
    sx, si, sl = cut(x), cut(initial), torch.empty(2 * END, 1, 3, device=DEV, dtype=BF16)
    sy = cm.causal_conv(sx, w, initial=si, last=sl)
    ends("forward", (y, sy), (last, sl))
    assert torch.equal(cut(last), sx)
    del y
    g = cm.causal_conv_grad(last, x, w, initial=initial)
    sg = cm.causal_conv_grad(cut(last), sx, w, initial=si)
    ends("gradient", (g["x"], sg["x"]), (g["initial"], sg["initial"]))
    assert torch.isfinite(g["weight"].float()).all()


def test_tokens():
    rows = (1 << 24) + 2 * END  # a workgroup of 256 lanes each
    x, w, state = rand(rows, 1, seed=1), rand(1, 3, seed=2), rand(rows + 7, 2, 1, seed=3)
    small = cut(state[:rows])
    y = cm.causal_conv_step(x, w, state, activation="silu")
    ends("convolution", (y, cm.causal_conv_step(cut(x), w, small, activation="silu")), (state[:rows], small))
    delta, A, b, h = rand(rows, 1, seed=4), -torch.ones(1, 1, device=DEV), rand(rows, 1, seed=5), rand(rows, 1, 1, seed=6, dtype=torch.float32)
    small = cut(h)
    y = cm.selective_step(x, delta, A, b, b, h)
    ends("scan", (y, cm.selective_step(cut(x), cut(delta), A, cut(b), cut(b), small)), (h, small))


def test_more_packed_sequences_than_half_of_all():
    S = (1 << 30) + 100_000  # sequences of a row each: their number doubled passes 2^31
    x, w, b = rand(S, 1, seed=1), torch.tensor([[3.0, 0.5]], device=DEV, dtype=BF16), torch.ones(1, device=DEV, dtype=BF16)
    starts = torch.arange(S + 1, dtype=torch.int32, device=DEV)
    last = torch.empty(S, 1, 1, device=DEV, dtype=BF16)
    y = cm.causal_conv(x, w, b, starts=starts, last=last)
    for cut in (slice(0, END), slice(S // 2, S // 2 + END), slice(S - END, S)):
        assert torch.equal(y[cut], (x[cut].float() * 0.5 + 1).to(BF16)) and torch.equal(last[cut, 0], x[cut])
