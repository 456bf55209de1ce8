"""Tensors, pools and lists past 2^31 elements: what lies behind there against the
same rows in small tensors."""
import pytest
import torch

import convolution_implicit_gemm_conv2d_amd as cm

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF16 = torch.bfloat16


@pytest.fixture(autouse=True)
def memory():
    yield
    torch.cuda.empty_cache()


def rand(*shape, seed, dtype=BF16, std=1.0):
    return torch.empty(shape, device=DEV, dtype=dtype).normal_(0, std, generator=torch.Generator(device=DEV).manual_seed(seed))


ROWS, C = 530_000, 4096  # 2.17e9 elements
LAST = 100               # rows of the last sequence


def near(a, b):
    # both are rounded once from sums in other orders: one step of bf16 apart at most
    return torch.allclose(a.float(), b.float(), rtol=2 ** -7, atol=2 ** -10)


def test_convolution():
    x, dy, w = rand(ROWS, C, seed=1), rand(ROWS, C, seed=2), rand(C, 4, seed=3)
    starts = torch.tensor([0, 1000, ROWS - LAST, ROWS], dtype=torch.int32, device=DEV)
    y = cm.causal_conv(x, w, activation="silu", starts=starts)
    g = cm.causal_conv_grad(dy, x, w, activation="silu", starts=starts)
    end = x[ROWS - LAST:]
    assert torch.equal(y[ROWS - LAST:], cm.causal_conv(end, w, activation="silu"))
    assert torch.equal(g["x"][ROWS - LAST:], cm.causal_conv_grad(dy[ROWS - LAST:], end, w, activation="silu")["x"])
    assert torch.equal(y[:1000], cm.causal_conv(x[:1000], w, activation="silu"))


def test_scan():
    N = 2
    x, dy, delta = rand(ROWS, C, seed=1), rand(ROWS, C, seed=2), rand(ROWS, C, seed=3, std=0.1)
    A, B, Cm = -torch.rand(C, N, device=DEV) - 0.5, rand(ROWS, N, seed=4), rand(ROWS, N, seed=5)
    starts = torch.tensor([0, 1000, ROWS - LAST, ROWS], dtype=torch.int32, device=DEV)
    y = cm.selective_scan(x, delta, A, B, Cm, starts=starts)
    cut = [t if t is A else t[ROWS - LAST:] for t in (x, delta, A, B, Cm)]
    assert near(y[ROWS - LAST:], cm.selective_scan(*cut))
    del y
    saved = cm.selective_scan_saved(x, A)
    cm.selective_scan(x, delta, A, B, Cm, starts=starts, saved=saved, out=torch.empty_like(x))
    g = cm.selective_scan_grad(dy, x, delta, A, B, Cm, starts=starts, saved=saved)
    want = cm.selective_scan_grad(dy[ROWS - LAST:], *cut)
    for k in ("x", "delta", "B", "C"):
        assert near(g[k][ROWS - LAST:], want[k]), k


def test_pools_of_states():
    count, D, N = 17_000, 8192, 16  # 2.2e9 fp32 states
    state = torch.zeros(count, D, N, device=DEV)
    slots = torch.tensor([count - 1, 0, count - 2], dtype=torch.int32, device=DEV)
    ins = [rand(3, D, seed=1), rand(3, D, seed=2), -torch.rand(D, N, device=DEV), rand(3, N, seed=3), rand(3, N, seed=4)]
    small = torch.zeros(3, D, N, device=DEV)
    for _ in range(2):
        y, want = cm.selective_step(*ins, state, slots=slots), cm.selective_step(*ins, small)
        assert torch.equal(y, want)
    assert torch.equal(state[slots.long()], small) and not state[1:count - 2].any()
    del state
    count = 90_000  # 2.2e9 values of bf16
    state = torch.zeros(count, 3, D, device=DEV, dtype=BF16)
    slots = torch.tensor([count - 1, 0, count - 2], dtype=torch.int32, device=DEV)
    w, small = rand(D, 4, seed=5), torch.zeros(3, 3, D, device=DEV, dtype=BF16)
    for _ in range(2):
        assert torch.equal(cm.causal_conv_step(ins[0], w, state, slots=slots), cm.causal_conv_step(ins[0], w, small))
    assert torch.equal(state[slots.long()], small)


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw(bits):
    n, tail = (1 << 31) + 128 * 7 + 5, 128 * 9 + 5
    p = torch.zeros(n, device=DEV, dtype=BF16)
    g = torch.zeros(n, device=DEV, dtype=BF16)
    p[-tail:], g[-tail:] = rand(tail, seed=1), rand(tail, seed=2)
    q, h = p[-tail:].clone(), g[-tail:].clone()
    big, small = cm.adamw_state([p], bits), cm.adamw_state([q], bits)
    for step in (1, 2):
        cm.adamw_step([p], [g], big, step, 1e-2)
        cm.adamw_step([q], [h], small, step, 1e-2)
    assert torch.equal(p[-tail:], q) and not p[:1000].any()
    for k in ("m", "v"):
        assert torch.equal(big[k][0][-tail:], small[k][0])
    if bits == 8:
        assert torch.equal(big["m_scale"][0][-10:], small["m_scale"][0])
