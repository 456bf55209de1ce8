"""Batches of many short sequences: a workgroup takes several of them, and the
gradient takes several launches.  Against the same sequences in smaller batches."""
import pytest
import torch

import convolution_implicit_gemm_conv2d_amd as cm

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def memory():
    yield
    torch.cuda.empty_cache()


def rand(*shape, seed, dtype=F32, std=1.0):
    return torch.empty(shape, device=DEV, dtype=dtype).normal_(0, std, generator=torch.Generator(device=DEV).manual_seed(seed))


class Batch:
    def __init__(self, S, L, C, N, dtype, groups=1):
        r = lambda *s, seed, t=dtype, std=1.0: rand(*s, seed=seed, dtype=t, std=std)  # noqa: E731
        self.x, self.z, self.dy, self.delta = (r(S, L, C, seed=i, std=0.5 if i == 4 else 1.0) for i in (1, 2, 3, 4))
        self.B, self.Cm = r(S, L, groups, N, seed=5), r(S, L, groups, N, seed=6)
        self.initial, self.dlast = r(S, C, N, seed=7, t=F32), r(S, C, N, seed=8, t=F32)
        self.A, self.D, self.bias = -torch.rand(C, N, device=DEV) - 0.1, r(C, seed=9, t=F32), r(C, seed=10, t=F32)

    def run(self, cut=slice(None), keep=True):
        ins = [t[cut] for t in (self.x, self.delta)] + [self.A] + [t[cut] for t in (self.B, self.Cm)]
        how = dict(D=self.D, z=self.z[cut], delta_bias=self.bias, initial=self.initial[cut])
        last = torch.full_like(self.initial[cut], float("nan"))
        saved = cm.selective_scan_saved(ins[0], self.A) if keep else None
        y = cm.selective_scan(*ins, last=last, saved=saved, **how)
        g = cm.selective_scan_grad(self.dy[cut], *ins, dlast=self.dlast[cut], saved=saved, **how)
        return {"y": y, "last": last, **g}


def check(batch, S, parts, keep=True):
    whole = batch.run(keep=keep)
    sums = {}
    for i in range(parts):
        cut = slice(S * i // parts, S * (i + 1) // parts)
        part = batch.run(cut, keep)
        for k, t in part.items():
            if k in ("A", "D", "delta_bias"):
                sums[k] = sums.get(k, 0) + t.double()
            else:
                assert torch.equal(whole[k][cut], t), (k, i)
        del part
    for k, t in sums.items():
        # n values of about one size, K of them one after another in a workgroup, the
        # n / K partial sums then: partial sums grow as the root of their values, so a
        # workgroup's roundings come to 2^-24 K values, all to root(n K) 2^-24, and the
        # sum itself to root(n): root(K) 2^-24 of the largest, 3e-6 for K = 2000
        assert torch.allclose(whole[k].double(), t, rtol=1e-4, atol=1e-4 * t.abs().max().item()), k


@pytest.mark.parametrize("keep", [True, False])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("S,L,C,N,G", [(40_001, 3, 20, 4, 1), (20_000, 1, 33, 16, 3), (17_000, 18, 8, 24, 1)])
def test_a_workgroup_takes_several_sequences(S, L, C, N, G, dtype, keep):
    check(Batch(S, L, C, N, dtype, G), S, 3, keep)


def test_launches_of_the_gradient():
    # the partials of dB and dC: 64 workgroups of 32 channels, 128 bytes for each row
    S, L, C, N = 12_000, 24, 2048, 16
    assert cm.conv_scan_bwd_workspace_size(S * L, S, C, N, 1, False, True) < C // 32 * S * L * 2 * N * 4
    b = Batch(S, L, C, N, BF16)
    for keep in (True, False):
        check(b, S, 5, keep)


def test_more_sequences_than_a_grid_holds():
    S = (1 << 24) + 3000  # a workgroup each
    b = Batch(S, 1, 1, 1, F32)
    whole = b.run()
    for cut in (slice(0, 1000), slice(S - 1000, S)):
        part = b.run(cut)
        for k, t in part.items():
            if k not in ("A", "D", "delta_bias"):
                assert torch.equal(whole[k][cut], t), k


def test_more_rows_of_states_than_a_grid_holds():
    rows, N = (1 << 25) + (1 << 20), 64  # 2 N sums of dB and dC a row
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 45 GB of device memory")
    x, dy, delta = (rand(rows, 1, seed=i, dtype=BF16) for i in (1, 2, 3))
    B, Cm, A = rand(rows, N, seed=4, dtype=BF16), rand(rows, N, seed=5, dtype=BF16), -torch.rand(1, N, device=DEV) - 1
    g = cm.selective_scan_grad(dy, x, delta, A, B, Cm)
    # 4000 rows fade what was before them: softplus steps of 0.7 at a time
    end = [t if t is A else t[-5000:] for t in (dy, x, delta, A, B, Cm)]
    want = cm.selective_scan_grad(*end)
    for k in ("x", "delta", "B", "C"):
        # both rounded once to bf16
        assert torch.allclose(g[k][-1000:].float(), want[k][-1000:].float(), rtol=2 ** -7, atol=2 ** -12), k
    start = [t if t is A else t[:5000] for t in (dy, x, delta, A, B, Cm)]
    want = cm.selective_scan_grad(*start)
    for k in ("x", "delta", "B", "C"):
        assert torch.allclose(g[k][:1000].float(), want[k][:1000].float(), rtol=2 ** -7, atol=2 ** -12), k
