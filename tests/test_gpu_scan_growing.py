"""States that grow along a sequence (A above 0, or steps below 0): rows that are
cut into pieces hand a state on by one power of all rows between, which leaves
fp32's range where the state itself does not."""
import pytest
import torch

import convolution_implicit_gemm_conv2d_amd as cm
import sequence_reference as sr
from running_bounds import B, within

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def rand(*shape, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed))


def check(rows, spans, x, delta, A, dy, plus, starts=None, extra=0.0, **states):
    """``extra``: units of 2^-24 that every value may be off beside its running bound."""
    N = A.shape[1]
    b, c = rand(rows, 1, N, seed=4), rand(rows, 1, N, seed=5)
    ref = sr.scan(x, delta, A, b, c, None, None, None, plus, "none", spans, states.get("initial"), dy, states.get("dlast"))
    lead = lambda t: t.to(DEV) if starts is not None else t.to(DEV).view(len(spans), -1, *t.shape[1:])  # noqa: E731
    ins = [lead(x), lead(delta), A.to(DEV), lead(b), lead(c)]
    how = dict(softplus=plus, starts=None if starts is None else torch.tensor(starts, dtype=torch.int32, device=DEV),
               initial=states["initial"].to(DEV) if "initial" in states else None)
    for keep in (True, False):
        saved = cm.selective_scan_saved(ins[0], ins[2]) if keep else None
        last = torch.empty(len(spans), x.shape[1], N, device=DEV)
        y = cm.selective_scan(*ins, last=last, saved=saved, **how)
        g = cm.selective_scan_grad(lead(dy), *ins, saved=saved, dlast=states["dlast"].to(DEV) if "dlast" in states else None, **how)
        torch.cuda.synchronize()
        for name, got, want in [("y", y, ref["y"]), ("last", last, ref["last"])] + [(k, v, ref[k]) for k, v in g.items() if v is not None]:
            want = B(want.v, want.e + extra * want.v.abs())
            within(name, got.reshape(want.v.shape), want)


# pieces of 32 rows from 128 rows on; 100 rows are one share
@pytest.mark.parametrize("rows,seqs", [(1024, 1), (1300, 2), (100, 1)])
@pytest.mark.parametrize("plus", [True, False])
def test_zeros_stay_zeros(rows, seqs, plus):
    """A factor of e^4 a row over states of zero, and over gradients of zero: the
    input is in the last rows of a sequence, its gradient in the first ones."""
    C, N, L = 64, 4, rows // seqs
    x, dy = rand(rows, C, seed=1), rand(rows, C, seed=2)
    at = torch.arange(rows) % L
    x[at < L - 8], dy[at >= 8] = 0, 0
    delta = rand(rows, C, seed=3) * 0.1 + 1.0 if plus else -(rand(rows, C, seed=3) * 0.1 + 1.3)
    A = (torch.rand(C, N, generator=torch.Generator().manual_seed(6)) + 2) * (1 if plus else -1)
    zeros = torch.zeros(seqs, C, N)
    check(rows, sr.spans_of(rows, seqs), x, delta, A, dy, plus)
    check(rows, sr.spans_of(rows, seqs), x, delta, A, dy, plus, initial=zeros, dlast=zeros)
    if rows > 100:
        starts = [0, 0, 5, rows]
        x[:5], dy[5:8] = 0, 0
        dy[5:13] = rand(8, C, seed=7)
        x[:rows - 8] = 0
        dy[13:] = 0
        check(rows, sr.spans_of(rows, starts=starts), x, delta, A, dy, plus, starts=starts)


def test_tiny_states_grow_and_large_ones_fade():
    """e^-70 grows to e^70 over 700 rows, and e^80 fades to e^-60: the state is an
    fp32 value all the way, the power between its ends is not."""
    rows, C, N = 700, 8, 2
    d = torch.rand(rows, C, generator=torch.Generator().manual_seed(3)) * 0.02 + 0.19
    # The steps' sums: 32 roundings in a piece of at most its sum, one for each of 22
    # pieces of at most all, three for the products: (32 + 22 + 3) units of the 140.
    extra = 57 * 140.0
    x, dy = torch.zeros(rows, C), torch.zeros(rows, C)
    x[0], dy[-1] = 1e-30 * rand(C, seed=1), 1e-30 * rand(C, seed=2)
    check(rows, [(0, rows)], x, d, torch.ones(C, N), dy, False, extra=extra)
    first = torch.exp(torch.tensor(80.0)) * rand(1, C, N, seed=8)
    x[0], dy[-1] = 0, 1e30
    check(rows, [(0, rows)], x, d, -torch.ones(C, N), dy, False, extra=extra, initial=first)
