"""Events armed for a block operator's call: its first launch stamps the start and
its last one the stop, whatever outputs the caller asks for."""
import itertools

import pytest
import torch

import convolution_implicit_gemm_conv2d_amd as cm

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF16, F32 = torch.bfloat16, torch.float32


def stamped(call):
    """The call's time by its events, both recorded before it too: a start that is
    not stamped leaves a time that is too long, a stop one below zero."""
    start, stop = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    stop.record()
    torch.cuda._sleep(1000)
    start.record()
    torch.cuda._sleep(48_000_000)  # 20 ms
    torch.cuda.synchronize()
    cm.conv_arm_launch_events(start.cuda_event, stop.cuda_event)
    call()
    torch.cuda.synchronize()
    ms = start.elapsed_time(stop)
    assert 0 < ms < 8, ms


def t(*shape, dtype=BF16):
    return torch.zeros(shape, dtype=dtype, device=DEV)


@pytest.mark.parametrize("rows,C,F,dtype", [(0, 64, 48, BF16), (5, 64, 48, BF16), (5, 33, 48, BF16), (300, 64, 1024, BF16), (300, 64, 48, F32)])
def test_gated_gradient(rows, C, F, dtype):
    x, dh, w, b = t(rows, C, dtype=dtype), t(rows, F, dtype=dtype), t(F, C, dtype=dtype), t(F, dtype=dtype)
    code = cm.CONV_BF16 if dtype == BF16 else cm.CONV_F32
    need = cm.conv_gated_bwd_workspace_size(rows, C, F, code)
    ws = t(max(need, 16), dtype=torch.uint8)
    saved = t(rows, 2 * F, dtype=F32)
    for kept, dx, dwg, dwu, db in itertools.product((None, saved), (None, t(rows, C, dtype=dtype)), (None, t(F, C, dtype=dtype)),
                                                    (None, t(F, C, dtype=dtype)), (None, t(F, dtype=dtype))):
        if rows == 0 and dwg is None and dwu is None and db is None:
            continue  # nothing to launch
        print(rows, C, F, dtype, [v is not None for v in (kept, dx, dwg, dwu, db)], flush=True)
        stamped(lambda: cm.conv_gated_bwd(dh, x, w, w, b, b, kept, dx, dwg, dwu, db, db if db is None else torch.empty_like(db), ws, need, rows, C, F, 2, code))


@pytest.mark.parametrize("rows,C,dtype", [(0, 64, BF16), (12, 64, BF16), (12, 1001, F32), (12, 9000, BF16), (12, 5, F32)])
def test_norm_gradient(rows, C, dtype):
    x, f, dy, da, p = t(rows, C, dtype=dtype), t(rows, C, dtype=dtype), t(rows, C, dtype=dtype), t(rows, C, dtype=dtype), t(C, dtype=dtype)
    code = cm.CONV_BF16 if dtype == BF16 else cm.CONV_F32
    for gate_rows in (0, 1, 4, 12):
        z = t(max(rows // gate_rows, 1), C, dtype=dtype) if gate_rows else None
        ws = t(max(cm.conv_block_norm_bwd_workspace_size(rows, C, gate_rows), 16), dtype=torch.uint8)
        for dx, dz, dw, db in itertools.product((None, t(rows, C, dtype=dtype)), (None, z), (None, t(C, dtype=dtype)), (None, t(C, dtype=dtype))):
            if rows == 0 and dw is None and db is None:
                continue  # nothing to launch
            if dz is not None:
                dz = t(*z.shape, dtype=dtype)
            print(rows, C, dtype, gate_rows, [v is not None for v in (dx, dz, dw, db)], flush=True)
            stamped(lambda: cm.conv_block_norm_bwd(dy, da, x, f, z, None, p, p, p, None, dx, None, dz, None, dw, db, None, None, ws,
                                                   ws.numel(), rows, C, gate_rows or 1, 2, 2, 1, 1e-6, code))


@pytest.mark.parametrize("n", [1, 129])
def test_forward_and_lists(n):
    x, w = t(2100, 1031), t(520, 1031)  # copied to padded rows first
    stamped(lambda: cm.gated_feed_forward(x, w, w))
    stamped(lambda: cm.block_norm(x, x))
    g = [t(100) for _ in range(n)]
    stamped(lambda: cm.gradient_norm(g))
    stamped(lambda: cm.clip_gradients(g, 1.0))
