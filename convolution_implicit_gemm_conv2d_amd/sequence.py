"""Operators along a sequence: the short causal convolution and the selective
state space scan, for prompts, for training and for single tokens.

Argument marshalling only, like the rest of the binding: ``conv_*`` functions
carry the C names and arguments, the others derive sizes from tensor shapes,
allocate outputs and workspaces, and check what the C side cannot see.

Rows and sequences.  ``x`` is a batch of prompts of one length [S, L, C], or one
prompt [L, C]; with ``starts`` (int32 on the device, S + 1 values) it is [T, C]
and sequence s has the rows from ``starts[s]`` up to ``starts[s + 1]``.  Sequences
may be empty; rows in front of the first and behind the last one belong to none:
an output given by the caller keeps them, one that the call allocates holds zeros
there.  The values of ``starts`` have to ascend; they are not read on the host.

Rows may lie apart: ``x``, ``delta``, ``z``, ``B`` and ``C`` may be parts of a wider
projection, as long as a row's own values are dense and rows evenly spaced.  All
other tensors are contiguous.  Outputs must not overlap inputs.

Streams, errors and automatic differentiation as in ``block``: a call works on the
current stream of its tensors' device or on ``stream``, results carry no graph, and
what a call writes in a caller's tensor counts a new version.
"""
from __future__ import annotations

from . import _check, _lib, _ptr, _stream
from .block import ACTIVATIONS, _choice, _current, _entered, _native, _result, _size

__all__ = [
    "conv_causal_fwd", "conv_causal_bwd", "conv_causal_bwd_workspace_size", "conv_causal_step", "conv_scan_fwd",
    "conv_scan_bwd", "conv_scan_saved_size", "conv_scan_fwd_workspace_size", "conv_scan_bwd_workspace_size",
    "conv_scan_step", "causal_conv", "causal_conv_grad", "causal_conv_step", "selective_scan",
    "selective_scan_saved", "selective_scan_grad", "selective_step",
]


def _raw(t):
    """A device address: of a tensor whose rows may lie apart, too."""
    if t is None or isinstance(t, int):
        return t
    if not t.is_cuda:
        raise ValueError("tensors passed to convmi must be on a GPU device")
    return t.data_ptr()


def conv_causal_bwd_workspace_size(rows, C, K, dtype) -> int:
    return _size("conv_causal_bwd_workspace_size", 0, rows, C, K, dtype)


def conv_scan_saved_size(rows, channels, N) -> int:
    return _size("conv_scan_saved_size", 0, rows, channels, N)


def conv_scan_fwd_workspace_size(rows, seqs, channels, N, groups, packed) -> int:
    return _size("conv_scan_fwd_workspace_size", 0, rows, seqs, channels, N, groups, int(packed))


def conv_scan_bwd_workspace_size(rows, seqs, channels, N, groups, packed, saved) -> int:
    return _size("conv_scan_bwd_workspace_size", 0, rows, seqs, channels, N, groups, int(packed), int(saved))


def conv_causal_fwd(x, w, bias, starts, initial, y, last, rows, seqs, C, K, x_stride, act, clear, dtype, stream=None) -> None:
    p = _ptr
    _check(_lib.load().conv_causal_fwd(_raw(x), p(w), p(bias), p(starts), p(initial), p(y), p(last), rows, seqs, C, K, x_stride,
                                      act, clear, dtype, _stream(stream)))


def conv_causal_bwd(dy, dlast, x, w, bias, starts, initial, dx, dw, dbias, dinitial, workspace, workspace_bytes, rows, seqs, C,
                    K, x_stride, act, clear, dtype, stream=None) -> None:
    p = _ptr
    _check(_lib.load().conv_causal_bwd(p(dy), p(dlast), _raw(x), p(w), p(bias), p(starts), p(initial), p(dx), p(dw), p(dbias),
                                      p(dinitial), p(workspace), workspace_bytes, rows, seqs, C, K, x_stride, act, clear,
                                      dtype, _stream(stream)))


def conv_causal_step(x, w, bias, state, slots, y, rows, count, C, K, x_stride, act, clear, dtype, stream=None) -> None:
    p = _ptr
    _check(_lib.load().conv_causal_step(_raw(x), p(w), p(bias), p(state), p(slots), p(y), rows, count, C, K, x_stride, act,
                                       clear, dtype, _stream(stream)))


def conv_scan_fwd(x, delta, A, B, C, D, z, delta_bias, starts, initial, y, last, saved, workspace, workspace_bytes, rows, seqs,
                  channels, N, groups, x_stride, delta_stride, z_stride, B_stride, C_stride, softplus, act, clear, dtype,
                  stream=None) -> None:
    p, r = _ptr, _raw
    _check(_lib.load().conv_scan_fwd(r(x), r(delta), p(A), r(B), r(C), p(D), r(z), p(delta_bias), p(starts), p(initial), p(y),
                                    p(last), p(saved), p(workspace), workspace_bytes, rows, seqs, channels, N, groups,
                                    x_stride, delta_stride, z_stride, B_stride, C_stride, softplus, act, clear, dtype,
                                    _stream(stream)))


def conv_scan_bwd(dy, dlast, x, delta, A, B, C, D, z, delta_bias, starts, initial, saved, dx, ddelta, dA, dB, dC, dD, dz,
                  ddelta_bias, dinitial, workspace, workspace_bytes, rows, seqs, channels, N, groups, x_stride, delta_stride,
                  z_stride, B_stride, C_stride, softplus, act, clear, dtype, stream=None) -> None:
    p, r = _ptr, _raw
    _check(_lib.load().conv_scan_bwd(p(dy), p(dlast), r(x), r(delta), p(A), r(B), r(C), p(D), r(z), p(delta_bias), p(starts),
                                    p(initial), p(saved), p(dx), p(ddelta), p(dA), p(dB), p(dC), p(dD), p(dz),
                                    p(ddelta_bias), p(dinitial), p(workspace), workspace_bytes, rows, seqs, channels, N,
                                    groups, x_stride, delta_stride, z_stride, B_stride, C_stride, softplus, act, clear,
                                    dtype, _stream(stream)))


def conv_scan_step(x, delta, A, B, C, D, z, delta_bias, state, slots, y, rows, count, channels, N, groups, x_stride,
                   delta_stride, z_stride, B_stride, C_stride, softplus, act, clear, dtype, stream=None) -> None:
    p, r = _ptr, _raw
    _check(_lib.load().conv_scan_step(r(x), r(delta), p(A), r(B), r(C), p(D), r(z), p(delta_bias), p(state), p(slots), p(y),
                                     rows, count, channels, N, groups, x_stride, delta_stride, z_stride, B_stride, C_stride,
                                     softplus, act, clear, dtype, _stream(stream)))


# ----------------------------------------------------------- tensor level --

def causal_conv(x, weight, bias=None, activation="none", starts=None, initial=None, last=None, out=None, stream=None):
    """``y[t] = act(bias + sum_k weight[k] x[t - K + 1 + k])`` for every channel,
    along each sequence.

    ``weight`` [C, K] with 2 to 8 taps (a depthwise conv1d weight, [C, K, 1] or
    [C, 1, K], too).  ``initial`` [S, K - 1, C] holds the rows before each sequence
    (zeros without it), ``last`` of the same shape receives the last K - 1 rows
    with those before them: what the next part of the sequence, or
    ``causal_conv_step``, goes on from."""
    s = _current(x, stream)
    if s is None:
        return _entered(causal_conv, x, stream, x, weight, bias, activation, starts, initial, last, out)
    act = _choice(ACTIVATIONS, activation, "activation")
    return _result(_native().causal(x, weight, bias, act, starts, initial, last, out, s))


def causal_conv_grad(dy, x, weight, bias=None, activation="none", starts=None, initial=None, dlast=None, workspace=None,
                     stream=None):
    """Gradient of ``causal_conv`` from ``dy`` (and ``dlast``, the gradient of
    ``last``): a dict with "x", "weight", "bias" and "initial", ``None`` for what the
    call does not have."""
    s = _current(x, stream)
    if s is None:
        return _entered(causal_conv_grad, x, stream, dy, x, weight, bias, activation, starts, initial, dlast, workspace)
    act = _choice(ACTIVATIONS, activation, "activation")
    return dict(zip(("x", "weight", "bias", "initial"),
                    _result(_native().causal_grad(dy, x, weight, bias, act, starts, initial, dlast, workspace, s))))


def causal_conv_step(x, weight, state, bias=None, activation="none", slots=None, out=None, stream=None):
    """``causal_conv`` of one row for each of many sequences.

    ``x`` [rows, C]; ``state`` [M, K - 1, C] holds the last rows of M sequences and
    moves on in place.  ``slots`` (int32 [rows] on the device) says which of them a
    row belongs to; without it row r has ``state[r]``.  A slot outside the pool marks
    a row of padding: ``out`` keeps it, an allocated output holds zeros there.  Rows
    of the same slot are taken in their order."""
    s = _current(x, stream)
    if s is None:
        return _entered(causal_conv_step, x, stream, x, weight, state, bias, activation, slots, out)
    act = _choice(ACTIVATIONS, activation, "activation")
    return _result(_native().causal_step(x, weight, state, bias, act, slots, out, s))


def selective_scan_saved(x, A):
    """A buffer for ``saved`` of ``selective_scan`` and ``selective_scan_grad``: states
    every 16 rows, float32."""
    import torch

    n = conv_scan_saved_size(x.numel() // max(x.shape[-1], 1), x.shape[-1], A.shape[-1]) // 4
    return torch.empty(n, dtype=torch.float32, device=x.device)


def selective_scan(x, delta, A, B, C, D=None, z=None, delta_bias=None, softplus=True, gate_activation="silu", starts=None,
                   initial=None, last=None, saved=None, out=None, stream=None):
    """The selective state space scan, along each sequence and for every channel:

        d = softplus(delta + delta_bias)      (without softplus: delta + delta_bias)
        h = exp(d A) h + d B x                N states
        y = (C . h + D x) act(z)              without z: no gate

    ``delta`` and ``z`` have the shape of ``x``; ``B`` and ``C`` [..., N], or [..., G, N]
    for G groups of neighbouring channels; ``A`` [C, N] with 1 to 64 states, ``D`` and
    ``delta_bias`` [C] in float32.  ``initial`` and ``last`` (float32 [S, C, N]) are the
    states before and behind the sequences.  ``saved`` (from ``selective_scan_saved``)
    receives what ``selective_scan_grad`` would otherwise compute again."""
    s = _current(x, stream)
    if s is None:
        return _entered(selective_scan, x, stream, x, delta, A, B, C, D, z, delta_bias, softplus, gate_activation, starts,
                        initial, last, saved, out)
    act = _choice(ACTIVATIONS, gate_activation, "gate_activation")
    return _result(_native().scan(x, delta, A, B, C, D, z, delta_bias, bool(softplus), act, starts, initial, last, saved, out, s))


_SCAN_INPUTS = ("x", "delta", "A", "B", "C", "D", "z", "delta_bias", "initial")


def selective_scan_grad(dy, x, delta, A, B, C, D=None, z=None, delta_bias=None, softplus=True, gate_activation="silu",
                        starts=None, initial=None, dlast=None, saved=None, workspace=None, stream=None):
    """Gradient of ``selective_scan`` from ``dy`` (and ``dlast``, the gradient of
    ``last``), with the forward call's inputs: a dict with "x", "delta", "A", "B", "C",
    "D", "z", "delta_bias" and "initial", ``None`` for what the call does not have."""
    s = _current(x, stream)
    if s is None:
        return _entered(selective_scan_grad, x, stream, dy, x, delta, A, B, C, D, z, delta_bias, softplus, gate_activation,
                        starts, initial, dlast, saved, workspace)
    act = _choice(ACTIVATIONS, gate_activation, "gate_activation")
    return dict(zip(_SCAN_INPUTS, _result(_native().scan_grad(
        x, delta, A, B, C, D, z, delta_bias, bool(softplus), act, starts, initial, dy, dlast, saved, workspace, s))))


def selective_step(x, delta, A, B, C, state, D=None, z=None, delta_bias=None, softplus=True, gate_activation="silu",
                   slots=None, out=None, stream=None):
    """``selective_scan`` of one row for each of many sequences: ``x`` [rows, C],
    ``state`` float32 [M, C, N] in place, ``slots`` as in ``causal_conv_step``."""
    s = _current(x, stream)
    if s is None:
        return _entered(selective_step, x, stream, x, delta, A, B, C, state, D, z, delta_bias, softplus, gate_activation, slots,
                        out)
    act = _choice(ACTIVATIONS, gate_activation, "gate_activation")
    return _result(_native().scan_step(x, delta, A, B, C, D, z, delta_bias, bool(softplus), act, state, slots, out, s))
