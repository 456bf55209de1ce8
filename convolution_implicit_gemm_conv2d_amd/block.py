"""Operators around a convolution: the gated feed-forward layer, the norms
before and after a block, and the gradients' global norm.

Argument marshalling only, like the rest of the binding: ``conv_*`` functions
carry the C names and arguments, the others derive sizes from tensor shapes,
allocate outputs and workspaces, and check what the C side cannot see.
Everything is channels-last: the last dimension of an input is its channels,
the ones before it are its rows.

A call works on the current stream of its tensors' device, or on ``stream``.
With ``stream``, what the call allocates belongs to that stream; inputs made on
another one must be ready (the caller orders the streams).

Automatic differentiation records no call: results carry no graph, also where
inputs require gradients (the ``_grad`` functions are the gradients).  A caller's
tensor that a call writes (``out``, ``saved``, a list clipped in place) counts a
new version, so a graph that had saved it refuses to run backwards.

The checks of tensors, the allocations and the calls are native
(``csrc/binding.cpp``): a small call costs its host time.
"""
from __future__ import annotations

import ctypes
import functools
from array import array

from . import _check, _lib, _ptr, _stream

ACTIVATIONS = {"none": 0, "sigmoid": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4, "relu": 5, "tanh": 6}
NORMS = {"none": 0, "rms": 1, "layer": 2}

__all__ = [
    "conv_gated_fwd", "conv_gated_fwd_ex", "conv_gated_fwd_workspace_size", "conv_gated_bwd", "conv_gated_bwd_workspace_size", "conv_block_norm_fwd", "conv_block_norm_bwd",
    "conv_block_norm_bwd_workspace_size", "conv_grad_norm", "conv_grad_clip", "conv_grad_workspace_size",
    "gated_feed_forward", "gated_feed_forward_grad", "block_norm", "block_norm_grad", "gradient_norm",
    "clip_gradients", "ACTIVATIONS", "NORMS",
]


@functools.lru_cache(maxsize=1024)
def _size(name, device, *args) -> int:
    out = ctypes.c_size_t(0)
    _check(getattr(_lib.load(), name)(*args, ctypes.byref(out)))
    return out.value


def _device() -> int:
    """The current device (sizes may depend on its compute units), -1 without one."""
    import torch

    return torch.cuda.current_device() if torch.cuda.is_available() else -1


def conv_gated_fwd_workspace_size(rows, C, F, dtype) -> int:
    return _size("conv_gated_fwd_workspace_size", _device(), rows, C, F, dtype)


def conv_gated_bwd_workspace_size(rows, C, F, dtype) -> int:
    return _size("conv_gated_bwd_workspace_size", _device(), rows, C, F, dtype)


def conv_block_norm_bwd_workspace_size(rows, C, gate_rows) -> int:
    return _size("conv_block_norm_bwd_workspace_size", _device(), rows, C, gate_rows)


def conv_grad_workspace_size(n) -> int:
    return _size("conv_grad_workspace_size", 0, n)


def conv_gated_fwd(x, w_gate, w_up, b_gate, b_up, h, saved, rows, C, F, act, dtype, stream=None) -> None:
    p, st = _ptr, _stream
    _check(_lib.load().conv_gated_fwd(p(x), p(w_gate), p(w_up), p(b_gate), p(b_up), p(h), p(saved), rows, C, F, act, dtype,
                                     st(stream)))


def conv_gated_fwd_ex(x, w_gate, w_up, b_gate, b_up, h, saved, workspace, workspace_bytes, rows, C, F, act, dtype,
                      stream=None) -> None:
    p, st = _ptr, _stream
    _check(_lib.load().conv_gated_fwd_ex(p(x), p(w_gate), p(w_up), p(b_gate), p(b_up), p(h), p(saved), p(workspace),
                                         workspace_bytes, rows, C, F, act, dtype, st(stream)))


def conv_gated_bwd(dh, x, w_gate, w_up, b_gate, b_up, saved, dx, dw_gate, dw_up, db_gate, db_up, workspace,
                   workspace_bytes, rows, C, F, act, dtype, stream=None) -> None:
    p, st = _ptr, _stream
    _check(_lib.load().conv_gated_bwd(p(dh), p(x), p(w_gate), p(w_up), p(b_gate), p(b_up), p(saved), p(dx), p(dw_gate),
                                     p(dw_up), p(db_gate), p(db_up), p(workspace), workspace_bytes, rows, C, F, act,
                                     dtype, st(stream)))


def conv_block_norm_fwd(x, branch, gate, scale, post_w, post_b, pre_w, pre_b, y, a, rows, C, gate_rows, post, pre, act,
                        eps, dtype, stream=None) -> None:
    p, st = _ptr, _stream
    _check(_lib.load().conv_block_norm_fwd(p(x), p(branch), p(gate), p(scale), p(post_w), p(post_b), p(pre_w), p(pre_b),
                                          p(y), p(a), rows, C, gate_rows, post, pre, act, eps, dtype, st(stream)))


def conv_block_norm_bwd(dy, da, x, branch, gate, scale, post_w, post_b, pre_w, pre_b, dx, dbranch, dgate, dscale,
                        dpost_w, dpost_b, dpre_w, dpre_b, workspace, workspace_bytes, rows, C, gate_rows, post, pre,
                        act, eps, dtype, stream=None) -> None:
    p, st = _ptr, _stream
    _check(_lib.load().conv_block_norm_bwd(p(dy), p(da), p(x), p(branch), p(gate), p(scale), p(post_w), p(post_b),
                                          p(pre_w), p(pre_b), p(dx), p(dbranch), p(dgate), p(dscale), p(dpost_w),
                                          p(dpost_b), p(dpre_w), p(dpre_b), p(workspace), workspace_bytes, rows, C,
                                          gate_rows, post, pre, act, eps, dtype, st(stream)))


def _list(values, code):
    return None if values is None else array(code, values)


def conv_grad_norm(grads, counts, dtypes, n, norm, workspace, workspace_bytes, stream=None) -> None:
    """``grads``, ``counts`` and ``dtypes`` are sequences of n ints (device
    pointers, element counts, ``CONV_F32`` / ``CONV_BF16``)."""
    p, st = _ptr, _stream
    g, c, d = _list(grads, "Q"), _list(counts, "Q"), _list(dtypes, "i")
    _check(_lib.load().conv_grad_norm(g.buffer_info()[0], c.buffer_info()[0], d.buffer_info()[0], n, p(norm),
                                     p(workspace), workspace_bytes, st(stream)))


def conv_grad_clip(grads, outs, counts, dtypes, n, max_norm, eps, norm, workspace, workspace_bytes, stream=None) -> None:
    """Sequences as in ``conv_grad_norm``; ``outs`` may be ``grads``."""
    p, st = _ptr, _stream
    g, o, c, d = _list(grads, "Q"), _list(outs, "Q"), _list(counts, "Q"), _list(dtypes, "i")
    _check(_lib.load().conv_grad_clip(g.buffer_info()[0], o.buffer_info()[0], c.buffer_info()[0], d.buffer_info()[0], n,
                                     max_norm, eps, p(norm), p(workspace), workspace_bytes, st(stream)))


# ----------------------------------------------------------- tensor level --

_ABI = ("conv_gated_fwd_ex", "conv_gated_fwd_workspace_size", "conv_gated_bwd",
        "conv_gated_bwd_workspace_size", "conv_block_norm_fwd", "conv_block_norm_bwd",
        "conv_block_norm_bwd_workspace_size", "conv_grad_norm", "conv_grad_clip", "conv_grad_workspace_size")


@functools.lru_cache(maxsize=None)
def _native():
    """The native part, bound to the loaded library."""
    import torch  # noqa: F401  (its libraries have to be there first)

    lib = _lib.load()
    try:
        from . import _native as native
    except ImportError as e:
        raise RuntimeError("the native binding has not been built (run convolution_implicit_gemm_conv2d_amd.build.build())") from e
    native.bind(*[ctypes.cast(getattr(lib, name), ctypes.c_void_p).value for name in _ABI])
    return native


def _current(t, stream):
    """The raw current stream, or None where the call has to enter another
    device or stream.  0 for a tensor that the checks refuse."""
    import torch

    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        return 0
    device = t.get_device()
    if stream is not None or device != torch.cuda.current_device():
        return None
    return torch._C._cuda_getCurrentRawStream(device)


def _entered(fn, t, stream, *args):
    """``fn(*args)`` on the device of ``t`` and on ``stream``."""
    import torch

    with torch.cuda.device(t.device):
        if stream is None:
            return fn(*args)
        s = torch.cuda.ExternalStream(stream, device=t.device) if isinstance(stream, int) else stream
        with torch.cuda.stream(s):
            return fn(*args)


def _result(r):
    if type(r) is int:
        _check(r)
    return r


def _choice(table, value, what):
    try:
        return table[value]
    except KeyError:
        raise ValueError(f"{what} must be one of {', '.join(table)}; got {value!r}") from None


def gated_feed_forward(x, w_gate, w_up, b_gate=None, b_up=None, activation="silu", out=None, saved=None, stream=None):
    """``act(x w_gate^T + b_gate) * (x w_up^T + b_up)``: both 1x1 projections,
    the activation and the product in one kernel.

    ``x`` [..., C] (an NHWC or NLC batch, or tokens), weights [F, C] or as a
    1x1 convolution's OHWI weight [F, 1, 1, C]; returns [..., F].  ``saved``, a
    float32 tensor [..., 2F], receives both projections for
    ``gated_feed_forward_grad``."""
    s = _current(x, stream)
    if s is None:
        return _entered(gated_feed_forward, x, stream, x, w_gate, w_up, b_gate, b_up, activation, out, saved)
    act = _choice(ACTIVATIONS, activation, "activation")
    return _result(_native().gated(x, w_gate, w_up, b_gate, b_up, act, out, saved, s))


def gated_feed_forward_grad(dh, x, w_gate, w_up, b_gate=None, b_up=None, activation="silu", saved=None,
                            workspace=None, stream=None):
    """Gradient of ``gated_feed_forward`` from ``dh``: ``(dx, dw_gate, dw_up,
    db_gate, db_up)``, the last two ``None`` without biases.

    With ``saved`` (from the forward call) the projections are read, without it
    they are computed again.  ``workspace`` (a byte tensor) is allocated when
    not given."""
    s = _current(x, stream)
    if s is None:
        return _entered(gated_feed_forward_grad, x, stream, dh, x, w_gate, w_up, b_gate, b_up, activation, saved, workspace)
    act = _choice(ACTIVATIONS, activation, "activation")
    return _result(_native().gated_grad(x, w_gate, w_up, b_gate, b_up, act, dh, saved, workspace, s))


def block_norm(x, branch=None, gate=None, scale=None, post_weight=None, post_bias=None, pre_weight=None, pre_bias=None,
               post="none", pre="rms", gate_activation="none", eps=1e-6, stream=None):
    """``y = x + scale * act(gate) * post(branch)`` and ``a = pre(y)``:
    returns ``(y, a)``.

    ``post`` is the norm after the block that made ``branch``, ``pre`` the norm
    before the next one ("none", "rms" or "layer"); ``a`` is ``None`` without
    ``pre``, and without ``branch`` the call is ``pre`` alone (``y`` is then
    ``x`` itself).  ``gate`` has the shape of ``x``, or one row for each entry
    of its first dimension ([N, C]), or is a single row [C]."""
    s = _current(x, stream)
    if s is None:
        return _entered(block_norm, x, stream, x, branch, gate, scale, post_weight, post_bias, pre_weight, pre_bias, post,
                        pre, gate_activation, eps)
    return _result(_native().norm(x, branch, gate, scale, post_weight, post_bias, pre_weight, pre_bias,
                                  _choice(NORMS, post, "post"), _choice(NORMS, pre, "pre"),
                                  _choice(ACTIVATIONS, gate_activation, "gate_activation"), eps, s))


_NORM_INPUTS = ("x", "branch", "gate", "scale", "post_weight", "post_bias", "pre_weight", "pre_bias")


def block_norm_grad(dy, da, x, branch=None, gate=None, scale=None, post_weight=None, post_bias=None, pre_weight=None,
                    pre_bias=None, post="none", pre="rms", gate_activation="none", eps=1e-6, workspace=None, stream=None):
    """Gradient of ``block_norm`` from ``dy`` and ``da`` (the gradients of
    ``y`` and ``a``; ``None`` for zeros): a dict with "x", "branch", "gate",
    "scale", "post_weight", "post_bias", "pre_weight" and "pre_bias", ``None``
    for what the call does not have.  Takes the forward call's inputs."""
    s = _current(x, stream)
    if s is None:
        return _entered(block_norm_grad, x, stream, dy, da, x, branch, gate, scale, post_weight, post_bias, pre_weight,
                        pre_bias, post, pre, gate_activation, eps, workspace)
    return dict(zip(_NORM_INPUTS, _result(_native().norm_grad(
        x, branch, gate, scale, post_weight, post_bias, pre_weight, pre_bias, _choice(NORMS, post, "post"),
        _choice(NORMS, pre, "pre"), _choice(ACTIVATIONS, gate_activation, "gate_activation"), eps, dy, da, workspace, s))))


def gradient_norm(grads, stream=None):
    """The 2-norm over all elements of a non-empty list of dense tensors (float32
    and bfloat16 may be mixed), as a float32 scalar on their device."""
    grads = list(grads)
    s = _current(grads[0], stream) if grads else 0
    if s is None:
        return _entered(gradient_norm, grads[0], stream, grads)
    return _result(_native().clip(grads, None, 0.0, 0.0, s))


def clip_gradients(grads, max_norm, out=None, eps=1e-6, stream=None):
    """Scales a list of gradients by ``min(1, max_norm / (norm + eps))``, in
    place or into the tensors of ``out``, and returns the norm before it, a
    float32 scalar on the device.  Nothing waits for the device.  What is written
    must not overlap another tensor of the call: a tensor twice in the list is
    refused in place.  Tensors are dense, in any order of dimensions (channels-last
    ones, say); an output lies in memory as its gradient does."""
    grads = list(grads)
    s = _current(grads[0], stream) if grads else 0
    if s is None:
        return _entered(clip_gradients, grads[0], stream, grads, max_norm, out, eps)
    return _result(_native().clip(grads, grads if out is None else list(out), max_norm, eps, s))
