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

A small call costs its host time (a token through a norm: 3 us on the device),
so each tensor is looked at once, sizes of workspaces are remembered, and the
usual call (the current stream of the current device) enters no context.
"""
from __future__ import annotations

import ctypes
import functools
from array import array

from . import _check, _dtype_code, _lib, _ptr, _stream

ACTIVATIONS = {"none": 0, "sigmoid": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4, "relu": 5, "tanh": 6}
NORMS = {"none": 0, "rms": 1, "layer": 2}

__all__ = [
    "conv_gated_fwd", "conv_gated_bwd", "conv_gated_bwd_workspace_size", "conv_block_norm_fwd", "conv_block_norm_bwd",
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

def _elsewhere(t, stream) -> bool:
    """Whether the call has to enter another device or stream."""
    import torch

    if not t.is_cuda:
        raise ValueError("tensors passed to convmi must be on a GPU device")
    return stream is not None or t.get_device() != torch.cuda.current_device()


def _entered(fn, t, stream, *args, **kwargs):
    """``fn`` on the device of ``t`` and on ``stream``."""
    import torch

    with torch.cuda.device(t.device):
        if stream is None:
            return fn(*args, **kwargs)
        s = torch.cuda.ExternalStream(stream, device=t.device) if isinstance(stream, int) else stream
        with torch.cuda.stream(s):
            return fn(*args, **kwargs)


def _here(device) -> int:
    """The raw current stream."""
    import torch

    return torch._C._cuda_getCurrentRawStream(device)


def _like():
    """Allocates a tensor like another (all inputs were found contiguous)."""
    import torch

    return torch.empty_like


def _at(name, t, shape, dtype, device):
    """Address of an optional tensor, after its checks."""
    if t is None:
        return None
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {list(shape)}; found {list(t.shape)}")
    if t.dtype is not dtype or t.get_device() != device:
        raise ValueError(f"{name} must have the dtype and device of the input ({dtype}, GPU {device}); "
                         f"found {t.dtype}, {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _choice(table, value, what):
    try:
        return table[value]
    except KeyError:
        raise ValueError(f"{what} must be one of {', '.join(table)}; got {value!r}") from None


def _rows(x):
    shape = x.shape
    if not shape or shape[-1] < 1:
        raise ValueError("an input has at least one dimension and one channel")
    C = shape[-1]
    return x.numel() // C, C


def _gated_args(x, w_gate, w_up, b_gate, b_up, saved):
    """Sizes and addresses that the layer and its gradient share."""
    rows, C = _rows(x)
    shape, dtype, device = w_gate.shape, x.dtype, x.get_device()
    if len(shape) < 2 or shape[0] < 1 or shape[-1] != C or w_gate.numel() != shape[0] * C:
        raise ValueError(f"w_gate must be a 1x1 weight [F, {C}] (or [F, 1, 1, {C}]); found {list(shape)}")
    F = shape[0]
    if (b_gate is None) != (b_up is None):
        raise ValueError("b_gate and b_up come together")
    at = (_at("x", x, x.shape, dtype, device), _at("w_gate", w_gate, shape, dtype, device),
          _at("w_up", w_up, shape, dtype, device), _at("b_gate", b_gate, (F,), dtype, device),
          _at("b_up", b_up, (F,), dtype, device))
    kept = None
    if saved is not None:
        import torch

        if saved.dtype is not torch.float32 or saved.numel() != rows * 2 * F or saved.shape[-1] != 2 * F \
                or saved.get_device() != device or not saved.is_contiguous():
            raise ValueError(f"saved must be contiguous float32 on the input's device, with {rows} rows of {2 * F} "
                             f"values; found {saved.dtype} {list(saved.shape)} on {saved.device}")
        kept = saved.data_ptr()
    return rows, C, F, at, kept


def gated_feed_forward(x, w_gate, w_up, b_gate=None, b_up=None, activation="silu", out=None, saved=None, stream=None):
    """``act(x w_gate^T + b_gate) * (x w_up^T + b_up)``: both 1x1 projections,
    the activation and the product in one kernel.

    ``x`` [..., C] (an NHWC or NLC batch, or tokens), weights [F, C] or as a
    1x1 convolution's OHWI weight [F, 1, 1, C]; returns [..., F].  ``saved``, a
    float32 tensor [..., 2F], receives both projections for
    ``gated_feed_forward_grad``."""
    dt, act = _dtype_code(x), _choice(ACTIVATIONS, activation, "activation")
    rows, C, F, at, kept = _gated_args(x, w_gate, w_up, b_gate, b_up, saved)
    shape = x.shape[:-1] + (F,)
    to = None if out is None else _at("out", out, shape, x.dtype, x.get_device())
    if _elsewhere(x, stream):
        return _entered(gated_feed_forward, x, stream, x, w_gate, w_up, b_gate, b_up, activation, out, saved)
    if out is None:
        out = x.new_empty(shape)
        to = out.data_ptr()
    _check(_lib.load().conv_gated_fwd(*at, to, kept, rows, C, F, act, dt, _here(x.get_device())))
    return out


def gated_feed_forward_grad(dh, x, w_gate, w_up, b_gate=None, b_up=None, activation="silu", saved=None,
                            workspace=None, stream=None):
    """Gradient of ``gated_feed_forward`` from ``dh``: ``(dx, dw_gate, dw_up,
    db_gate, db_up)``, the last two ``None`` without biases.

    With ``saved`` (from the forward call) the projections are read, without it
    they are computed again.  ``workspace`` (a byte tensor) is allocated when
    not given."""
    dt, act = _dtype_code(x), _choice(ACTIVATIONS, activation, "activation")
    rows, C, F, at, kept = _gated_args(x, w_gate, w_up, b_gate, b_up, saved)
    dh_at = _at("dh", dh, x.shape[:-1] + (F,), x.dtype, x.get_device())
    if dh_at is None:
        raise ValueError("dh must be a tensor")
    if _elsewhere(x, stream):
        return _entered(gated_feed_forward_grad, x, stream, dh, x, w_gate, w_up, b_gate, b_up, activation, saved, workspace)
    device, like = x.get_device(), _like()
    dx, dwg, dwu = like(x), like(w_gate), like(w_up)
    dbg = dbu = pbg = pbu = None
    if b_gate is not None:
        dbg, dbu = like(b_gate), like(b_up)
        pbg, pbu = dbg.data_ptr(), dbu.data_ptr()
    ws, size = _workspace(workspace, x, _size("conv_gated_bwd_workspace_size", device, rows, C, F, dt))
    _check(_lib.load().conv_gated_bwd(dh_at, *at, kept, dx.data_ptr(), dwg.data_ptr(), dwu.data_ptr(), pbg, pbu,
                                      ws.data_ptr(), size, rows, C, F, act, dt, _here(device)))
    return dx, dwg, dwu, dbg, dbu


def _workspace(given, x, need):
    """(workspace, its bytes)"""
    import torch

    if given is None:
        need = max(need, 16)
        return torch.empty(need, dtype=torch.uint8, device=x.device), need
    if given.get_device() != x.get_device() or not given.is_contiguous():
        raise ValueError("the workspace must be a contiguous tensor on the input's device")
    return given, given.numel() * given.element_size()


def _norm_args(x, branch, gate, scale, post_weight, post_bias, pre_weight, pre_bias, post, pre, gate_activation):
    """Sizes, addresses and codes that the norms and their gradient share."""
    rows, C = _rows(x)
    kinds = _choice(NORMS, post, "post"), _choice(NORMS, pre, "pre"), _choice(ACTIVATIONS, gate_activation,
                                                                             "gate_activation")
    shape, dtype, device = x.shape, x.dtype, x.get_device()
    gate_rows, gate_shape = 1, None
    if gate is not None:
        gate_shape = gate.shape
        if gate_shape == shape:
            gate_rows = 1
        elif len(shape) > 1 and gate_shape == (shape[0], C):
            gate_rows = max(rows // max(shape[0], 1), 1)
        elif gate_shape == (C,):
            gate_rows = max(rows, 1)
        else:
            raise ValueError(f"gate must have shape {list(shape)}, {[shape[0], C]} or {[C]}; found {list(gate_shape)}")
    row = (C,)
    at = (_at("x", x, shape, dtype, device), _at("branch", branch, shape, dtype, device),
          _at("gate", gate, gate_shape, dtype, device), _at("scale", scale, row, dtype, device),
          _at("post_weight", post_weight, row, dtype, device), _at("post_bias", post_bias, row, dtype, device),
          _at("pre_weight", pre_weight, row, dtype, device), _at("pre_bias", pre_bias, row, dtype, device))
    return rows, C, gate_rows, at, kinds


def block_norm(x, branch=None, gate=None, scale=None, post_weight=None, post_bias=None, pre_weight=None, pre_bias=None,
               post="none", pre="rms", gate_activation="none", eps=1e-6, stream=None):
    """``y = x + scale * act(gate) * post(branch)`` and ``a = pre(y)``:
    returns ``(y, a)``.

    ``post`` is the norm after the block that made ``branch``, ``pre`` the norm
    before the next one ("none", "rms" or "layer"); ``a`` is ``None`` without
    ``pre``, and without ``branch`` the call is ``pre`` alone (``y`` is then
    ``x`` itself).  ``gate`` has the shape of ``x``, or one row for each entry
    of its first dimension ([N, C]), or is a single row [C]."""
    dt = _dtype_code(x)
    rows, C, gate_rows, at, (k_post, k_pre, act) = _norm_args(x, branch, gate, scale, post_weight, post_bias, pre_weight,
                                                              pre_bias, post, pre, gate_activation)
    if branch is None and pre == "none":
        raise ValueError("without a branch and a pre norm there is nothing to compute")
    if _elsewhere(x, stream):
        return _entered(block_norm, x, stream, x, branch, gate, scale, post_weight, post_bias, pre_weight, pre_bias, post,
                        pre, gate_activation, eps)
    y = a = to_y = to_a = None
    like = _like()
    if branch is not None:
        y = like(x)
        to_y = y.data_ptr()
    if pre != "none":
        a = like(x)
        to_a = a.data_ptr()
    _check(_lib.load().conv_block_norm_fwd(*at, to_y, to_a, rows, C, gate_rows, k_post, k_pre, act, eps, dt,
                                           _here(x.get_device())))
    return (x if branch is None else y), a


_NORM_INPUTS = ("x", "branch", "gate", "scale", "post_weight", "post_bias", "pre_weight", "pre_bias")


def block_norm_grad(dy, da, x, branch=None, gate=None, scale=None, post_weight=None, post_bias=None, pre_weight=None,
                    pre_bias=None, post="none", pre="rms", gate_activation="none", eps=1e-6, workspace=None, stream=None):
    """Gradient of ``block_norm`` from ``dy`` and ``da`` (the gradients of
    ``y`` and ``a``; ``None`` for zeros): a dict with "x", "branch", "gate",
    "scale", "post_weight", "post_bias", "pre_weight" and "pre_bias", ``None``
    for what the call does not have.  Takes the forward call's inputs."""
    dt = _dtype_code(x)
    rows, C, gate_rows, at, (k_post, k_pre, act) = _norm_args(x, branch, gate, scale, post_weight, post_bias, pre_weight,
                                                              pre_bias, post, pre, gate_activation)
    device = x.get_device()
    grads_at = _at("dy", dy, x.shape, x.dtype, device), _at("da", da, x.shape, x.dtype, device)
    if _elsewhere(x, stream):
        return _entered(block_norm_grad, x, stream, dy, da, x, branch, gate, scale, post_weight, post_bias, pre_weight,
                        pre_bias, post, pre, gate_activation, eps, workspace)
    like = _like()
    d = [None if t is None else like(t)
         for t in (x, branch, gate, scale, post_weight, post_bias, pre_weight, pre_bias)]
    ws, size = _workspace(workspace, x, _size("conv_block_norm_bwd_workspace_size", device, rows, C,
                                              gate_rows if gate is not None else 0))
    _check(_lib.load().conv_block_norm_bwd(*grads_at, *at, *[None if t is None else t.data_ptr() for t in d],
                                           ws.data_ptr(), size, rows, C, gate_rows, k_post, k_pre, act, eps, dt,
                                           _here(device)))
    return dict(zip(_NORM_INPUTS, d))


_CODES = {}  # dtype: code, filled with the first list


def _tensor_list(grads):
    """(pointers, element counts, dtype codes) of a list of dense tensors on
    one device."""
    import torch

    T = torch.Tensor
    if not _CODES:
        _CODES.update({torch.float32: 0, torch.bfloat16: 1})
    try:
        dtypes = array("i", [_CODES[t.dtype] for t in grads])
    except KeyError as e:
        raise ValueError(f"unsupported dtype {e.args[0]}; convmi takes float32 or bfloat16") from None
    devices = set(map(T.get_device, grads))
    if len(devices) > 1 or min(devices) < 0:
        raise ValueError("tensors passed to convmi must be on one GPU device")
    if not all(map(T.is_contiguous, grads)):
        raise ValueError("tensors passed to convmi must be contiguous")
    return array("Q", map(T.data_ptr, grads)), array("Q", map(T.numel, grads)), dtypes


def _list_scratch(t, n):
    """The norm, the workspace and its bytes for a list of n tensors."""
    import torch

    size = _size("conv_grad_workspace_size", 0, n)
    return t.new_empty((), dtype=torch.float32), t.new_empty(size, dtype=torch.uint8), size


def gradient_norm(grads, stream=None):
    """The 2-norm over all elements of a non-empty list of tensors (float32 and
    bfloat16 may be mixed), as a float32 scalar on their device."""
    grads = list(grads)
    if not grads:
        raise ValueError("the list of gradients is empty")
    if _elsewhere(grads[0], stream):
        return _entered(gradient_norm, grads[0], stream, grads)
    g, c, d = _tensor_list(grads)
    n = len(grads)
    norm, ws, size = _list_scratch(grads[0], n)
    _check(_lib.load().conv_grad_norm(g.buffer_info()[0], c.buffer_info()[0], d.buffer_info()[0], n, norm.data_ptr(),
                                      ws.data_ptr(), size, _here(grads[0].get_device())))
    return norm


def clip_gradients(grads, max_norm, out=None, eps=1e-6, stream=None):
    """Scales a list of gradients by ``min(1, max_norm / (norm + eps))``, in
    place or into the tensors of ``out``, and returns the norm before it, a
    float32 scalar on the device.  Nothing waits for the device."""
    grads = list(grads)
    if not grads:
        raise ValueError("the list of gradients is empty")
    out = grads if out is None else list(out)
    if len(out) != len(grads):
        raise ValueError(f"out has {len(out)} tensors for {len(grads)} gradients")
    if _elsewhere(grads[0], stream):
        return _entered(clip_gradients, grads[0], stream, grads, max_norm, out, eps)
    g, c, d = _tensor_list(grads)
    o = g
    if out is not grads:
        o, co, do = _tensor_list(out)
        if co != c or do != d or out[0].get_device() != grads[0].get_device():
            raise ValueError("the tensors of out must have the sizes, dtypes and device of the gradients")
    n = len(grads)
    norm, ws, size = _list_scratch(grads[0], n)
    _check(_lib.load().conv_grad_clip(g.buffer_info()[0], o.buffer_info()[0], c.buffer_info()[0], d.buffer_info()[0], n,
                                      max_norm, eps, norm.data_ptr(), ws.data_ptr(), size,
                                      _here(grads[0].get_device())))
    return norm
