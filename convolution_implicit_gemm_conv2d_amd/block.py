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
"""
from __future__ import annotations

import contextlib
import ctypes
from array import array

from . import _lib

ACTIVATIONS = {"none": 0, "sigmoid": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4, "relu": 5, "tanh": 6}
NORMS = {"none": 0, "rms": 1, "layer": 2}

__all__ = [
    "conv_gated_fwd", "conv_gated_bwd", "conv_gated_bwd_workspace_size", "conv_block_norm_fwd", "conv_block_norm_bwd",
    "conv_block_norm_bwd_workspace_size", "conv_grad_norm", "conv_grad_clip", "conv_grad_workspace_size",
    "gated_feed_forward", "gated_feed_forward_grad", "block_norm", "block_norm_grad", "gradient_norm",
    "clip_gradients", "ACTIVATIONS", "NORMS",
]


def _checks():
    from . import _check, _dtype_code, _ptr, _stream  # the binding's own helpers

    return _check, _dtype_code, _ptr, _stream


def _size(name, *args) -> int:
    out = ctypes.c_size_t(0)
    _checks()[0](getattr(_lib.load(), name)(*args, ctypes.byref(out)))
    return out.value


def conv_gated_bwd_workspace_size(rows, C, F, dtype) -> int:
    return _size("conv_gated_bwd_workspace_size", rows, C, F, dtype)


def conv_block_norm_bwd_workspace_size(rows, C, gate_rows) -> int:
    return _size("conv_block_norm_bwd_workspace_size", rows, C, gate_rows)


def conv_grad_workspace_size(n) -> int:
    return _size("conv_grad_workspace_size", n)


def conv_gated_fwd(x, w_gate, w_up, b_gate, b_up, h, saved, rows, C, F, act, dtype, stream=None) -> None:
    check, _, p, st = _checks()
    check(_lib.load().conv_gated_fwd(p(x), p(w_gate), p(w_up), p(b_gate), p(b_up), p(h), p(saved), rows, C, F, act, dtype,
                                     st(stream)))


def conv_gated_bwd(dh, x, w_gate, w_up, b_gate, b_up, saved, dx, dw_gate, dw_up, db_gate, db_up, workspace,
                   workspace_bytes, rows, C, F, act, dtype, stream=None) -> None:
    check, _, p, st = _checks()
    check(_lib.load().conv_gated_bwd(p(dh), p(x), p(w_gate), p(w_up), p(b_gate), p(b_up), p(saved), p(dx), p(dw_gate),
                                     p(dw_up), p(db_gate), p(db_up), p(workspace), workspace_bytes, rows, C, F, act,
                                     dtype, st(stream)))


def conv_block_norm_fwd(x, branch, gate, scale, post_w, post_b, pre_w, pre_b, y, a, rows, C, gate_rows, post, pre, act,
                        eps, dtype, stream=None) -> None:
    check, _, p, st = _checks()
    check(_lib.load().conv_block_norm_fwd(p(x), p(branch), p(gate), p(scale), p(post_w), p(post_b), p(pre_w), p(pre_b),
                                          p(y), p(a), rows, C, gate_rows, post, pre, act, eps, dtype, st(stream)))


def conv_block_norm_bwd(dy, da, x, branch, gate, scale, post_w, post_b, pre_w, pre_b, dx, dbranch, dgate, dscale,
                        dpost_w, dpost_b, dpre_w, dpre_b, workspace, workspace_bytes, rows, C, gate_rows, post, pre,
                        act, eps, dtype, stream=None) -> None:
    check, _, p, st = _checks()
    check(_lib.load().conv_block_norm_bwd(p(dy), p(da), p(x), p(branch), p(gate), p(scale), p(post_w), p(post_b),
                                          p(pre_w), p(pre_b), p(dx), p(dbranch), p(dgate), p(dscale), p(dpost_w),
                                          p(dpost_b), p(dpre_w), p(dpre_b), p(workspace), workspace_bytes, rows, C,
                                          gate_rows, post, pre, act, eps, dtype, st(stream)))


def _list(values, code):
    return None if values is None else array(code, values)


def conv_grad_norm(grads, counts, dtypes, n, norm, workspace, workspace_bytes, stream=None) -> None:
    """``grads``, ``counts`` and ``dtypes`` are sequences of n ints (device
    pointers, element counts, ``CONV_F32`` / ``CONV_BF16``)."""
    check, _, p, st = _checks()
    g, c, d = _list(grads, "Q"), _list(counts, "Q"), _list(dtypes, "i")
    check(_lib.load().conv_grad_norm(g.buffer_info()[0], c.buffer_info()[0], d.buffer_info()[0], n, p(norm),
                                     p(workspace), workspace_bytes, st(stream)))


def conv_grad_clip(grads, outs, counts, dtypes, n, max_norm, eps, norm, workspace, workspace_bytes, stream=None) -> None:
    """Sequences as in ``conv_grad_norm``; ``outs`` may be ``grads``."""
    check, _, p, st = _checks()
    g, o, c, d = _list(grads, "Q"), _list(outs, "Q"), _list(counts, "Q"), _list(dtypes, "i")
    check(_lib.load().conv_grad_clip(g.buffer_info()[0], o.buffer_info()[0], c.buffer_info()[0], d.buffer_info()[0], n,
                                     max_norm, eps, p(norm), p(workspace), workspace_bytes, st(stream)))


# ----------------------------------------------------------- tensor level --

@contextlib.contextmanager
def _entered(device, stream):
    import torch

    with torch.cuda.device(device):
        if stream is None:
            yield
        else:
            s = torch.cuda.ExternalStream(stream, device=device) if isinstance(stream, int) else stream
            with torch.cuda.stream(s):
                yield


_HERE = contextlib.nullcontext()


def _on(t, stream):
    """The context a call allocates and launches in; nothing to enter on the
    current stream of the current device."""
    import torch

    if not t.is_cuda:
        raise ValueError("tensors passed to convmi must be on a GPU device")
    if stream is None and t.device.index == torch.cuda.current_device():
        return _HERE
    return _entered(t.device, stream)


def _same(x, **tensors):
    for name, t in tensors.items():
        if t is not None and (t.dtype != x.dtype or t.device != x.device):
            raise ValueError(f"{name} must have the dtype and device of the input ({x.dtype}, {x.device}); "
                             f"found {t.dtype}, {t.device}")


def _shaped(shape, **tensors):
    for name, t in tensors.items():
        if t is not None and tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name} must have shape {list(shape)}; found {list(t.shape)}")


def _choice(table, value, what):
    try:
        return table[value]
    except KeyError:
        raise ValueError(f"{what} must be one of {', '.join(table)}; got {value!r}") from None


def _rows(x):
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError("an input has at least one dimension and one channel")
    C = x.shape[-1]
    return x.numel() // C, C


def _gated_sizes(x, w_gate, w_up, b_gate, b_up):
    rows, C = _rows(x)
    for name, w in (("w_gate", w_gate), ("w_up", w_up)):
        if w.dim() < 2 or w.shape[-1] != C or w.numel() != w.shape[0] * C:
            raise ValueError(f"{name} must be a 1x1 weight [F, {C}] (or [F, 1, 1, {C}]); found {list(w.shape)}")
    if w_gate.shape != w_up.shape or w_gate.shape[0] < 1:
        raise ValueError(f"w_gate and w_up must have one shape; found {list(w_gate.shape)}, {list(w_up.shape)}")
    F = w_gate.shape[0]
    _shaped((F,), b_gate=b_gate, b_up=b_up)
    if (b_gate is None) != (b_up is None):
        raise ValueError("b_gate and b_up come together")
    _same(x, w_gate=w_gate, w_up=w_up, b_gate=b_gate, b_up=b_up)
    return rows, C, F


def _check_saved(saved, x, rows, F):
    import torch

    if saved is not None and (saved.dtype != torch.float32 or saved.numel() != rows * 2 * F or saved.shape[-1] != 2 * F
                              or saved.device != x.device):
        raise ValueError(f"saved must be float32 on {x.device} with {rows} rows of {2 * F} values; "
                         f"found {saved.dtype} {list(saved.shape)}")


def gated_feed_forward(x, w_gate, w_up, b_gate=None, b_up=None, activation="silu", out=None, saved=None, stream=None):
    """``act(x w_gate^T + b_gate) * (x w_up^T + b_up)``: both 1x1 projections,
    the activation and the product in one kernel.

    ``x`` [..., C] (an NHWC or NLC batch, or tokens), weights [F, C] or as a
    1x1 convolution's OHWI weight [F, 1, 1, C]; returns [..., F].  ``saved``, a
    float32 tensor [..., 2F], receives both projections for
    ``gated_feed_forward_grad``."""
    import torch

    check, code, p, st = _checks()
    dt, act = code(x), _choice(ACTIVATIONS, activation, "activation")
    rows, C, F = _gated_sizes(x, w_gate, w_up, b_gate, b_up)
    shape = (*x.shape[:-1], F)
    _shaped(shape, out=out)
    _same(x, out=out)
    _check_saved(saved, x, rows, F)
    with _on(x, stream):
        if out is None:
            out = torch.empty(shape, dtype=x.dtype, device=x.device)
        check(_lib.load().conv_gated_fwd(p(x), p(w_gate), p(w_up), p(b_gate), p(b_up), p(out), p(saved), rows, C, F, act,
                                         dt, st(stream)))
    return out


def gated_feed_forward_grad(dh, x, w_gate, w_up, b_gate=None, b_up=None, activation="silu", saved=None,
                            workspace=None, stream=None):
    """Gradient of ``gated_feed_forward`` from ``dh``: ``(dx, dw_gate, dw_up,
    db_gate, db_up)``, the last two ``None`` without biases.

    With ``saved`` (from the forward call) the projections are read, without it
    they are computed again.  ``workspace`` (a byte tensor) is allocated when
    not given."""
    import torch

    check, code, p, st = _checks()
    dt, act = code(x), _choice(ACTIVATIONS, activation, "activation")
    rows, C, F = _gated_sizes(x, w_gate, w_up, b_gate, b_up)
    _shaped((*x.shape[:-1], F), dh=dh)
    _same(x, dh=dh)
    _check_saved(saved, x, rows, F)
    with _on(x, stream):
        dx = torch.empty_like(x, memory_format=torch.contiguous_format)
        dwg = torch.empty_like(w_gate, memory_format=torch.contiguous_format)
        dwu = torch.empty_like(w_up, memory_format=torch.contiguous_format)
        dbg = dbu = None
        if b_gate is not None:
            dbg, dbu = torch.empty_like(b_gate), torch.empty_like(b_up)
        if workspace is None:
            workspace = torch.empty(max(conv_gated_bwd_workspace_size(rows, C, F, dt), 16), dtype=torch.uint8,
                                    device=x.device)
        check(_lib.load().conv_gated_bwd(p(dh), p(x), p(w_gate), p(w_up), p(b_gate), p(b_up), p(saved), p(dx), p(dwg),
                                         p(dwu), p(dbg), p(dbu), p(workspace),
                                         workspace.numel() * workspace.element_size(), rows, C, F, act, dt, st(stream)))
    return dx, dwg, dwu, dbg, dbu


def _norm_sizes(x, branch, gate, scale, post_weight, post_bias, pre_weight, pre_bias, post, pre, gate_activation):
    rows, C = _rows(x)
    kinds = _choice(NORMS, post, "post"), _choice(NORMS, pre, "pre"), _choice(ACTIVATIONS, gate_activation,
                                                                             "gate_activation")
    _shaped(x.shape, branch=branch)
    _shaped((C,), scale=scale, post_weight=post_weight, post_bias=post_bias, pre_weight=pre_weight, pre_bias=pre_bias)
    _same(x, branch=branch, gate=gate, scale=scale, post_weight=post_weight, post_bias=post_bias,
          pre_weight=pre_weight, pre_bias=pre_bias)
    gate_rows = 1
    if gate is not None:
        if gate.shape == x.shape:
            gate_rows = 1
        elif tuple(gate.shape) == (x.shape[0], C) and x.dim() > 1:
            gate_rows = max(rows // max(x.shape[0], 1), 1)
        elif tuple(gate.shape) == (C,):
            gate_rows = max(rows, 1)
        else:
            raise ValueError(f"gate must have shape {list(x.shape)}, {[x.shape[0], C]} or {[C]}; "
                             f"found {list(gate.shape)}")
    return rows, C, gate_rows, kinds


def block_norm(x, branch=None, gate=None, scale=None, post_weight=None, post_bias=None, pre_weight=None, pre_bias=None,
               post="none", pre="rms", gate_activation="none", eps=1e-6, stream=None):
    """``y = x + scale * act(gate) * post(branch)`` and ``a = pre(y)``:
    returns ``(y, a)``.

    ``post`` is the norm after the block that made ``branch``, ``pre`` the norm
    before the next one ("none", "rms" or "layer"); ``a`` is ``None`` without
    ``pre``, and without ``branch`` the call is ``pre`` alone (``y`` is then
    ``x`` itself).  ``gate`` has the shape of ``x``, or one row for each entry
    of its first dimension ([N, C]), or is a single row [C]."""
    import torch

    check, code, p, st = _checks()
    dt = code(x)
    rows, C, gate_rows, (k_post, k_pre, act) = _norm_sizes(x, branch, gate, scale, post_weight, post_bias, pre_weight,
                                                           pre_bias, post, pre, gate_activation)
    if branch is None and pre == "none":
        raise ValueError("without a branch and a pre norm there is nothing to compute")
    with _on(x, stream):
        y = None if branch is None else torch.empty_like(x, memory_format=torch.contiguous_format)
        a = None if pre == "none" else torch.empty_like(x, memory_format=torch.contiguous_format)
        check(_lib.load().conv_block_norm_fwd(p(x), p(branch), p(gate), p(scale), p(post_weight), p(post_bias),
                                              p(pre_weight), p(pre_bias), p(y), p(a), rows, C, gate_rows, k_post, k_pre,
                                              act, eps, dt, st(stream)))
    return (x if branch is None else y), a


def block_norm_grad(dy, da, x, branch=None, gate=None, scale=None, post_weight=None, post_bias=None, pre_weight=None,
                    pre_bias=None, post="none", pre="rms", gate_activation="none", eps=1e-6, workspace=None, stream=None):
    """Gradient of ``block_norm`` from ``dy`` and ``da`` (the gradients of
    ``y`` and ``a``; ``None`` for zeros): a dict with "x", "branch", "gate",
    "scale", "post_weight", "post_bias", "pre_weight" and "pre_bias", ``None``
    for what the call does not have.  Takes the forward call's inputs."""
    import torch

    check, code, p, st = _checks()
    dt = code(x)
    rows, C, gate_rows, (k_post, k_pre, act) = _norm_sizes(x, branch, gate, scale, post_weight, post_bias, pre_weight,
                                                           pre_bias, post, pre, gate_activation)
    _shaped(x.shape, dy=dy, da=da)
    _same(x, dy=dy, da=da)
    with _on(x, stream):
        like = {"x": x, "branch": branch, "gate": gate, "scale": scale, "post_weight": post_weight,
                "post_bias": post_bias, "pre_weight": pre_weight, "pre_bias": pre_bias}
        d = {k: None if t is None else torch.empty_like(t, memory_format=torch.contiguous_format) for k, t in like.items()}
        if workspace is None:
            need = conv_block_norm_bwd_workspace_size(rows, C, gate_rows if gate is not None else 0)
            workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=x.device)
        check(_lib.load().conv_block_norm_bwd(
            p(dy), p(da), p(x), p(branch), p(gate), p(scale), p(post_weight), p(post_bias), p(pre_weight), p(pre_bias),
            p(d["x"]), p(d["branch"]), p(d["gate"]), p(d["scale"]), p(d["post_weight"]), p(d["post_bias"]),
            p(d["pre_weight"]), p(d["pre_bias"]), p(workspace), workspace.numel() * workspace.element_size(), rows, C,
            gate_rows, k_post, k_pre, act, eps, dt, st(stream)))
    return d


def _tensor_list(grads):
    """(pointers, element counts, dtype codes) of a list of dense tensors on
    one device."""
    import torch

    T = torch.Tensor
    codes = {torch.float32: 0, torch.bfloat16: 1}
    try:
        dtypes = array("i", [codes[t.dtype] for t in grads])
    except KeyError as e:
        raise ValueError(f"unsupported dtype {e.args[0]}; convmi takes float32 or bfloat16") from None
    if not all([t.is_cuda for t in grads]) or len({t.get_device() for t in grads}) > 1:
        raise ValueError("tensors passed to convmi must be on one GPU device")
    if not all(map(T.is_contiguous, grads)):
        raise ValueError("tensors passed to convmi must be contiguous")
    return array("Q", map(T.data_ptr, grads)), array("Q", map(T.numel, grads)), dtypes


def _list_call(grads, stream, call):
    import torch

    check, _, _, st = _checks()
    with _on(grads[0], stream):
        n = len(grads)
        norm = torch.empty((), dtype=torch.float32, device=grads[0].device)
        workspace = torch.empty(conv_grad_workspace_size(n), dtype=torch.uint8, device=grads[0].device)
        check(call(n, norm.data_ptr(), workspace.data_ptr(), workspace.numel(), st(stream)))
    return norm


def gradient_norm(grads, stream=None):
    """The 2-norm over all elements of a non-empty list of tensors (float32 and
    bfloat16 may be mixed), as a float32 scalar on their device."""
    grads = list(grads)
    if not grads:
        raise ValueError("the list of gradients is empty")
    g, c, d = _tensor_list(grads)
    return _list_call(grads, stream, lambda n, norm, ws, size, s: _lib.load().conv_grad_norm(
        g.buffer_info()[0], c.buffer_info()[0], d.buffer_info()[0], n, norm, ws, size, s))


def clip_gradients(grads, max_norm, out=None, eps=1e-6, stream=None):
    """Scales a list of gradients by ``min(1, max_norm / (norm + eps))``, in
    place or into the tensors of ``out``, and returns the norm before it, a
    float32 scalar on the device.  Nothing waits for the device."""
    grads = list(grads)
    if not grads:
        raise ValueError("the list of gradients is empty")
    g, c, d = _tensor_list(grads)
    o = g
    if out is not None:
        out = list(out)
        if len(out) != len(grads):
            raise ValueError(f"out has {len(out)} tensors for {len(grads)} gradients")
        o, co, do = _tensor_list(out)
        if co != c or do != d or out[0].device != grads[0].device:
            raise ValueError("the tensors of out must have the sizes, dtypes and device of the gradients")
    return _list_call(grads, stream, lambda n, norm, ws, size, s: _lib.load().conv_grad_clip(
        g.buffer_info()[0], o.buffer_info()[0], c.buffer_info()[0], d.buffer_info()[0], n, max_norm, eps, norm, ws,
        size, s))
