"""AdamW over a list of parameters, with states in 32 or 8 bits.

Argument marshalling only, like the rest of the binding: ``conv_adamw`` and
``conv_adamw_moments`` carry the C names and arguments, the others take lists of
tensors.  Streams, errors and automatic differentiation as in ``block``: nothing
waits for the device, and what a call writes counts a new version.
"""
from __future__ import annotations

from . import _check, _lib, _ptr, _stream
from .block import _current, _entered, _list, _native, _result

__all__ = ["conv_adamw", "conv_adamw_moments", "adamw_state", "adamw_step", "adamw_moments"]

BLOCK = 128  # elements that share a scale of 8-bit states


def _at(values, code="Q"):
    a = _list(values, code)
    return a, None if a is None else a.buffer_info()[0]


def conv_adamw(params, grads, m, v, m_scales, v_scales, copies, counts, param_dtypes, grad_dtypes, copy_dtypes, n, bits, lr, beta1,
               beta2, eps, weight_decay, step, lr_dev=None, step_dev=None, norm=None, max_norm=0.0, norm_eps=0.0, stream=None) -> None:
    """Lists are sequences of n ints (device pointers, element counts, ``CONV_F32`` /
    ``CONV_BF16``) or ``None``."""
    lists = [_at(t) for t in (params, grads, m, v, m_scales, v_scales, copies, counts)]
    lists += [_at(t, "i") for t in (param_dtypes, grad_dtypes, copy_dtypes)]
    _check(_lib.load().conv_adamw(*(at for _, at in lists), n, bits, lr, beta1, beta2, eps, weight_decay, step, _ptr(lr_dev),
                                 _ptr(step_dev), _ptr(norm), max_norm, norm_eps, _stream(stream)))


def conv_adamw_moments(m, v, m_scales, v_scales, m_out, v_out, counts, n, stream=None) -> None:
    """Lists as in ``conv_adamw``."""
    lists = [_at(t) for t in (m, v, m_scales, v_scales, m_out, v_out, counts)]
    _check(_lib.load().conv_adamw_moments(*(at for _, at in lists), n, _stream(stream)))


def adamw_state(params, bits=32):
    """States of a list of parameters before the first step: a dict of lists of
    tensors, "m" and "v" and with 8 bits "m_scale" and "v_scale".

    32 bits: float32, in the memory order of their parameter.  8 bits: a byte an
    element in that order, and a float32 scale for each 128: m = scale q |q| (q int8)
    and v = (scale q^2)^2 (q uint8)."""
    import torch

    params = list(params)
    if bits == 32:
        return {k: [torch.zeros_like(p, dtype=torch.float32) for p in params] for k in ("m", "v")}
    if bits != 8:
        raise ValueError(f"bits must be 8 or 32; got {bits!r}")
    zeros = lambda per, t: [torch.zeros(-(-p.numel() // per), dtype=t, device=p.device) for p in params]  # noqa: E731
    return {"m": zeros(1, torch.int8), "v": zeros(1, torch.uint8), "m_scale": zeros(BLOCK, torch.float32),
            "v_scale": zeros(BLOCK, torch.float32)}


def adamw_step(params, grads, state, step, lr, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, norm=None, max_norm=1.0,
               norm_eps=1e-6, copies=None, stream=None):
    """One AdamW step over a non-empty list of float32 and bfloat16 parameters, in place:

        g' = g min(1, max_norm / (norm + norm_eps))     without ``norm``: g
        m = b1 m + (1 - b1) g',   v = b2 v + (1 - b2) g'^2
        p = p (1 - lr weight_decay) - lr / (1 - b1^step) m / (sqrt(v / (1 - b2^step)) + eps)

    ``state`` is ``adamw_state``'s, ``step`` counts from 1.  ``norm`` is ``gradient_norm``'s
    result: clipping by it here saves ``clip_gradients``' pass over the gradients.
    ``copies`` (a list with ``None`` where there is none) receives the parameters once
    more, in its tensors' type: bfloat16 weights beside float32 parameters.  ``lr`` may
    be a float32 and ``step`` an int64 tensor of one value on the device, which a captured
    graph reads anew at each replay.  Gradients, float32 states and copies lie in
    memory as their parameters do; nothing may overlap what is written."""
    import torch

    params = list(params)
    s = _current(params[0], stream) if params else 0
    if s is None:
        return _entered(adamw_step, params[0], stream, params, grads, state, step, lr, betas, eps, weight_decay, norm, max_norm,
                        norm_eps, copies)
    lr_t, step_t = (t if isinstance(t, torch.Tensor) else None for t in (lr, step))
    rest = [None if t is None else list(t) for t in (grads, state["m"], state["v"], state.get("m_scale"), state.get("v_scale"), copies)]
    return _result(_native().adamw(params, *rest, 0.0 if lr_t is not None else lr, lr_t, betas[0], betas[1], eps, weight_decay,
                                   1 if step_t is not None else step, step_t, norm, max_norm, norm_eps, s))


def adamw_moments(state, out=None, stream=None):
    """The values that 8-bit states stand for, for a checkpoint: a dict of lists of
    float32 tensors "m" and "v" (those of ``out``, where given; contiguous, flat in the
    memory order of the parameters)."""
    import torch

    m = list(state["m"])
    if "m_scale" not in state:
        raise ValueError("states of 32 bits are their own values")
    s = _current(m[0], stream) if m else 0
    if s is None:
        return _entered(adamw_moments, m[0], stream, state, out)
    if out is None:
        out = {k: [torch.empty(t.numel(), dtype=torch.float32, device=t.device) for t in m] for k in ("m", "v")}
    _result(_native().moments(m, list(state["v"]), list(state["m_scale"]), list(state["v_scale"]), list(out["m"]), list(out["v"]), s))
    return out
