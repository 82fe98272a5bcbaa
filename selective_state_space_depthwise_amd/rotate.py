"""Torch-tensor front end of the head norm with position rotation: argument marshalling only, as in
api.py."""
from __future__ import annotations

import math
from typing import NamedTuple, Optional

import torch

from . import _abi
from ._abi import AxonError
from .api import _act_dtype
from .delta import _dense, _gpu, _handle, _lib, _ptr, _row_stride, _rows
from .linear import _Launch, _made, _optional, _workspace


def _inputs(q, k, positions, freqs, q_weight, k_weight, eps, interleaved, device):
    """Checks that both directions share; the desc without the output gradients' strides."""
    bf16 = _act_dtype(q)
    if q.dim() < 2:
        raise ValueError("q must be (..., heads, head_dim)")
    lead = tuple(q.shape[:-2])
    hq, D = q.shape[-2:]
    qs = _row_stride(q, "q", (hq, D))
    hk, ks = 0, 0
    if k is None:
        if k_weight is not None:
            raise ValueError("k_weight belongs to k")
    else:
        if not isinstance(k, torch.Tensor):
            raise TypeError("k must be a torch.Tensor")
        if k.dim() != q.dim():
            raise ValueError("q and k must have the same leading axes")
        hk = k.shape[-2]
        if hk < 1:
            raise ValueError("k has no heads")
        ks = _rows(k, "k", lead, (hk, D), q.dtype, device)
    _dense(positions, "positions", lead, torch.int32, device)
    if not isinstance(freqs, torch.Tensor) or freqs.dim() != 1:
        raise ValueError("freqs must be a tensor (rotary_dim / 2,)")
    _dense(freqs, "freqs", tuple(freqs.shape), torch.float64, device)
    _optional(q_weight, "q_weight", (D,), torch.float32, device)
    _optional(k_weight, "k_weight", (D,), torch.float32, device)
    return lead, _abi.NormRotateDesc(math.prod(lead), hq, hk, D, 2 * freqs.shape[0], qs, ks, 0, 0,
                                     float(eps), _abi.AXON_BF16 if bf16 else _abi.AXON_F32,
                                     1 if interleaved else 0)


def norm_rotate(q, k, positions, freqs, *, q_weight=None, k_weight=None, eps=1e-6,
                interleaved=False, q_out=None, k_out=None, stream=None):
    """RMS norm of every head of q (..., Hq, D) and k (..., Hk, D; or None) and the rotation of its
    first 2 len(freqs) channels by the row's position, in one pass (axon_norm_rotate).

    float32 or bfloat16; the rows of q and k may lie apart (parts of one projection). positions (...)
    int32; freqs (R / 2,) float64, radians a token (base ** (-2 i / R)); pairs are (i, i + R / 2), with
    ``interleaved`` (2 i, 2 i + 1). D even, up to 256. Weights (D,) float32, None = ones. q_out may be
    q and k_out k where they are contiguous. Returns (q_out, k_out). As every call here it records no
    autograd graph (norm_rotate_backward is its gradient). Asynchronous on ``stream`` (default:
    torch's current stream)."""
    device = _gpu(q, "q", "norm_rotate")
    _, desc = _inputs(q, k, positions, freqs, q_weight, k_weight, eps, interleaved, device)
    if k is None and k_out is not None:
        raise ValueError("k_out belongs to k")
    with _Launch(device, stream) as on:
        mine = []
        q_out = _made(q_out, "q_out", q, mine)
        if k is not None:
            k_out = _made(k_out, "k_out", k, mine)
        on.keep(mine)
        st = _lib().axon_norm_rotate(desc, q.data_ptr(), _ptr(k), positions.data_ptr(),
                                     freqs.data_ptr(), _ptr(q_weight), _ptr(k_weight),
                                     q_out.data_ptr(), _ptr(k_out), _handle(device, stream))
    if st != _abi.AXON_OK:
        raise AxonError(st, "axon_norm_rotate")
    return q_out, k_out


class NormRotateGrads(NamedTuple):
    """Gradients of norm_rotate, like what they belong to; None where that was None."""
    dq: torch.Tensor
    dk: Optional[torch.Tensor]
    dq_weight: Optional[torch.Tensor]
    dk_weight: Optional[torch.Tensor]


def norm_rotate_backward(dq_out, dk_out, q, k, positions, freqs, *, q_weight=None, k_weight=None,
                         eps=1e-6, interleaved=False, workspace=None,
                         stream=None) -> NormRotateGrads:
    """Gradients of norm_rotate from those of its outputs (their rows may lie apart; dk_out None
    without k), with the inputs of the forward call. Sums over rows are the same in every call."""
    device = _gpu(q, "q", "norm_rotate_backward")
    lead, desc = _inputs(q, k, positions, freqs, q_weight, k_weight, eps, interleaved, device)
    desc.dq_stride = _rows(dq_out, "dq_out", lead, tuple(q.shape[-2:]), q.dtype, device)
    if (k is None) != (dk_out is None):
        raise ValueError("dk_out belongs to k")
    if k is not None:
        desc.dk_stride = _rows(dk_out, "dk_out", lead, tuple(k.shape[-2:]), q.dtype, device)
    with _Launch(device, stream) as on:
        mine = []
        dq = _made(None, "", q, mine)
        dk = None if k is None else _made(None, "", k, mine)
        dw = [None if w is None else _made(None, "", w, mine) for w in (q_weight, k_weight)]
        ws, size = _workspace(workspace, _lib().axon_norm_rotate_backward_workspace_bytes(desc), q, mine)
        on.keep(mine)
        st = _lib().axon_norm_rotate_backward(
            desc, dq_out.data_ptr(), _ptr(dk_out), q.data_ptr(), _ptr(k), positions.data_ptr(),
            freqs.data_ptr(), _ptr(q_weight), _ptr(k_weight), dq.data_ptr(), _ptr(dk), _ptr(dw[0]),
            _ptr(dw[1]), ws, size, _handle(device, stream))
    if st != _abi.AXON_OK:
        raise AxonError(st, "axon_norm_rotate_backward")
    return NormRotateGrads(dq, dk, *dw)


__all__ = ["NormRotateGrads", "norm_rotate", "norm_rotate_backward"]
