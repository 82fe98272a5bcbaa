"""Torch-tensor front end of the gated linear recurrence and of the causal convolution: argument
marshalling only, as in api.py."""
from __future__ import annotations

import math
from typing import NamedTuple, Optional

import torch

from . import _abi
from ._abi import AxonError
from .api import D_CONV, _act_dtype
from .delta import (DELTA_CHUNK, SequenceTables, _dense, _gpu, _handle, _lib, _on, _ptr, _row_stride,
                    _rows, _slots, sequence_tables)


class _Launch:
    """Allocations and launches of one call on ``stream`` (None: torch's current stream), with the
    tensors' device as the current one. What is allocated inside comes from the memory of the stream
    that uses it, since memory freed on the caller's stream may still be in use there; ``keep`` records
    the streams that also use a tensor."""

    __slots__ = ("_device", "_stream", "_caller", "_context")

    def __init__(self, device, stream):
        if stream is not None and stream.device != device:
            raise ValueError(f"stream is on {stream.device}, expected {device}")
        self._device, self._stream, self._caller = device, stream, None

    def __enter__(self):
        if self._stream is None:
            self._context = _on(self._device)
        else:
            self._caller = torch.cuda.current_stream(self._device)
            self._context = torch.cuda.stream(self._stream)
        self._context.__enter__()
        return self

    def __exit__(self, *what):
        return self._context.__exit__(*what)

    def keep(self, made, tables=None):
        # tables may have been built from another stream's memory
        if tables is not None and (tables.owner is None or tables.owner != _handle(self._device, None)):
            tables.buffer.record_stream(torch.cuda.current_stream(self._device))
        if self._caller is not None and self._caller != self._stream:
            for t in made:
                t.record_stream(self._caller)


def _sequences(lead, lengths, tables, device, stream):
    """(number of sequences, tables or None) of a buffer with these leading axes."""
    if tables is None and lengths is None:
        return lead[0], None
    if tables is None:
        if not isinstance(lengths, torch.Tensor) or lengths.device != device:
            raise ValueError(f"lengths must be a tensor on {device}")
        with _Launch(device, stream) as on:
            tables = sequence_tables(lengths, lead[0])
            on.keep([tables.buffer])
        return tables.sequences, tables
    if lengths is not None:
        raise ValueError("give lengths or tables, not both")
    if not isinstance(tables, SequenceTables):
        raise TypeError("tables must come from sequence_tables")
    if tables.block != DELTA_CHUNK or tables.total_tokens != lead[0]:
        raise ValueError(f"tables are for {tables.total_tokens} tokens in blocks of "
                         f"{tables.block}, expected {lead[0]} in blocks of {DELTA_CHUNK}")
    n = tables.sequences
    _dense(tables.buffer, "tables.buffer", (2 * (2 * n + 1 + lead[0] // DELTA_CHUNK),),
           torch.int32, device)
    return n, tables


def _lead(x, lengths, tables):
    packed = lengths is not None or tables is not None
    if x.dim() != (2 if packed else 3):
        raise ValueError("x must be (tokens, channels) for packed sequences (with lengths or "
                         "tables), else (batch, seqlen, channels)")
    return tuple(x.shape[:-1])


def _pool(t, name, tail, device):
    """Check a pool (any number, *tail) of float32; returns how many it holds."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != 1 + len(tail):
        raise ValueError(f"{name} must be (states, {', '.join(map(str, tail))})")
    _dense(t, name, (t.shape[0], *tail), torch.float32, device)
    return t.shape[0]


def _optional(t, name, shape, dtype, device):
    if t is not None:
        _dense(t, name, shape, dtype, device)


def _new(like, shape, dtype):
    """Memory beside `like`, dense (the quickest of torch's ways to it: these calls are short)."""
    return like.new_empty(shape) if dtype == like.dtype else like.new_empty(shape, dtype=dtype)


def _workspace(workspace, need, like, mine):
    device = like.device
    if workspace is None:
        if need == 0:
            return None, 0
        workspace = _new(like, (need,), torch.uint8)
        mine.append(workspace)
    elif workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {device}")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _made(t, name, like, mine):
    """A given output like `like`, checked, or a new one."""
    if t is None:
        t = torch.empty_like(like) if like.is_contiguous() else like.new_empty(like.shape)
        mine.append(t)
    else:
        _dense(t, name, like.shape, like.dtype, like.device)
    return t


def _linear_inputs(x, dt_raw, A_log, dt_bias, in_raw, in_bias, lead, gate, input_scale, device):
    """Checks that all forms share; the shape (without sequences and slots) and the parameters."""
    bf16 = _act_dtype(x)
    if gate not in _abi.LINEAR_GATES or input_scale not in _abi.LINEAR_INPUT_SCALES:
        raise ValueError(f"unknown gate {gate!r} or input_scale {input_scale!r}")
    E = x.shape[-1]
    xs = _row_stride(x, "x", (E,))
    ds = _rows(dt_raw, "dt_raw", lead, (E,), x.dtype, device)
    if in_raw is None and in_bias is not None:
        raise ValueError("in_bias belongs to in_raw")
    ins = _rows(in_raw, "in_raw", lead, (E,), x.dtype, device) if in_raw is not None else 0
    _dense(A_log, "A_log", (E,), torch.float32, device)
    _optional(dt_bias, "dt_bias", (E,), torch.float32, device)
    _optional(in_bias, "in_bias", (E,), torch.float32, device)
    shape = _abi.LinearShape(1, math.prod(lead), E, xs, ds, ins, 0, 0, 0,
                             _abi.AXON_BF16 if bf16 else _abi.AXON_F32, _abi.LINEAR_GATES[gate],
                             _abi.LINEAR_INPUT_SCALES[input_scale], 0)
    return shape, _abi.LinearParams(A_log.data_ptr(), _ptr(dt_bias), _ptr(in_bias))


def linear_checkpoints(x, *, tables=None):
    """An empty tensor for the ``checkpoints`` of linear_scan over x: float32 (blocks of 64 tokens,
    channels); with ``tables`` for packed sequences x (T, E), else x (B, L, E)."""
    device = _gpu(x, "x", "linear_checkpoints")
    lead = _lead(x, None, tables)
    n, _ = _sequences(lead, None, tables, device, None)
    rows = _lib().axon_linear_checkpoint_rows(n, math.prod(lead), 0 if tables is None else 1)
    return _new(x, (rows, x.shape[-1]), torch.float32)


def linear_scan(x, dt_raw, A_log, dt_bias=None, in_raw=None, in_bias=None, *, gate="sigmoid",
                input_scale="sqrt", lengths=None, tables=None, state_in=None, in_slots=None, y=None,
                state_out=None, out_slots=None, checkpoints=None, workspace=None, stream=None):
    """The gated linear recurrence over whole sequences on the GPU (axon_linear_scan):
    h = a h + m u with log a = -exp(A_log) dt, dt the ``gate`` ("sigmoid" or "softplus") of dt_raw +
    dt_bias, u = x sigmoid(in_raw + in_bias) (x without in_raw), and ``input_scale`` m "sqrt"
    (sqrt(1 - a^2)), "complement" (1 - a) or "none" (1).

    A uniform batch: x, dt_raw, in_raw (B, L, E). Packed sequences: (T, E) with ``lengths`` (N,) int32
    on the GPU, or ``tables`` = sequence_tables(lengths, T) built once for many layers. float32 or
    bfloat16, all the same; the rows may lie apart (parts of one projection). A_log, dt_bias, in_bias
    (E,) float32. States are float32 (N, E); ``state_in`` None starts from zeros, ``in_slots`` /
    ``out_slots`` (N,) int32 address pools of states (a slot outside the pool: zeros / not stored), and
    ``state_out`` may be ``state_in``. ``checkpoints`` = linear_checkpoints(x) receives what
    linear_scan_backward reads. Returns (y, state_out). Rows behind the last packed sequence are zeros
    in a y made here, and left as they were in a given one. As every call here it records no autograd
    graph. Asynchronous on ``stream`` (default: torch's current stream)."""
    device = _gpu(x, "x", "linear_scan")
    lead = _lead(x, lengths, tables)
    shape, params = _linear_inputs(x, dt_raw, A_log, dt_bias, in_raw, in_bias, lead, gate,
                                   input_scale, device)
    n, tables = _sequences(lead, lengths, tables, device, stream)
    shape.sequences = n
    E = shape.channels
    if state_in is not None:
        shape.state_slots = _pool(state_in, "state_in", (E,), device)
    with _Launch(device, stream) as on:
        mine = []
        shape.clear_behind = 1 if y is None else 0
        y = _made(y, "y", x, mine)
        if state_out is None:
            if out_slots is not None:
                raise ValueError("out_slots address a pool: give state_out")
            state_out = _new(x, (n, E), torch.float32)
            mine.append(state_out)
        shape.out_slots = _pool(state_out, "state_out", (E,), device)
        if checkpoints is not None:
            rows = _lib().axon_linear_checkpoint_rows(n, shape.tokens, 0 if tables is None else 1)
            _dense(checkpoints, "checkpoints", (rows, E), torch.float32, device)
        ws, size = _workspace(workspace, _lib().axon_linear_scan_workspace_bytes(shape), x, mine)
        on.keep(mine, tables)
        st = _lib().axon_linear_scan(
            shape, params, x.data_ptr(), dt_raw.data_ptr(), _ptr(in_raw),
            None if tables is None else tables.buffer.data_ptr(), _ptr(state_in),
            _slots(in_slots, "in_slots", n, device), y.data_ptr(), state_out.data_ptr(),
            _slots(out_slots, "out_slots", n, device), _ptr(checkpoints), ws, size,
            _handle(device, stream))
    if st != _abi.AXON_OK:
        raise AxonError(st, "axon_linear_scan")
    return y, state_out


class LinearScanGrads(NamedTuple):
    """Gradients of linear_scan, like what they belong to; din_raw and din_bias None without
    in_raw."""
    dx: torch.Tensor
    ddt_raw: torch.Tensor
    dA_log: torch.Tensor
    ddt_bias: torch.Tensor
    din_raw: Optional[torch.Tensor]
    din_bias: Optional[torch.Tensor]
    dstate_in: torch.Tensor


def linear_scan_backward(dy, x, dt_raw, A_log, dt_bias=None, in_raw=None, in_bias=None, *,
                         checkpoints, gate="sigmoid", input_scale="sqrt", lengths=None, tables=None,
                         dstate_out=None, workspace=None, stream=None) -> LinearScanGrads:
    """Gradients of linear_scan from ``dy`` (like y; its rows may lie apart) and ``dstate_out`` (N, E)
    float32 (None = zeros), with the inputs of the forward call and the ``checkpoints`` that it wrote.
    dstate_in is (N, E), for the states that the sequences began with. Rows behind the last packed
    sequence get zeros. Sums over tokens are the same in every call."""
    device = _gpu(x, "x", "linear_scan_backward")
    lead = _lead(x, lengths, tables)
    shape, params = _linear_inputs(x, dt_raw, A_log, dt_bias, in_raw, in_bias, lead, gate,
                                   input_scale, device)
    E = shape.channels
    shape.dy_stride = _rows(dy, "dy", lead, (E,), x.dtype, device)
    n, tables = _sequences(lead, lengths, tables, device, stream)
    shape.sequences = n
    _optional(dstate_out, "dstate_out", (n, E), torch.float32, device)
    rows = _lib().axon_linear_checkpoint_rows(n, shape.tokens, 0 if tables is None else 1)
    _dense(checkpoints, "checkpoints", (rows, E), torch.float32, device)
    with _Launch(device, stream) as on:
        mine = []
        acts = [None if t is None else _made(None, "", x, mine) for t in (x, dt_raw, in_raw)]
        sums = _new(x, (2 if in_raw is None else 3, E), torch.float32)
        dstate_in = _new(x, (n, E), torch.float32)
        mine += [sums, dstate_in]
        ws, size = _workspace(workspace, _lib().axon_linear_scan_backward_workspace_bytes(shape), x, mine)
        on.keep(mine, tables)
        parts = [*sums.unbind(0), None]
        st = _lib().axon_linear_scan_backward(
            shape, params, dy.data_ptr(), x.data_ptr(), dt_raw.data_ptr(), _ptr(in_raw),
            None if tables is None else tables.buffer.data_ptr(), checkpoints.data_ptr(),
            _ptr(dstate_out), *map(_ptr, acts), *map(_ptr, parts[:3]), dstate_in.data_ptr(), ws, size,
            _handle(device, stream))
    if st != _abi.AXON_OK:
        raise AxonError(st, "axon_linear_scan_backward")
    return LinearScanGrads(acts[0], acts[1], parts[0], parts[1], acts[2], parts[2], dstate_in)


def linear_step(x, dt_raw, A_log, dt_bias, in_raw, in_bias, state, *, gate="sigmoid",
                input_scale="sqrt", slots=None, y=None, stream=None):
    """One token of linear_scan for each of B rows: x, dt_raw, in_raw (B, E); the states (pool, E)
    float32 are updated in place, row b's at ``slots[b]`` (int32; default b). A row whose slot lies
    outside the pool is idle: a given y stays as it was there, one made here is zero. Returns y."""
    device = _gpu(x, "x", "linear_step")
    if x.dim() != 2:
        raise ValueError("x must be (batch, channels)")
    n, E = x.shape
    shape, params = _linear_inputs(x, dt_raw, A_log, dt_bias, in_raw, in_bias, (n,), gate,
                                   input_scale, device)
    shape.sequences = n
    shape.state_slots = _pool(state, "state", (E,), device)
    with _Launch(device, stream) as on:
        y = _step_output(y, x, slots, on)
        st = _lib().axon_linear_step(shape, params, x.data_ptr(), dt_raw.data_ptr(), _ptr(in_raw),
                                     state.data_ptr(), _slots(slots, "slots", n, device),
                                     y.data_ptr(), _handle(device, stream))
    if st != _abi.AXON_OK:
        raise AxonError(st, "axon_linear_step")
    return y


def _step_output(y, x, slots, on):
    if y is not None:
        _dense(y, "y", x.shape, x.dtype, x.device)
        return y
    # rows may be idle where there are slots
    y = _new(x, x.shape, x.dtype) if slots is None else x.new_zeros(x.shape)
    on.keep([y])
    return y


def _conv_inputs(x, conv_w, conv_b, lead, activation, device):
    bf16 = _act_dtype(x)
    if activation not in _abi.CONV_ACTIVATIONS:
        raise ValueError(f"unknown activation {activation!r}")
    E = x.shape[-1]
    xs = _row_stride(x, "x", (E,))
    _dense(conv_w, "conv_w", (E, D_CONV), torch.float32, device)
    _optional(conv_b, "conv_b", (E,), torch.float32, device)
    return _abi.ConvShape(1, math.prod(lead), E, xs, 0, 0, 0,
                          _abi.AXON_BF16 if bf16 else _abi.AXON_F32,
                          _abi.CONV_ACTIVATIONS[activation], 0)


def causal_conv(x, conv_w, conv_b=None, *, activation="none", lengths=None, tables=None,
                cache_in=None, in_slots=None, y=None, cache_out=None, out_slots=None, stream=None):
    """The causal depthwise convolution (width 4) in front of a scan, over whole sequences on the GPU
    (axon_causal_conv), with ``activation`` "none" or "silu".

    A uniform batch: x (B, L, E). Packed sequences: (T, E) with ``lengths`` or ``tables`` as for
    linear_scan. float32 or bfloat16; the rows of x may lie apart. conv_w (E, 4) and conv_b (E,)
    float32. Caches are float32 (N, 3, E), the last three inputs, oldest first, as prefill's
    conv_cache; pools, slots and in-place updates as for linear_scan's states. Returns (y, cache_out).
    Rows behind the last packed sequence as for linear_scan."""
    device = _gpu(x, "x", "causal_conv")
    lead = _lead(x, lengths, tables)
    shape = _conv_inputs(x, conv_w, conv_b, lead, activation, device)
    n, tables = _sequences(lead, lengths, tables, device, stream)
    shape.sequences = n
    tail = (D_CONV - 1, shape.channels)
    if cache_in is not None:
        shape.cache_slots = _pool(cache_in, "cache_in", tail, device)
    with _Launch(device, stream) as on:
        mine = []
        shape.clear_behind = 1 if y is None else 0
        y = _made(y, "y", x, mine)
        if cache_out is None:
            if out_slots is not None:
                raise ValueError("out_slots address a pool: give cache_out")
            cache_out = _new(x, (n, *tail), torch.float32)
            mine.append(cache_out)
        shape.out_slots = _pool(cache_out, "cache_out", tail, device)
        on.keep(mine, tables)
        st = _lib().axon_causal_conv(
            shape, x.data_ptr(), conv_w.data_ptr(), _ptr(conv_b),
            None if tables is None else tables.buffer.data_ptr(), _ptr(cache_in),
            _slots(in_slots, "in_slots", n, device), y.data_ptr(), cache_out.data_ptr(),
            _slots(out_slots, "out_slots", n, device), _handle(device, stream))
    if st != _abi.AXON_OK:
        raise AxonError(st, "axon_causal_conv")
    return y, cache_out


class CausalConvGrads(NamedTuple):
    """Gradients of causal_conv, like what they belong to."""
    dx: torch.Tensor
    dconv_w: torch.Tensor
    dconv_b: torch.Tensor
    dcache_in: torch.Tensor


def causal_conv_backward(dy, x, conv_w, conv_b=None, *, activation="none", lengths=None, tables=None,
                         cache_in=None, dcache_out=None, workspace=None,
                         stream=None) -> CausalConvGrads:
    """Gradients of causal_conv from ``dy`` (like y; its rows may lie apart) and ``dcache_out``
    (N, 3, E) float32 (None = zeros), with the inputs of the forward call; ``cache_in`` (N, 3, E) is
    what the sequences began with (None = zeros). Rows behind the last packed sequence get zeros. Sums
    over tokens are the same in every call."""
    device = _gpu(x, "x", "causal_conv_backward")
    lead = _lead(x, lengths, tables)
    shape = _conv_inputs(x, conv_w, conv_b, lead, activation, device)
    E = shape.channels
    shape.dy_stride = _rows(dy, "dy", lead, (E,), x.dtype, device)
    n, tables = _sequences(lead, lengths, tables, device, stream)
    shape.sequences = n
    tail = (D_CONV - 1, E)
    _optional(cache_in, "cache_in", (n, *tail), torch.float32, device)
    _optional(dcache_out, "dcache_out", (n, *tail), torch.float32, device)
    with _Launch(device, stream) as on:
        mine = []
        dx = _made(None, "", x, mine)
        dw, db, dcache = (_new(x, t, torch.float32) for t in ((E, D_CONV), (E,), (n, *tail)))
        mine += [dw, db, dcache]
        ws, size = _workspace(workspace, _lib().axon_causal_conv_backward_workspace_bytes(shape), x, mine)
        on.keep(mine, tables)
        st = _lib().axon_causal_conv_backward(
            shape, dy.data_ptr(), x.data_ptr(), conv_w.data_ptr(), _ptr(conv_b),
            None if tables is None else tables.buffer.data_ptr(), _ptr(cache_in), _ptr(dcache_out),
            dx.data_ptr(), dw.data_ptr(), db.data_ptr(), dcache.data_ptr(), ws, size,
            _handle(device, stream))
    if st != _abi.AXON_OK:
        raise AxonError(st, "axon_causal_conv_backward")
    return CausalConvGrads(dx, dw, db, dcache)


def causal_conv_step(x, conv_w, conv_b, cache, *, activation="none", slots=None, y=None,
                     stream=None):
    """One token of causal_conv for each of B rows: x (B, E); the caches (pool, 3, E) float32 are
    updated in place, row b's at ``slots[b]`` (int32; default b). Idle rows as for linear_step.
    Returns y."""
    device = _gpu(x, "x", "causal_conv_step")
    if x.dim() != 2:
        raise ValueError("x must be (batch, channels)")
    n, E = x.shape
    shape = _conv_inputs(x, conv_w, conv_b, (n,), activation, device)
    shape.sequences = n
    shape.cache_slots = _pool(cache, "cache", (D_CONV - 1, E), device)
    with _Launch(device, stream) as on:
        y = _step_output(y, x, slots, on)
        st = _lib().axon_causal_conv_step(shape, x.data_ptr(), conv_w.data_ptr(), _ptr(conv_b),
                                          cache.data_ptr(), _slots(slots, "slots", n, device),
                                          y.data_ptr(), _handle(device, stream))
    if st != _abi.AXON_OK:
        raise AxonError(st, "axon_causal_conv_step")
    return y


__all__ = ["CausalConvGrads", "LinearScanGrads", "causal_conv", "causal_conv_backward",
           "causal_conv_step", "linear_checkpoints", "linear_scan", "linear_scan_backward",
           "linear_step"]
