"""Torch-tensor front end of the gated delta rule, the tables of packed sequences and the group
norm: argument marshalling only, as in api.py."""
from __future__ import annotations

import contextlib
import math

import torch

from . import _abi
from ._abi import AxonError
from .api import _act_dtype, _check, _keep_for, _stream_handle

DELTA_CHUNK = 64
_NOTHING = contextlib.nullcontext()
# A decode step's kernels take a few microseconds, so what is looked up on every call is kept short:
# the current stream's handle without a Stream object around it, and one test of a good tensor before
# the checks that name what is wrong with a bad one.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _on(device):
    """Kernels are launched with the tensors' device as the current one."""
    if device.index == torch.cuda.current_device():
        return _NOTHING
    return torch.cuda.device(device)


def _handle(device, stream):
    if stream is None and _raw_stream is not None:
        return _raw_stream(device.index)
    return _stream_handle(device, stream)


def _dense(t, name, shape, dtype, device):
    if not (isinstance(t, torch.Tensor) and t.shape == shape and t.dtype == dtype
            and t.device == device and t.is_contiguous()):
        _check(t, name, shape, dtype, device)


def _lib():
    return _abi._lib or _abi.load()


def _gpu(t, name, what):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{what} runs on the GPU only; {name} is on {t.device}")
    return t.device


def _row_stride(t, name, tail):
    """Elements between the rows of t, whose last len(tail) axes hold a row: 0 where t is
    contiguous, else the one stride that all leading axes agree on."""
    if t.is_contiguous():
        return 0
    want = 1
    for axis in range(1, len(tail) + 1):
        if t.shape[-axis] > 1 and t.stride(-axis) != want:
            raise ValueError(f"{name}: a row must lie contiguous in memory")
        want *= t.shape[-axis]
    stride = 0
    for axis in range(t.dim() - len(tail) - 1, -1, -1):
        if t.shape[axis] == 1:
            continue
        if t.stride(axis) < 1:
            raise ValueError(f"{name}: rows overlap (an expanded tensor)")
        if stride == 0:
            stride = step = t.stride(axis)
        elif t.stride(axis) != step:
            raise ValueError(f"{name}: the rows must be evenly spaced")
        step *= t.shape[axis]
    if stride and stride < want:
        raise ValueError(f"{name}: rows overlap (stride {stride})")
    return stride


def _rows(t, name, lead, tail, dtype, device):
    """Check t of shape lead + tail, whose rows may lie apart; returns the stride (0 = dense)."""
    shape = lead + tail
    if (isinstance(t, torch.Tensor) and t.shape == shape and t.dtype == dtype
            and t.device == device):
        return 0 if t.is_contiguous() else _row_stride(t, name, tail)
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {shape}")


class SequenceTables:
    """Tables of packed sequences (axon_sequence_tables): ``starts`` and ``block_starts``
    (sequences + 1), ``block_seq`` and ``block_first`` (total_tokens // block + sequences), int32
    parts of the one tensor ``buffer``."""

    __slots__ = ("buffer", "sequences", "total_tokens", "block", "_parts")

    def __init__(self, buffer, sequences, total_tokens, block):
        self.buffer = buffer
        self.sequences, self.total_tokens, self.block = sequences, total_tokens, block
        self._parts = None

    def _part(self, index):
        if self._parts is None:
            rows = self.total_tokens // self.block + self.sequences
            self._parts = self.buffer.split_with_sizes(
                [self.sequences + 1, self.sequences + 1, rows, rows])
        return self._parts[index]

    starts = property(lambda self: self._part(0))
    block_starts = property(lambda self: self._part(1))
    block_seq = property(lambda self: self._part(2))
    block_first = property(lambda self: self._part(3))


def sequence_tables(lengths, total_tokens, *, block=DELTA_CHUNK, stream=None) -> SequenceTables:
    """Where packed sequences and their blocks of ``block`` tokens begin, from the request lengths
    on the GPU: lengths (N,) int32; ``total_tokens`` the rows of the packed buffer. One kernel, no
    host synchronisation; a captured graph may replay it with other lengths."""
    device = _gpu(lengths, "lengths", "sequence_tables")
    if lengths.dim() != 1:
        raise ValueError("lengths must be (sequences,)")
    n = lengths.shape[0]
    _dense(lengths, "lengths", (n,), torch.int32, device)
    total_tokens, block = int(total_tokens), int(block)
    count = _lib().axon_sequence_tables_count(n, total_tokens, block)
    if count == 0:
        raise ValueError(f"unsupported packed sequences: {n} sequences, {total_tokens} tokens, "
                         f"block {block}")
    with _on(device):
        buffer = torch.empty(count, dtype=torch.int32, device=device)
        _keep_for(device, stream, buffer)
        st = _lib().axon_sequence_tables(n, total_tokens, block, lengths.data_ptr(),
                                         buffer.data_ptr(), _handle(device, stream))
    if st != _abi.AXON_OK:
        raise AxonError(st, "axon_sequence_tables")
    return SequenceTables(buffer, n, total_tokens, block)


def _delta_inputs(q, k, v, dt_raw, beta_raw, A_log, dt_bias, lead, device):
    """Checks of the tensors both forms share; the shape struct without sequences and slots."""
    bf16 = _act_dtype(q)
    hk, K = q.shape[-2:]
    hv, V = v.shape[-2:]
    qs = _rows(q, "q", lead, (hk, K), q.dtype, device)
    ks = _rows(k, "k", lead, (hk, K), q.dtype, device)
    vs = _rows(v, "v", lead, (hv, V), q.dtype, device)
    for t, n in ((dt_raw, "dt_raw"), (beta_raw, "beta_raw")):
        _dense(t, n, lead + (hv,), q.dtype, device)
    for t, n in ((A_log, "A_log"), (dt_bias, "dt_bias")):
        _dense(t, n, (hv,), torch.float32, device)
    return _abi.GatedDeltaShape(1, math.prod(lead), hk, hv, K, V, qs, ks, vs, 0, 0,
                                _abi.AXON_BF16 if bf16 else _abi.AXON_F32)


def _delta_params(A_log, dt_bias, dt_min, dt_max, scale, eps, K):
    return _abi.GatedDeltaParams(A_log.data_ptr(), dt_bias.data_ptr(), float(dt_min), float(dt_max),
                                 K ** -0.5 if scale is None else float(scale), float(eps))


def _slots(t, name, n, device):
    if t is None:
        return None
    _dense(t, name, (n,), torch.int32, device)
    return t.data_ptr()


def _pool(t, name, shape, device):
    """Check a pool of states (any number, *shape); returns how many it holds."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != 4:
        raise ValueError(f"{name} must be (states, {', '.join(map(str, shape))})")
    _dense(t, name, (t.shape[0], *shape), torch.float32, device)
    return t.shape[0]


def _ptr(t):
    return None if t is None else t.data_ptr()


def gated_delta_workspace_bytes(sequences: int, tokens: int, key_heads: int, value_heads: int,
                                key_dim: int = 128, value_dim: int = 128,
                                bf16: bool = False) -> int:
    """Device workspace bytes axon_gated_delta_scan needs (tokens: of all sequences)."""
    return _abi.gated_delta_workspace_bytes(_abi.GatedDeltaShape(
        sequences, tokens, key_heads, value_heads, key_dim, value_dim, 0, 0, 0, 0, 0,
        _abi.AXON_BF16 if bf16 else _abi.AXON_F32))


def gated_delta_scan(q, k, v, dt_raw, beta_raw, A_log, dt_bias, *, dt_min=1e-4, dt_max=100.0,
                     scale=None, eps=1e-6, lengths=None, tables=None, state_in=None, in_slots=None,
                     y=None, state_out=None, out_slots=None, workspace=None, stream=None):
    """The gated delta rule over whole sequences on the GPU (axon_gated_delta_scan).

    A uniform batch: q, k (B, L, Hk, K), v (B, L, Hv, V), dt_raw, beta_raw (B, L, Hv). Packed
    sequences: the same without the batch axis, (T, ...), with ``lengths`` (N,) int32 on the GPU, or
    ``tables`` = sequence_tables(lengths, T) built once for many layers. float32 or bfloat16, all the
    same; the rows of q, k, v may lie apart (parts of one projection, each 16-byte aligned, strides a
    multiple of 8 elements). A_log, dt_bias (Hv,) float32.
    K is 64 or 128, V a multiple of 16 up to 256, Hv a multiple of Hk; ``scale`` defaults to
    K ** -0.5.
    States are float32 (N, Hv, V, K). ``state_in`` None starts from zeros; ``in_slots`` /
    ``out_slots`` (N,) int32 address pools of states (a slot outside the pool: zeros / not stored).
    ``state_out`` may be ``state_in``. Returns (y, state_out); y has v's shape. Rows behind the last
    packed sequence are zeros in a y made here, and left as they were in a given one. Asynchronous on
    ``stream`` (default: torch's current stream)."""
    device = _gpu(q, "q", "gated_delta_scan")
    packed = lengths is not None or tables is not None
    if q.dim() != (3 if packed else 4) or v.dim() != q.dim():
        raise ValueError("q, k, v must be (tokens, heads, dim) for packed sequences (with lengths "
                         "or tables), else (batch, seqlen, heads, dim)")
    lead = tuple(q.shape[:-2])
    shape = _delta_inputs(q, k, v, dt_raw, beta_raw, A_log, dt_bias, lead, device)
    if tables is not None:
        if lengths is not None:
            raise ValueError("give lengths or tables, not both")
        if not isinstance(tables, SequenceTables):
            raise TypeError("tables must come from sequence_tables")
        if tables.block != DELTA_CHUNK or tables.total_tokens != lead[0]:
            raise ValueError(f"tables are for {tables.total_tokens} tokens in blocks of "
                             f"{tables.block}, expected {lead[0]} in blocks of {DELTA_CHUNK}")
        n = tables.sequences
        _dense(tables.buffer, "tables.buffer", (2 * (2 * n + 1 + lead[0] // DELTA_CHUNK),), torch.int32,
               device)
    elif lengths is not None:
        if not isinstance(lengths, torch.Tensor) or lengths.device != device:
            raise ValueError(f"lengths must be a tensor on {device}")
        tables = sequence_tables(lengths, lead[0], stream=stream)
        n = tables.sequences
    else:
        n = lead[0]
    shape.sequences = n
    K, hv, V = shape.key_dim, shape.value_heads, shape.value_dim
    if state_in is not None:
        shape.state_slots = _pool(state_in, "state_in", (hv, V, K), device)
    with _on(device):
        # The tables' buffer is the binding's too, on whatever stream they were built.
        mine = [] if tables is None else [tables.buffer]
        own_y = y is None
        if own_y:
            y = torch.empty(v.shape, dtype=v.dtype, device=device)
            mine.append(y)
        else:
            _dense(y, "y", v.shape, v.dtype, device)
        if state_out is None:
            if out_slots is not None:
                raise ValueError("out_slots address a pool: give state_out")
            state_out = torch.empty((n, hv, V, K), dtype=torch.float32, device=device)
            mine.append(state_out)
        shape.out_slots = _pool(state_out, "state_out", (hv, V, K), device)
        need = _abi.gated_delta_workspace_bytes(shape)
        if workspace is None and need > 0:
            workspace = torch.empty(need, dtype=torch.uint8, device=device)
            mine.append(workspace)
        elif workspace is not None and (workspace.device != device or not workspace.is_contiguous()):
            raise ValueError(f"workspace must be a contiguous tensor on {device}")
        _keep_for(device, stream, *mine)
        st = _lib().axon_gated_delta_scan(
            shape, _delta_params(A_log, dt_bias, dt_min, dt_max, scale, eps, K), q.data_ptr(),
            k.data_ptr(), v.data_ptr(), dt_raw.data_ptr(), beta_raw.data_ptr(),
            tables.buffer.data_ptr() if tables is not None else None, _ptr(state_in),
            _slots(in_slots, "in_slots", n, device), y.data_ptr(), state_out.data_ptr(),
            _slots(out_slots, "out_slots", n, device), _ptr(workspace),
            workspace.numel() * workspace.element_size() if workspace is not None else 0,
            _handle(device, stream))
        if st == _abi.AXON_OK and own_y and packed:
            st = _lib().axon_clear_behind_sequences(n, lead[0], hv * V * y.element_size(),
                                                    tables.buffer.data_ptr(), y.data_ptr(),
                                                    _handle(device, stream))
    if st != _abi.AXON_OK:
        raise AxonError(st, "axon_gated_delta_scan")
    return y, state_out


def gated_delta_step(q, k, v, dt_raw, beta_raw, A_log, dt_bias, state, *, slots=None, dt_min=1e-4,
                     dt_max=100.0, scale=None, eps=1e-6, y=None, stream=None):
    """One token for each of B rows: q, k (B, Hk, K), v (B, Hv, V), dt_raw, beta_raw (B, Hv); the
    states (pool, Hv, V, K) float32 are updated in place, row b's at ``slots[b]`` (int32; default
    b). A row whose slot lies outside the pool is idle: a given y stays as it was there, one made here
    is zero. Returns y (B, Hv, V)."""
    device = _gpu(q, "q", "gated_delta_step")
    if q.dim() != 3 or v.dim() != 3:
        raise ValueError("q, k, v must be (batch, heads, dim)")
    n = q.shape[0]
    shape = _delta_inputs(q, k, v, dt_raw, beta_raw, A_log, dt_bias, (n,), device)
    shape.sequences = n
    K = shape.key_dim
    shape.state_slots = _pool(state, "state", (shape.value_heads, shape.value_dim, K), device)
    with _on(device):
        if y is None:
            y = torch.empty(v.shape, dtype=v.dtype, device=device)
            _keep_for(device, stream, y)
            if slots is not None:  # rows may be idle
                with _NOTHING if stream is None else torch.cuda.stream(stream):
                    y.zero_()
        else:
            _dense(y, "y", v.shape, v.dtype, device)
        st = _lib().axon_gated_delta_step(
            shape, _delta_params(A_log, dt_bias, dt_min, dt_max, scale, eps, K), q.data_ptr(),
            k.data_ptr(), v.data_ptr(), dt_raw.data_ptr(), beta_raw.data_ptr(), state.data_ptr(),
            _slots(slots, "slots", n, device), y.data_ptr(), _handle(device, stream))
    if st != _abi.AXON_OK:
        raise AxonError(st, "axon_gated_delta_step")
    return y


def group_norm(x, groups, weight=None, bias=None, z=None, *, eps=1e-5, centered=True,
               activation="none", gate=None, y=None, stream=None):
    """Group norm over the channels of each token, channels last, with activation and gate
    (axon_group_norm): x (..., C), ``groups`` groups of C / groups channels with statistics of their
    own. weight and bias are float32 (C,), or (C / groups,) shared by the groups (heads). ``centered``
    False takes no mean off. ``activation`` "none" or "silu" on the result; ``gate`` "before" (x SiLU(z)
    is normalised) or "after" (the result times SiLU(z)) with z like x ("after" is the default with
    z). The rows of x and z may lie apart. Returns y (contiguous; ``y`` may be x itself)."""
    device = _gpu(x, "x", "group_norm")
    bf16 = _act_dtype(x)
    if x.dim() < 1:
        raise ValueError("x must have a channel axis")
    C, groups = x.shape[-1], int(groups)
    if groups < 1 or C < 1 or C % groups:
        raise ValueError(f"{C} channels do not split into {groups} groups")
    lead = tuple(x.shape[:-1])
    if gate is None:
        gate = "none" if z is None else "after"
    if gate not in _abi.NORM_GATES or activation not in _abi.NORM_ACTIVATIONS:
        raise ValueError(f"unknown gate {gate!r} or activation {activation!r}")
    if (gate == "none") != (z is None):
        raise ValueError(f"gate {gate!r} and z do not go together")
    xs = _row_stride(x, "x", (C,))
    zs = _rows(z, "z", lead, (C,), x.dtype, device) if z is not None else 0
    shared = False
    for t, n in ((weight, "weight"), (bias, "bias")):
        if t is None:
            continue
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{n} must be a torch.Tensor")
        if t.numel() != C:
            shared = True
    for t, n in ((weight, "weight"), (bias, "bias")):
        if t is not None:
            _dense(t, n, (C // groups if shared else C,), torch.float32, device)
    with _on(device):
        if y is None:
            y = torch.empty(x.shape, dtype=x.dtype, device=device)
            _keep_for(device, stream, y)
        else:
            _dense(y, "y", x.shape, x.dtype, device)
        desc = _abi.GroupNormDesc(math.prod(lead), groups, C // groups, xs, zs, float(eps),
                                  _abi.AXON_BF16 if bf16 else _abi.AXON_F32, 1 if centered else 0,
                                  _abi.NORM_ACTIVATIONS[activation], _abi.NORM_GATES[gate],
                                  1 if shared else 0)
        st = _lib().axon_group_norm(desc, x.data_ptr(), _ptr(z), _ptr(weight), _ptr(bias),
                                    y.data_ptr(), _handle(device, stream))
    if st != _abi.AXON_OK:
        raise AxonError(st, "axon_group_norm")
    return y


__all__ = ["SequenceTables", "gated_delta_scan", "gated_delta_step", "gated_delta_workspace_bytes",
           "group_norm", "sequence_tables"]
