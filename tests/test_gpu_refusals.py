"""What the recurrence, the convolution, the head norm and their steps refuse, each with its own error: a wrong type
or shape before anything is asked of the library (TypeError, ValueError), what the library itself refuses with its
status (AxonError)."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

from test_gpu_linear import _axon, _gpu, grad, make, states  # noqa: E402,F401

pytestmark = pytest.mark.gpu
BAD, SMALL, UNSUPPORTED = 1, 3, 2


def ints(*v):
    return torch.tensor(v, dtype=torch.int32).cuda()


def refused(call, args, change, error):
    """error: an exception's type, or the status of an AxonError."""
    axon = _axon()
    if isinstance(error, int):
        with pytest.raises(axon.AxonError) as caught:
            call(**{**args, **change})
        assert caught.value.status == error
    else:
        with pytest.raises(error):
            call(**{**args, **change})


def bytes_of(n):
    return torch.zeros(n, dtype=torch.uint8, device="cuda")


def test_linear_scan():
    axon = _axon()
    z = dict(**make((2, 700), 24, seed=1), state_in=states(2, 24))
    axon.linear_scan(**z)
    pool = states(3, 24)
    for change, error in (
            (dict(state_in=states(1, 24)), BAD), (dict(state_out=states(1, 24)), BAD), (dict(y=z["x"]), BAD),
            (dict(y=z["dt_raw"]), BAD), (dict(workspace=bytes_of(8)), SMALL),
            (dict(state_in=pool[:2], state_out=pool[1:]), BAD), (dict(checkpoints=z["x"][0, :22]), BAD),
            (dict(checkpoints=z["x"][0, :21]), ValueError), (dict(stream=7.5), AttributeError),
            (dict(in_slots=ints(0, 1).long()), TypeError), (dict(in_slots=ints(0)), ValueError),
            (dict(x=z["x"].half(), dt_raw=z["dt_raw"].half(), in_raw=z["in_raw"].half()), TypeError),
            (dict(workspace=torch.zeros(1 << 16, dtype=torch.uint8)), ValueError)):
        refused(axon.linear_scan, z, change, error)


def test_linear_backward():
    axon = _axon()
    z = make((2, 70), 24, seed=1)
    dy = grad((2, 70), 24, "f32")
    z.update(dy=dy, checkpoints=torch.zeros_like(axon.linear_checkpoints(z["x"])))
    p = z["checkpoints"]
    axon.linear_scan_backward(**z)
    for change, error in (
            (dict(checkpoints=p[:-1]), ValueError), (dict(checkpoints=p.double()), TypeError),
            (dict(dstate_out=states(3, 24)), ValueError), (dict(dstate_out=states(2, 24).cpu()), ValueError),
            (dict(dy=dy[:, :-1]), ValueError), (dict(dy=dy.bfloat16()), TypeError), (dict(dy=dy.cpu()), ValueError),
            (dict(dy=dy[:1].expand(2, 70, 24)), ValueError), (dict(workspace=bytes_of(16)), SMALL),
            (dict(in_raw=None), ValueError)):
        refused(axon.linear_scan_backward, z, change, error)


def test_linear_step():
    axon = _axon()
    z = {k: v[:, 0].contiguous() if v.dim() == 3 else v for k, v in make((2, 70), 24, seed=1).items()}
    pool = states(5, 24)
    z["state"] = pool
    axon.linear_step(**z)
    for change, error in (
            (dict(state=pool[:1]), BAD), (dict(state=pool.bfloat16()), TypeError), (dict(state=pool[:, :-1]), ValueError),
            (dict(slots=ints(0, 1, 2)), ValueError), (dict(slots=ints(0, 1).long()), TypeError),
            (dict(y=torch.zeros(2, 24)), ValueError), (dict(x=z["x"][None]), ValueError), (dict(y=pool[:2]), BAD),
            (dict(y=z["x"]), BAD)):
        refused(axon.linear_step, z, change, error)


def test_causal_conv():
    axon = _axon()
    x, w = make((2, 30), 24, seed=1)["x"], torch.zeros(24, 4, device="cuda")
    b, cache = torch.zeros(24, device="cuda"), torch.zeros(2, 3, 24, device="cuda")
    z = dict(x=x, conv_w=w, conv_b=b, cache_in=cache)
    axon.causal_conv(**z)
    for change, error in (
            (dict(conv_w=w[:, :3]), ValueError), (dict(conv_w=torch.zeros(4, 24, device="cuda").t()), ValueError),
            (dict(conv_w=w.bfloat16()), TypeError), (dict(conv_b=b[:-1]), ValueError), (dict(activation="relu"), ValueError),
            (dict(cache_in=cache[:, :2]), ValueError), (dict(cache_in=cache[:1]), BAD), (dict(y=x), BAD),
            (dict(cache_out=cache[:1]), BAD), (dict(x=x.double()), TypeError), (dict(out_slots=ints(0, 0)), ValueError),
            (dict(cache_in=torch.zeros(3, 3, 24, device="cuda")[:2], cache_out=cache[:2].double()), TypeError)):
        refused(axon.causal_conv, z, change, error)
    z = dict(dy=x, x=x, conv_w=w, conv_b=b)
    axon.causal_conv_backward(**z)
    for change, error in (
            (dict(dy=x[:, 1:]), ValueError), (dict(dy=x.bfloat16()), TypeError), (dict(cache_in=cache[:1]), ValueError),
            (dict(dcache_out=cache[:1]), ValueError), (dict(workspace=bytes_of(1)), SMALL)):
        refused(axon.causal_conv_backward, z, change, error)
    z = dict(x=x[:, 0].contiguous(), conv_w=w, conv_b=b, cache=cache)
    axon.causal_conv_step(**z)
    for change, error in (
            (dict(cache=cache[:1]), BAD), (dict(x=x), ValueError), (dict(slots=ints(0)), ValueError),
            (dict(slots=ints(0, 1).long()), TypeError), (dict(y=z["x"]), BAD), (dict(cache=cache.bfloat16()), TypeError)):
        refused(axon.causal_conv_step, z, change, error)


def test_norm_rotate():
    axon = _axon()
    q, k = torch.zeros(9, 4, 16, device="cuda"), torch.zeros(9, 2, 16, device="cuda")
    positions, freqs = ints(*range(9)), torch.ones(8, dtype=torch.float64, device="cuda")
    z = dict(q=q, k=k, positions=positions, freqs=freqs, q_weight=torch.ones(16, device="cuda"))
    axon.norm_rotate(**z)
    odd, wide = torch.zeros(9, 4, 15, device="cuda"), torch.zeros(9, 4, 258, device="cuda")
    for change, error in (
            (dict(k=k[:8]), ValueError), (dict(k=k[..., :14]), ValueError), (dict(k=k.bfloat16()), TypeError),
            (dict(k=k[:, :0]), ValueError), (dict(positions=positions.long()), TypeError),
            (dict(positions=positions[:8]), ValueError), (dict(freqs=freqs.float()), TypeError),
            (dict(freqs=torch.ones(9, dtype=torch.float64, device="cuda")), BAD), (dict(freqs=freqs[:0]), BAD),
            (dict(q_weight=torch.ones(15, device="cuda")), ValueError), (dict(eps=-1.0), BAD),
            (dict(eps=float("nan")), BAD), (dict(k=None, k_weight=z["q_weight"]), ValueError),
            (dict(q_out=q[:8]), ValueError), (dict(q_out=k), ValueError), (dict(k_out=q), ValueError),
            (dict(k=None, k_out=k), ValueError),
            (dict(q=odd, k=None, q_weight=None, freqs=freqs[:7].clone()), UNSUPPORTED),
            (dict(q=wide, k=None, q_weight=None), UNSUPPORTED)):
        refused(axon.norm_rotate, z, change, error)
    z = dict(dq_out=q, dk_out=k, **z)
    axon.norm_rotate_backward(**z)
    for change, error in (
            (dict(dk_out=None), ValueError), (dict(dq_out=q.bfloat16()), TypeError), (dict(dq_out=q[:8]), ValueError),
            (dict(k=None), ValueError), (dict(workspace=bytes_of(4)), SMALL), (dict(eps=-1.0), BAD)):
        refused(axon.norm_rotate_backward, z, change, error)
