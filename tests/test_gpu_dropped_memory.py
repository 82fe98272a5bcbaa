"""Workspaces that a call makes and drops while another stream still uses them: their memory does not come back to
the caller's stream before that stream has run. Shown at the allocator: requests of the same size on the caller's
stream, while the other one is busy, get other memory (memory dropped by the caller's stream itself they do get)."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

import test_gpu_conv as conv  # noqa: E402
import test_gpu_linear as linear  # noqa: E402
import test_gpu_rotate as rotate  # noqa: E402
from test_gpu_linear import _axon, _gpu  # noqa: E402,F401

pytestmark = pytest.mark.gpu


def ranges(tensors):
    return [(t.data_ptr(), t.numel() * t.element_size()) for t in tensors]


def touches(a, b):
    return any(p < q + m and q < p + n for p, n in a for q, m in b)


def again(count):
    """Memory that the current stream gets for requests of `count` bytes."""
    held = [torch.empty(count, dtype=torch.uint8, device="cuda") for _ in range(64)]
    return ranges(held)


def _scan(stream):
    axon = _axon()
    z = linear.make((2, 700), 256, "bf16", seed=3)
    return lambda: axon.linear_scan(**z, stream=stream)


def _scan_back(stream):
    axon = _axon()
    z, dy = linear.make((2, 700), 256, "bf16", seed=3), linear.grad((2, 700), 256, "bf16")
    points = torch.zeros_like(axon.linear_checkpoints(z["x"]))
    return lambda: axon.linear_scan_backward(dy, **z, checkpoints=points, stream=stream)


def _conv_back(stream):
    axon = _axon()
    z, dy = conv.make((2, 700), 256, "f32", seed=3), conv.grad((2, 700), 256, "f32")
    return lambda: axon.causal_conv_backward(dy, **z, stream=stream)


def _rotate_back(stream):
    axon = _axon()
    z, kw = rotate.make(700, 8, 2, 128, 64, "bf16", seed=1)
    d = [torch.ones_like(z["q"]), torch.ones_like(z["k"])]
    return lambda: axon.norm_rotate_backward(*d, **z, **kw, stream=stream)


@pytest.mark.parametrize("make", [_scan, _scan_back, _conv_back, _rotate_back])
def test_a_dropped_workspace_is_not_handed_out(make, monkeypatch):
    import selective_state_space_depthwise_amd.linear as front

    made, new = [], front._new

    def watched(like, shape, dtype):
        t = new(like, shape, dtype)
        if dtype == torch.uint8:  # the workspace
            made.extend(ranges([t]))
        return t

    side = torch.cuda.Stream()
    call = make(side)
    want = call()
    torch.cuda.synchronize()
    monkeypatch.setattr(front, "_new", watched)
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)
    got = call()
    assert len(made) == 1 and made[0][1] > 0
    after = again(made[0][1])
    assert not side.query()  # the call has not run yet
    assert not touches(made, after)
    # what the caller's own stream drops comes back at once
    t = torch.empty(made[0][1], dtype=torch.uint8, device="cuda")
    dropped = ranges([t])
    del t
    assert touches(dropped, again(made[0][1]))
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
