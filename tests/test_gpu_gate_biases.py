"""Gates whose raw value and bias nearly cancel: what counts is their sum, and the bounds of the plain form are
those of the sum, whatever the size of the two."""
from __future__ import annotations

import pytest

from gpu_util import say

torch = pytest.importorskip("torch")

from test_gpu_linear import T, _axon, _gpu, compare, grad, make, sequence, states  # noqa: E402,F401

import recurrent_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu


def cancelling(lead, E, act, bias):
    """Raw values of about -bias (4000 is 125 x 32, exact in bf16), gates between sigmoid(-8) and sigmoid(8)."""
    z = make(lead, E, act, seed=11)
    for raw, name in (("dt_raw", "dt_bias"), ("in_raw", "in_bias")):
        z[raw] = (z[raw].float() - bias).to(T[act])
        z[name] = bias + 2 * z[name]
    return z


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("bias", [4000.0, -4000.0])
@pytest.mark.parametrize("gate", ["sigmoid", "softplus"])
def test_scan(gate, bias, act):
    say(f"[gates] {gate} {bias} {act}")
    axon = _axon()
    B, L, E = 2, 100, 70
    z = cancelling((B, L), E, act, bias)
    s0, ds, dy = states(B, E, 1), states(B, E, 2), grad((B, L), E, act)
    points = axon.linear_checkpoints(z["x"])
    y, s1 = axon.linear_scan(**z, gate=gate, state_in=s0, checkpoints=points)
    grads = axon.linear_scan_backward(dy, **z, gate=gate, checkpoints=points, dstate_out=ds)
    torch.cuda.synchronize()
    compare(z, list(range(B)), s0, ds, dy, y, s1, grads, gate, "sqrt")


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("gate", ["sigmoid", "softplus"])
def test_step(gate, act):
    """The step's gates, and the scan of one token with the same state bit for bit."""
    axon = _axon()
    n, E = 5, 70
    z = cancelling((n,), E, act, 4000.0)
    s0 = states(n, E)
    pool = s0.clone()
    y = axon.linear_step(**z, state=pool, gate=gate)
    lead = {k: v[:, None] if v.dim() == 2 else v for k, v in z.items()}
    y1, s1 = axon.linear_scan(**lead, gate=gate, state_in=s0)
    torch.cuda.synchronize()
    for r in range(n):
        want = sequence(z, s0[r], slice(r, r + 1), gate, "sqrt")
        ref.within(y[r:r + 1], want.y, want.bound, f"y {r}")
        ref.within(pool[r], want.state, want.state_bound, f"state {r}")
    assert torch.equal(s1, pool) and torch.equal(y1[:, 0], y)
