"""Decays of 1e-7 to 1e-6 a token on the GPU: states and their gradients over scans of a few tokens that
continue one another, and over long sequences, against 64 bits with the bounds of slow_decay_ref.py (which the
rounding of a, once a token, exceeds); a scan of one token against the step."""
from __future__ import annotations

import pytest

from gpu_util import say

torch = pytest.importorskip("torch")

import slow_decay_ref as slow  # noqa: E402
from test_gpu_linear import T, _axon, _gpu, make, states  # noqa: E402,F401

pytestmark = pytest.mark.gpu
E = 32


def still(lead, act, seed=0):
    """Inputs of zeros, gates of 1/2: only the decay acts. Its log in 64 bits."""
    A_log, log_a = slow.rates(E, seed=seed)
    zeros = torch.zeros(*lead, E, dtype=T[act], device="cuda")
    return dict(x=zeros, dt_raw=zeros.clone(), A_log=A_log.cuda()), log_a


def first(n, seed=3):
    return 1 + torch.rand(n, E, generator=torch.Generator().manual_seed(seed))


def held(got, want, bound, what):
    off = (got.double().cpu() - want).abs()
    assert bool((off <= bound).all()), f"{what}: {float((off / bound).max()):.2f} times the bound"


CHAINS = [(8, 400), (16, 300), (40, 100), (64, 100)]


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("scale", ["sqrt", "none"])
@pytest.mark.parametrize("tokens,calls", CHAINS)
def test_states_of_short_scans(tokens, calls, scale, act):
    say(f"[slow] {calls} scans of {tokens} {scale} {act}")
    axon = _axon()
    z, log_a = still((2, tokens), act)
    s0 = first(2)
    state = s0.cuda()
    for _ in range(calls):
        y, _ = axon.linear_scan(**z, input_scale=scale, state_in=state, state_out=state)
    torch.cuda.synchronize()
    want = s0.double() * torch.exp(log_a * tokens * calls)
    held(state, want, calls * slow.hand_overs(tokens, 16, 192) * slow.HAND_OVER * s0.double(), "state")
    # what a scan says last is the state that it hands back
    assert torch.equal(y[:, -1], state.to(y.dtype))


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("tokens,calls", CHAINS)
def test_gradients_of_short_scans(tokens, calls, act):
    say(f"[slow] {calls} backward scans of {tokens} {act}")
    axon = _axon()
    z, log_a = still((2, tokens), act)
    points = torch.zeros_like(axon.linear_checkpoints(z["x"]))
    d0 = first(2)
    d = d0.cuda()
    for _ in range(calls):
        d = axon.linear_scan_backward(z["x"], **z, checkpoints=points, dstate_out=d).dstate_in
    torch.cuda.synchronize()
    want = d0.double() * torch.exp(log_a * tokens * calls)
    wave = 8 if act == "f32" else 16
    held(d, want, calls * slow.hand_overs(tokens, wave, 64) * slow.HAND_OVER * d0.double(), "dstate_in")


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("lengths", [[3000], [7001], [100, 2500, 0, 1, 900]])
def test_long_sequences(lengths, act):
    """States, outputs, checkpoints and gradients along sequences of many tiles."""
    say(f"[slow] {lengths} {act}")
    axon = _axon()
    total, n = sum(lengths), len(lengths)
    z, log_a = still((total,), act, seed=1)
    tables = axon.sequence_tables(torch.tensor(lengths, dtype=torch.int32).cuda(), total)
    points = axon.linear_checkpoints(z["x"], tables=tables)
    s0, d0 = first(n), first(n, 4)
    y, s1 = axon.linear_scan(**z, tables=tables, state_in=s0.cuda(), checkpoints=points)
    d = axon.linear_scan_backward(z["x"], **z, tables=tables, checkpoints=points, dstate_out=d0.cuda())
    torch.cuda.synchronize()
    wave = 8 if act == "f32" else 16
    at, block = 0, 0
    for j, length in enumerate(lengths):
        s = s0[j].double()
        forward = slow.hand_overs(length, 16, 192) * slow.HAND_OVER * s
        held(s1[j], s * torch.exp(log_a * length), forward, f"state {j}")
        held(d.dstate_in[j], d0[j].double() * torch.exp(log_a * length),
             slow.hand_overs(length, wave, 64) * slow.HAND_OVER * d0[j].double(), f"dstate_in {j}")
        steps = torch.arange(1, length + 1, dtype=torch.float64)[:, None]
        want = s * torch.exp(log_a * steps)
        # 16 products with a besides, which end with the wave: a is the exponential instruction's, exact to
        # one unit in the last place (u below 1), and each product rounds, u
        near = ((steps / 16).ceil() + 3) * slow.HAND_OVER * s + 32 * slow.U * s
        if act == "bf16":
            near = near + 2.0 ** -8 * want
        held(y[at:at + length], want, near, f"y {j}")
        for k in range(-(-length // 64)):
            held(points[block + k], s * torch.exp(log_a * 64 * k),
                 (4 * k + 3) * slow.HAND_OVER * s, f"checkpoint {k} of {j}")
        at, block = at + length, block + -(-length // 64)


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("scale", ["sqrt", "complement", "none"])
@pytest.mark.parametrize("gate", ["sigmoid", "softplus"])
@pytest.mark.parametrize("rate", [(-17.0, -13.0), (-3.0, 2.0)])
def test_one_token_is_a_step(rate, gate, scale, act):
    """The scan's state behind one token is the step's, bit for bit: both advance it in the same way."""
    axon = _axon()
    n, width = 40, 200
    z = make((n,), width, act, seed=5, rate=rate, bias=False)
    s0 = 1e3 * states(n, width)
    lead = {k: None if v is None else v[:, None] if v.dim() == 2 else v for k, v in z.items()}
    y, s1 = axon.linear_scan(**lead, gate=gate, input_scale=scale, state_in=s0)
    pool = s0.clone()
    y2 = axon.linear_step(**z, state=pool, gate=gate, input_scale=scale)
    torch.cuda.synchronize()
    assert torch.equal(s1, pool) and torch.equal(y[:, 0], y2)
