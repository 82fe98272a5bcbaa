"""The gated delta scan to the precision of its fp32 arithmetic: y and the states against the 64-bit
recurrence with bounds of the size of y, and bf16 outputs that are the rounding of such a y.

Tolerance. A state behind a chunk is the end of three sums over K or 64 products (S k, T X and the
state's own), y of two more (S q, A E), and the chunk before it has gone through its own three: eight
sums. Their operands are held to 2^-23 of the largest of a column or row (two fp16 pieces), a product
leaves out the two low pieces (2^-22 at most, 2^-24 in the mean), and accumulators are fp32. The
roundings of one sum are independent and of either sign, so that their total stays below 8 times the
largest of them, 2^-23 R with R the largest row norm of a state (keys and queries have length one, and
the writes are no larger than R allows). That is 8 * 8 * 2^-23 R for a state, times the scale for y;
older chunks are forgotten by the decays and the writes. The last rounding of an fp32 value adds
2^-24 of it, and the decays' exponents (all below 2^4 here where they matter) no more. A bf16 output
must be a rounding of a number within this bound: nearer to the exact value than half a step only
helps where the exact value lies next to a border between two bf16 numbers."""
from __future__ import annotations

import pytest

from gpu_util import say

torch = pytest.importorskip("torch")

import delta_ref as ref  # noqa: E402
from test_gpu_delta import _axon, _gpu, make, rows, state  # noqa: E402,F401

pytestmark = pytest.mark.gpu
STEP = 2.0 ** -23


def near(got, want, size, what):
    got, bf = got.detach().double().cpu(), got.dtype == torch.bfloat16
    off = 64 * STEP * size + STEP * want.abs()
    low, high = want - off, want + off
    if bf:
        low, high = (t.bfloat16().double() for t in (low, high))
    bad = ~((got >= low) & (got <= high))
    assert not bool(bad.any()), (f"{what}: {int(bad.sum())} of {bad.numel()} outside, largest error "
                                 f"{float((got - want).abs().max()):.3e}, size {size:.3e}")


CASES = [
    # (B, L, hk, hv, K, V)
    (1, 260, 2, 4, 128, 128),
    (1, 260, 2, 4, 64, 64),
    (1, 200, 1, 2, 128, 48),
    (2, 130, 1, 3, 64, 240),
    (2, 2200, 1, 2, 128, 128),   # walked in segments
    (32, 130, 8, 16, 128, 128),  # a large uniform batch
    (32, 70, 8, 16, 64, 80),
]


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("B,L,hk,hv,K,V", CASES)
def test_precision(B, L, hk, hv, K, V, act):
    say(f"[delta precision] B={B} L={L} heads {hk}/{hv} K={K} V={V} {act}")
    d = make((B, L), hk, hv, K, V, act, seed=L + V)
    s0 = state(B, hv, V, K, L)
    y, s1 = _axon().gated_delta_scan(**d, state_in=s0)
    torch.cuda.synchronize()
    for b in range(0, B, 15):
        yr, sr, big = ref.delta_tokens(s0[b], **rows(d, b))
        near(s1[b], sr, big, f"state[{b}]")
        near(y[b], yr, K ** -0.5 * big, f"y[{b}]")


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_precision_of_packed_sequences(act):
    lengths = [100, 0, 1, 64, 257, 40]
    hk, hv, K, V = 2, 4, 128, 64
    d = make((sum(lengths),), hk, hv, K, V, act, seed=17)
    y, s1 = _axon().gated_delta_scan(**d, lengths=torch.tensor(lengths, dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    at = 0
    for n, length in enumerate(lengths):
        yr, sr, big = ref.delta_tokens(torch.zeros(hv, V, K), **rows(d, slice(at, at + length)))
        near(s1[n], sr, big, f"state {n}")
        near(y[at:at + length], yr, K ** -0.5 * big, f"y of sequence {n}")
        at += length


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("K", [64, 128])
@pytest.mark.parametrize("halvings", [3.3, 6.3, 12.6, 19.7])
def test_states_that_only_decay(halvings, K, act):
    """A state that nothing is written to loses `halvings` powers of two every 576 tokens (a segment of
    this call) and is carried through the segments: errors count against what is left of it, token by
    token. Each decay's exponent is a product of rounded factors (step, rate, log2 e), each off by 2^-24
    of it and the step by twice that, all of them alike, so the bound grows by 4 * 2^-23 of the sum of
    the exponents; the products with M of every segment are sums of their own (8 * 2^-23 each, four at
    most)."""
    say(f"[delta precision] {halvings} halvings a segment, K={K} {act}")
    L, hv, V = 2200, 2, 32
    d = make((1, L), 1, hv, K, V, act, seed=5)
    d["v"].zero_()
    d["beta_raw"].fill_(-20.0)
    d["A_log"].zero_()
    d["dt_bias"].zero_()
    d["dt_raw"].fill_(float(torch.tensor(halvings * 0.6931 / 576, dtype=torch.float64).expm1().log()))
    s0 = state(1, hv, V, K, 1)
    y, s1 = _axon().gated_delta_scan(**d, state_in=s0)
    torch.cuda.synchronize()
    yr, sr, _ = ref.delta_tokens(s0[0], **rows(d, 0))
    gone = torch.log1p(torch.exp(d["dt_raw"][0, :, 0].double().cpu())).cumsum(0)
    left = float(s0[0].double().norm(dim=-1).max()) * torch.exp(-gone)
    bound = (64 + 4 * 8 + 4 * gone) * STEP * left
    off = float((s1[0].double().cpu() - sr).abs().max())
    assert off <= float(bound[-1]), f"state: {off / float(bound[-1]):.2f} times the bound"
    bound = (K ** -0.5 * bound)[:, None, None] + (2.0 ** -8 * yr.abs() if act == "bf16" else 0.0)
    off = float(((y[0].double().cpu() - yr).abs() / bound).max())
    assert off <= 1.0, f"y: {off:.2f} times the bound"


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("halvings", [135, 100000])
def test_large_values_that_are_forgotten(halvings, act):
    """One column of v is large, then one token's decay takes nearly all or all of its state away, and
    other columns grow afterwards: the first column stays finite, and no larger than what is left.
    The unit of a column holds for a chunk, here the one that begins with that decay: its writes are
    2^-135 of the unit where pieces end at 2^-25, so they are lost, and the state behind the chunk is
    the decayed one without what the later tokens take off. Either is at most 2^-halvings R long, with R
    the largest row norm before, so they differ by twice that; the decay is a subnormal fp32 number of
    14 bits, which the factor of 2.01 covers. The outputs are those of such a state."""
    L, hv, K, V = 200, 1, 128, 32
    d = make((1, L), 1, hv, K, V, act, seed=5)
    d["v"][:, :64, :, 0] *= 1e30
    d["v"][:, 64:, :, 0] = 0
    d["v"][:, 128:, :, 1:] *= 4096
    d["dt_raw"][:, 64] = 300.0  # cut to dt_max = 100
    d["A_log"].fill_(float(torch.tensor(halvings * 0.69314718 / 100).log()))
    d["dt_bias"].fill_(-30.0 if halvings > 1000 else -9.0)
    y, s1 = _axon().gated_delta_scan(**d)
    torch.cuda.synchronize()
    assert bool(torch.isfinite(y).all()) and bool(torch.isfinite(s1).all())
    column = rows({x: (t if x in ("A_log", "dt_bias") else t[0])
                   for x, t in dict(d, v=d["v"][..., :1]).items()}, slice(None))
    yr, sr, big = ref.delta_tokens(torch.zeros(hv, 1, K), **column)
    bound = 2.01 * big * 2.0 ** -halvings
    assert float((s1[0, :, :1].double().cpu() - sr).abs().max()) <= bound
    off = (y[0, 65:, :, :1].double().cpu() - yr[65:]).abs()
    assert float(off.max()) <= K ** -0.5 * bound * (1 + 2.0 ** -8)


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("what", ["q", "k", "v", "dt_raw", "beta_raw"])
@pytest.mark.parametrize("L", [200, 2300])  # whole, and in segments
def test_nan_is_not_lost(L, what, act):
    """NaN at one token: the outputs from there on and the state are NaN in its head (for q the output
    of the token alone has to be), and those before its chunk and of the other head do not change."""
    d = make((1, L), 2, 2, 64, 32, act, seed=5)
    d["A_log"][0] = -10.0  # nothing is forgotten
    y0, s0 = _axon().gated_delta_scan(**d)
    d[what][0, 70, 0] = float("nan")
    y, s1 = _axon().gated_delta_scan(**d)
    torch.cuda.synchronize()
    assert torch.equal(y[:, :, 1], y0[:, :, 1]) and torch.equal(s1[:, 1], s0[:, 1])
    assert torch.equal(y[:, :64], y0[:, :64])
    if what == "q":
        assert bool(y[0, 70, 0].isnan().all()) and torch.equal(s1, s0)
        assert torch.equal(y[:, 128:], y0[:, 128:])
    else:
        assert bool(y[0, 70:, 0].isnan().all()) and bool(s1[0, 0].isnan().all())


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("what", ["q", "k", "v", "dt_raw", "beta_raw"])
def test_nan_is_not_lost_by_a_step(what, act):
    d = make((3,), 2, 2, 64, 32, act, seed=6)
    s0, s = state(3, 2, 32, 64), state(3, 2, 32, 64)
    y0 = _axon().gated_delta_step(**d, state=s0)
    d[what][1, 0] = float("nan")
    y = _axon().gated_delta_step(**d, state=s)
    torch.cuda.synchronize()
    assert bool(y[1, 0].isnan().all())
    assert torch.equal(s, s0) if what == "q" else bool(s[1, 0].isnan().all())
    y[1, 0], s[1, 0] = y0[1, 0], s0[1, 0]
    assert torch.equal(y, y0) and torch.equal(s, s0)


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_infinite_gates_are_their_limits(act):
    """dt_raw of either infinity is dt_max or dt_min, beta_raw 1 or 0."""
    d = make((1, 100), 1, 2, 64, 32, act, seed=7)
    d["dt_raw"][:, 30], d["dt_raw"][:, 50] = float("inf"), float("-inf")
    d["beta_raw"][:, 31], d["beta_raw"][:, 51] = float("inf"), float("-inf")
    s0 = state(1, 2, 32, 64)
    y, s1 = _axon().gated_delta_scan(**d, state_in=s0, dt_max=2.0)
    one = state(1, 2, 32, 64)
    step = [_axon().gated_delta_step(**{x: (t if x in ("A_log", "dt_bias") else t[:, j].clone())
                                        for x, t in d.items()}, state=one, dt_max=2.0) for j in range(100)]
    torch.cuda.synchronize()
    yr, sr, big = ref.delta_tokens(s0[0], **rows(d, 0), dt_max=2.0)
    near(y[0], yr, 64 ** -0.5 * big, "y")
    near(torch.cat(step), yr, 64 ** -0.5 * big, "y of the steps")
    near(s1[0], sr, big, "state")
    near(one[0], sr, big, "state of the steps")
