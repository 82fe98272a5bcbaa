"""The bound that the GPU tests of slow decays use, on float32 forms of the recurrence on the CPU: states handed on
by expm1 keep it, and states multiplied by the rounded a do not, so that the bound tells the two apart."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

import slow_decay_ref as slow  # noqa: E402


# tokens of a call, calls one behind the other
CHAINS = [(8, 400), (16, 300), (40, 100), (64, 100), (3000, 1), (7001, 1)]


@pytest.mark.parametrize("tokens,calls", CHAINS)
def test_the_bound_tells_the_forms_apart(tokens, calls):
    A_log, log_a = slow.rates(32)
    s0 = 1 + torch.rand(32, generator=torch.Generator().manual_seed(3))
    want = s0.double() * torch.exp(log_a * tokens * calls)
    bound = calls * slow.hand_overs(tokens, 16, 192) * slow.HAND_OVER * s0.double()
    h = s0
    for _ in range(calls):
        h = slow.handed_on(h, log_a, tokens)
    assert bool(((h.double() - want).abs() <= bound).all())
    off = (slow.multiplied(s0, log_a, tokens * calls).double() - want).abs()
    assert float((off / bound).max()) > 1.5


def test_a_product_at_either_end_of_a_call_is_seen():
    """A call of 40 tokens that multiplies in its first and last 16 and hands on in between."""
    A_log, log_a = slow.rates(32)
    s0 = 1 + torch.rand(32, generator=torch.Generator().manual_seed(3))
    calls = 100
    want = s0.double() * torch.exp(log_a * 40 * calls)
    bound = calls * slow.hand_overs(40, 16, 192) * slow.HAND_OVER * s0.double()
    h = s0
    for _ in range(calls):
        h = slow.multiplied(slow.handed_on(slow.multiplied(h, log_a, 16), log_a, 8), log_a, 16)
    assert float(((h.double() - want).abs() / bound).max()) > 1.5
