"""Refusals of axon_clear_behind_sequences (nothing here reaches the GPU)."""
import pytest

from selective_state_space_depthwise_amd import _abi as A

P = 0x7F0000000000
Q = P + (1 << 40)
BAD, UNS = A.AXON_ERR_INVALID_ARGUMENT, A.AXON_ERR_UNSUPPORTED


@pytest.mark.parametrize("args,status", [
    ((0, 10, 16, P, Q), BAD), ((1, -1, 16, P, Q), BAD), ((1, 10, 0, P, Q), BAD), ((1, 10, 24, P, Q), BAD),
    ((65536, 10, 16, P, Q), UNS), ((1, 1 << 31, 16, P, Q), UNS), ((1, 1 << 30, 1 << 13, P, Q), UNS),
    ((1, 10, 16, None, Q), BAD), ((1, 10, 16, P, None), BAD), ((1, 10, 16, P + 2, Q), BAD),
    ((1, 10, 16, P, Q + 8), BAD), ((1, 10, 16, Q + 64, Q), BAD), ((3, 10, 16, Q - 12, Q), BAD),
    ((1, 0, 16, None, None), A.AXON_OK),
])
def test_refused(args, status):
    assert A.raw_clear_behind_sequences(*args, None) == status
