"""The group norm of very long groups, whose values are alike so that every rounding of a running sum
goes the same way. Tolerances of test_gpu_groupnorm.py: a sum of any length counts as one of at most 42
roundings."""
from __future__ import annotations

import pytest

from gpu_util import say

torch = pytest.importorskip("torch")

import delta_ref as ref  # noqa: E402
from test_gpu_groupnorm import _axon, _check, _gpu, T  # noqa: E402,F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("centered", [False, True])
@pytest.mark.parametrize("width", [(1 << 22) + 1, 1 << 23])  # value by value, and 16 bytes a lane
def test_long_groups(width, centered, act):
    say(f"[norm long] {width} {act} centered={centered}")
    x = torch.full((2, width), 1.1, dtype=T[act])
    x[:, ::2] = 0.1
    x[1, width // 2:] *= 3
    x = x.cuda()
    y = _axon().group_norm(x, 1, eps=1e-5, centered=centered)
    torch.cuda.synchronize()
    _check(y, ref.group_norm(x, 1, None, None, None, 1e-5, centered, "none", "none"), "y")
