"""The gated delta step where a wave takes several passes over its rows of the state (2048 waves and
more), with states that pass by the caches (above 16 MB) and that do not, V that ends inside a wave's
rows, and idle rows."""
from __future__ import annotations

import pytest

from gpu_util import say

torch = pytest.importorskip("torch")

import delta_ref as ref  # noqa: E402
from test_gpu_delta import T, _axon, _gpu, close, make, rows, state  # noqa: E402,F401

pytestmark = pytest.mark.gpu

CASES = [
    # (rows, heads, K, V, act)
    (32, 16, 128, 128, "bf16"),
    (32, 16, 128, 112, "bf16"),
    (64, 16, 64, 112, "bf16"),
    (64, 16, 64, 240, "f32"),
    (128, 16, 128, 16, "bf16"),  # 16 MB
    (128, 16, 64, 16, "f32"),
    (128, 16, 64, 16, "bf16"),
]


@pytest.mark.parametrize("B,hv,K,V,act", CASES)
def test_step(B, hv, K, V, act):
    say(f"[delta step] rows={B} heads={hv} K={K} V={V} {act}")
    d = make((B,), hv // 2, hv, K, V, act, seed=B + V)
    s = state(B + 2, hv, V, K, B)
    before = s.clone()
    slots = torch.randperm(B + 2, generator=torch.Generator().manual_seed(B))[:B].int()
    slots[3], slots[B - 2] = -1, B + 2
    y = torch.full((B, hv, V), 3.0, dtype=T[act]).cuda()
    _axon().gated_delta_step(**d, state=s, slots=slots.cuda(), y=y)
    torch.cuda.synchronize()
    live = [b for b in range(B) if 0 <= int(slots[b]) < B + 2]
    for b in (*live[:4], *live[B // 2:B // 2 + 2], *live[-3:]):
        i = int(slots[b])
        yr, sr, big = ref.delta_tokens(before[i], **rows(d, slice(b, b + 1)))
        close(y[b], yr[0], big, f"y[{b}]")
        close(s[i], sr, big, f"state[{i}]")
    assert bool((y[3] == 3.0).all()) and bool((y[B - 2] == 3.0).all())
    for i in set(range(B + 2)) - {int(slots[b]) for b in live}:
        assert torch.equal(s[i], before[i]), f"state {i} changed"
