"""Packed batches of many short sequences: around the number up to which they start in the order of
their lengths, and far above it, where the time must not jump."""
from __future__ import annotations

import pytest

from gpu_util import say

torch = pytest.importorskip("torch")

import delta_ref as ref  # noqa: E402
from test_gpu_delta import _axon, _gpu, close, make, rows  # noqa: E402,F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [63, 64, 65, 600, 1024, 1030])
@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_many_sequences(n, act):
    say(f"[delta many] {n} sequences, {act}")
    g = torch.Generator().manual_seed(n)
    lengths = torch.randint(0, 150, (n,), generator=g) * (torch.rand(n, generator=g) > 0.2)
    lengths = (lengths if n < 100 else lengths % 70).int()
    total = int(lengths.sum()) + 5
    d = make((total,), 1, 1, 64, 16, act, seed=n)
    y, s = _axon().gated_delta_scan(**d, lengths=lengths.cuda())
    torch.cuda.synchronize()
    at = 0
    for j, length in enumerate(lengths.tolist()):
        yr, sr, big = ref.delta_tokens(torch.zeros(1, 16, 64), **rows(d, slice(at, at + length)))
        close(y[at:at + length], yr, big, f"y of sequence {j}")
        close(s[j], sr, big, f"state of sequence {j}")
        at += length


def test_time_does_not_jump():
    """1024 sequences of 32 tokens take no longer than 2 times what 1030 take (1 in the mean)."""
    axon = _axon()

    def least(n):
        d = make((32 * n,), 2, 4, 128, 128, "bf16", seed=1)
        tables = axon.sequence_tables(torch.full((n,), 32, dtype=torch.int32).cuda(), 32 * n)
        times = []
        for _ in range(6):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            axon.gated_delta_scan(**d, tables=tables)
            b.record()
            torch.cuda.synchronize()
            times.append(a.elapsed_time(b))
        return min(times[1:])

    few, many = least(1024), least(1030)
    say(f"[delta many] 1024 sequences {few * 1000:.0f} us, 1030 {many * 1000:.0f} us")
    assert few <= 2 * many
