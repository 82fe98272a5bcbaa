"""Tables of packed sequences against their plain form: every value has to be equal."""
from __future__ import annotations

import pytest

from gpu_util import say

torch = pytest.importorskip("torch")

import delta_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import selective_state_space_depthwise_amd as axon

    axon.load()
    yield
    torch.cuda.synchronize()


def _random(n, longest, seed, zeros=0.2):
    g = torch.Generator().manual_seed(seed)
    x = torch.randint(0, longest + 1, (n,), generator=g)
    return (x * (torch.rand(n, generator=g) > zeros)).tolist()


CASES = [
    ([0], 0, 64), ([1], 1, 64), ([7], 3, 1), ([64], 64, 64), ([65], 65, 64), ([0, 0, 0], 10, 64),
    ([3, -5, 2, 0, 9], 40, 4), ([2 ** 31 - 1, 5, 2 ** 31 - 1], 1000, 64),
    ([2 ** 31 - 1] * 300, 5000, 7), ([5000], 5000, 64), ([10, 20], 12, 64),
    (_random(256, 300, 1), 40000, 64), (_random(257, 300, 2), 40000, 100),
    (_random(4096, 20, 3), 42000, 16), (_random(4097, 20, 4), 50000, 16),
    (_random(9000, 8, 5), 30000, 3), (_random(65535, 3, 6), 99999, 64), ([100000], 200000, 1),
    ([50] * 10, 500, 2 ** 40),
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_tables(case):
    import selective_state_space_depthwise_amd as axon

    lengths, total, block = CASES[case]
    say(f"[tables] {len(lengths)} sequences, {total} rows, block {block}")
    t = axon.sequence_tables(torch.tensor(lengths, dtype=torch.int32).cuda(), total, block=block)
    torch.cuda.synchronize()
    want = ref.tables(lengths, total, block)
    for name, w in zip(("starts", "block_starts", "block_seq", "block_first"), want):
        assert getattr(t, name).tolist() == w, name


def test_refused():
    import selective_state_space_depthwise_amd as axon

    n = torch.tensor([1, 2], dtype=torch.int32).cuda()
    for bad in (n.long(), n.cpu(), n[:0], n.view(1, 2), torch.zeros(65536, dtype=torch.int32).cuda()):
        with pytest.raises((TypeError, ValueError)):
            axon.sequence_tables(bad, 10)
    for total, block in ((-1, 64), (2 ** 31, 64), (10, 0), (2 ** 31 - 1, 1)):
        with pytest.raises(ValueError):
            axon.sequence_tables(n, total, block=block)
