"""Rows that no sequence or slot covers: zeros in an output that the call makes, untouched in a given
one; and the call that clears them."""
from __future__ import annotations

import pytest

from gpu_util import say

torch = pytest.importorskip("torch")

from test_gpu_delta import T, _axon, _gpu, make, state  # noqa: E402,F401

pytestmark = pytest.mark.gpu


def poison(shape, dtype):
    """Leaves memory of this size behind, full of NaN, for the next allocation to find."""
    torch.full(shape, float("nan"), dtype=dtype, device="cuda")
    torch.cuda.synchronize()


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("lengths,spare", [([70, 0, 30], 45), ([65], 62), ([0, 0], 9), ([64], 0),
                                           ([3], 4000)])
@pytest.mark.parametrize("side", [False, True])
def test_scan_clears_what_it_makes(lengths, spare, act, side):
    say(f"[delta rows] {lengths} and {spare} more, {act}, other stream {side}")
    axon = _axon()
    total = sum(lengths) + spare
    d = make((total,), 1, 2, 64, 48, act, seed=total)
    n = torch.tensor(lengths, dtype=torch.int32).cuda()
    given = torch.full((total, 2, 48), 7.0, dtype=T[act]).cuda()
    axon.gated_delta_scan(**d, lengths=n, y=given)
    torch.cuda.synchronize()
    poison(given.shape, given.dtype)
    stream = torch.cuda.Stream() if side else None
    for kw in (dict(lengths=n), dict(tables=axon.sequence_tables(n, total))):
        torch.cuda.synchronize()
        y, _ = axon.gated_delta_scan(**d, **kw, stream=stream)
        torch.cuda.synchronize()
        end = sum(lengths)
        assert torch.equal(y[:end], given[:end])
        assert bool((y[end:] == 0).all()) and bool((given[end:] == 7).all())
        del y
        poison(given.shape, given.dtype)


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("side", [False, True])
def test_step_clears_what_it_makes(act, side):
    axon = _axon()
    d = make((9,), 1, 2, 64, 48, act, seed=1)
    slots = torch.tensor([3, -1, 0, 99, 5, 1, -7, 2, 4], dtype=torch.int32).cuda()
    given = torch.full((9, 2, 48), 7.0, dtype=T[act]).cuda()
    axon.gated_delta_step(**d, state=state(6, 2, 48, 64), slots=slots, y=given)
    pool = state(6, 2, 48, 64)
    poison(given.shape, given.dtype)
    stream = torch.cuda.Stream() if side else None
    y = axon.gated_delta_step(**d, state=pool, slots=slots, stream=stream)
    torch.cuda.synchronize()
    idle = torch.tensor([1, 3, 6]).cuda()
    assert bool((y[idle] == 0).all()) and bool((given[idle] == 7).all())
    given[idle] = 0
    assert torch.equal(y, given)


def test_captured():
    """The rows cleared follow the lengths of each replay."""
    axon = _axon()
    d = make((200,), 1, 2, 64, 48, "bf16", seed=2)
    n = torch.tensor([100, 60], dtype=torch.int32).cuda()
    axon.gated_delta_scan(**d, lengths=n)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, _ = axon.gated_delta_scan(**d, lengths=n)
    for lengths in ([100, 60], [200, 0], [0, 1], [64, 100]):
        n.copy_(torch.tensor(lengths, dtype=torch.int32))
        y.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        want, _ = axon.gated_delta_scan(**d, lengths=n)
        assert torch.equal(y, want) and bool((y[sum(lengths):] == 0).all())


@pytest.mark.parametrize("total,row,end", [(1, 16, 0), (5, 48, 5), (5, 48, 3), (70000, 512, 1), (9, 16, -4),
                                           (9, 16, 100), (0, 16, 0)])
def test_clear(total, row, end):
    from selective_state_space_depthwise_amd import _abi

    tables = torch.tensor([0, 0, end], dtype=torch.int32).cuda()
    x = torch.full(((total + 1) * row,), 5, dtype=torch.uint8).cuda()  # one row behind the buffer
    st = _abi.raw_clear_behind_sequences(2, total, row, tables.data_ptr(), x.data_ptr(),
                                         torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert st == 0
    first = min(max(end, 0), total) * row
    assert bool((x[:first] == 5).all()) and bool((x[first:total * row] == 0).all())
    assert bool((x[total * row:] == 5).all())


@pytest.mark.parametrize("what", ["short", "long", "type", "host", "spread", "more sequences"])
def test_refused_tables(what):
    """Tables whose buffer is not what the kernels read from are refused before any launch."""
    axon = _axon()
    d = make((100,), 1, 2, 64, 48, "f32", seed=1)
    good = axon.sequence_tables(torch.tensor([60, 40], dtype=torch.int32).cuda(), 100)
    torch.cuda.synchronize()
    b, n = good.buffer, 2
    if what == "more sequences":
        n = 3
    else:
        b = {"short": b[:-1], "long": torch.cat([b, b[:1]]), "type": b.long(), "host": b.cpu(),
             "spread": b.repeat_interleave(2)[::2]}[what]
    with pytest.raises((TypeError, ValueError)):
        axon.gated_delta_scan(**d, tables=axon.SequenceTables(b, n, 100, 64))


def test_tables_dropped_while_in_use():
    """Tables built on one stream, used on another that is behind, and dropped: their memory is not
    handed out again before the scan has read it."""
    axon = _axon()
    total, lengths = 6400, [3000, 0, 3400]
    d = make((total,), 1, 2, 64, 48, "bf16", seed=3)
    n = torch.tensor(lengths, dtype=torch.int32).cuda()
    y0, s0 = axon.gated_delta_scan(**d, lengths=n)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    tables = axon.sequence_tables(n, total)
    size = tables.buffer.numel()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    y, s = axon.gated_delta_scan(**d, tables=tables, stream=side)
    del tables
    others = [torch.full((size,), -1, dtype=torch.int32, device="cuda") for _ in range(8)]
    torch.cuda.synchronize()
    assert torch.equal(y, y0) and torch.equal(s, s0)
    assert all(bool((t == -1).all()) for t in others)
