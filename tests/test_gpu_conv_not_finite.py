"""Values of the convolution that are not finite inside a sequence: they reach the outputs and gradients whose
formula has them, in their own channel and sequence, and nothing else."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

import test_gpu_conv as conv  # noqa: E402
from test_gpu_linear import _axon, _gpu  # noqa: E402,F401

pytestmark = pytest.mark.gpu
LENGTHS, E = [100, 2, 130, 0, 1], 72
TOTAL = sum(LENGTHS) + 4


def calls(z, dy, c0, dc, activation):
    axon = _axon()
    tables = axon.sequence_tables(torch.tensor(LENGTHS, dtype=torch.int32).cuda(), TOTAL)
    y, c1 = axon.causal_conv(**z, activation=activation, cache_in=c0, tables=tables)
    g = axon.causal_conv_backward(dy, **z, activation=activation, cache_in=c0, dcache_out=dc, tables=tables)
    torch.cuda.synchronize()
    return [t.cpu() for t in (y, c1, *g)]


def rows(mask, *ranges):
    for a, b, channel in ranges:
        mask[a:b, channel] = True
    return mask


def check(got, want, bad, what):
    assert torch.equal(~torch.isfinite(got), bad), what
    assert torch.equal(got[~bad], want[~bad]), what


# an infinite sum is infinite or NaN behind SiLU, by the sign of the tap: not compared
@pytest.mark.parametrize("activation,value", [("none", float("nan")), ("none", float("inf")), ("silu", float("nan"))])
@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_an_input(act, activation, value):
    """Rows 61 and 99 (a block's third last and the sequence's last), 231 (a sequence's last), 232 (its only one)."""
    z, dy = conv.make((TOTAL,), E, act, seed=2), conv.grad((TOTAL,), E, act)
    c0, dc = conv.caches(5, E), conv.caches(5, E, 1)
    want = calls(z, dy, c0, dc, activation)
    for row, channel in ((61, 3), (99, 5), (231, 70), (232, 71)):
        z["x"][row, channel] = value
    y, c1, dx, dw, db, dcache = calls(z, dy, c0, dc, activation)

    def none(like):
        return torch.zeros_like(like, dtype=torch.bool)

    ys = rows(none(y), (61, 65, 3), (99, 100, 5), (231, 232, 70), (232, 233, 71))
    check(y, want[0], ys, "y")
    kept = none(c1)
    kept[0, 2, 5] = kept[2, 2, 70] = kept[4, 2, 71] = True
    check(c1, want[1], kept, "caches")
    weights = none(dw)
    weights[[3, 5, 70, 71], 3] = True  # the tap of the token itself
    weights[3, :] = True               # and the others where tokens follow
    if activation == "silu":           # the token's own slope is in all of them
        weights[[5, 70, 71], :] = True
    check(dw, want[3], weights, "dconv_w")
    if activation == "none":  # the sums in front of the activation do not enter
        for got, w, what in ((dx, want[2], "dx"), (db, want[4], "dconv_b"), (dcache, want[5], "dcache_in")):
            check(got, w, none(got), what)
        return
    # the slopes of tokens 61 to 64 reach dx of the three in front of each
    check(dx, want[2], rows(none(dx), (58, 65, 3), (96, 100, 5), (228, 232, 70), (232, 233, 71)), "dx")
    biases = none(db)
    biases[[3, 5, 70, 71]] = True
    check(db, want[4], biases, "dconv_b")
    first = none(dcache)
    first[4, :, 71] = True  # a sequence of one token: all that its cache feeds
    check(dcache, want[5], first, "dcache_in")


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_a_gradient(act, value):
    z, dy = conv.make((TOTAL,), E, act, seed=2), conv.grad((TOTAL,), E, act)
    c0, dc = conv.caches(5, E), conv.caches(5, E, 1)
    want = calls(z, dy, c0, dc, "silu")
    for row, channel in ((64, 3), (1, 5), (102, 70)):
        dy[row, channel] = value
    dc[1, 2, 40] = value
    y, c1, dx, dw, db, dcache = calls(z, dy, c0, dc, "silu")
    assert torch.equal(y, want[0]) and torch.equal(c1, want[1])
    bad = rows(torch.zeros_like(dx, dtype=torch.bool), (61, 65, 3), (0, 2, 5), (102, 103, 70), (101, 102, 40))
    check(dx, want[2], bad, "dx")
    first = torch.zeros_like(dcache, dtype=torch.bool)
    first[0, 1:, 5] = True       # token 1 reads the last two of its cache
    first[2, :, 70] = True       # token 0 all of it
    check(dcache, want[5], first, "dcache_in")
    weights = torch.zeros_like(dw, dtype=torch.bool)
    weights[[3, 5, 70]] = True
    check(dw, want[3], weights, "dconv_w")
    check(db, want[4], weights[:, 0], "dconv_b")


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_a_step(act):
    axon = _axon()
    z, pool = conv.make((3,), E, act, seed=2), conv.caches(4, E)
    want_pool = pool.clone()
    want = axon.causal_conv_step(**z, cache=want_pool)
    z["x"][1, 7] = float("nan")
    pool[2, 0, 9] = float("inf")
    y = axon.causal_conv_step(**z, cache=pool)
    torch.cuda.synchronize()
    check(y.cpu(), want.cpu(), rows(torch.zeros(3, E, dtype=torch.bool), (1, 2, 7), (2, 3, 9)), "y")
    bad = torch.zeros(4, 3, E, dtype=torch.bool)
    bad[1, 2, 7] = True
    check(pool.cpu(), want_pool.cpu(), bad, "caches")
