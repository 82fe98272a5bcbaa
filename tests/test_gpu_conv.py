"""The causal depthwise convolution on the GPU against its plain 64-bit form, forward, backward and
step: sequences shorter than the taps, packed and empty ones, caches in pools and in place, parts of
one projection, streams, graphs."""
from __future__ import annotations

import pytest

from gpu_util import say

torch = pytest.importorskip("torch")

import recurrent_ref as ref  # noqa: E402
from test_gpu_linear import T, _axon, _gpu, parts_of  # noqa: E402,F401

pytestmark = pytest.mark.gpu


def make(lead, E, act="f32", seed=0, bias=True):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(*lead, E, generator=g) * 2).to(T[act]).cuda()
    w = torch.randn(E, 4, generator=g).cuda()
    return dict(x=x, conv_w=w, conv_b=torch.randn(E, generator=g).cuda() if bias else None)


def caches(n, E, seed=0):
    return torch.randn(n, 3, E, generator=torch.Generator().manual_seed(5 + seed)).cuda()


def grad(lead, E, act, seed=0):
    return torch.randn(*lead, E, generator=torch.Generator().manual_seed(3 + seed)).to(T[act]).cuda()


def compare(z, parts, c0, dc, dy, y, c1, grads, act, slots=None):
    E = y.shape[-1]
    dw = [torch.zeros(E, 4, dtype=torch.float64)] * 2
    db = [torch.zeros(E, dtype=torch.float64)] * 2
    for n, at in enumerate(parts):
        want, off, cache = ref.conv(z["x"][at], z["conv_w"], z["conv_b"], c0[n], act == "silu")
        ref.within(y[at], want, off, f"y {at}")
        if c1 is not None:
            assert torch.equal(c1[n].cpu().double(), cache), f"cache {n}"
        if grads is None:
            continue
        g = ref.conv_backward(dy[at], z["x"][at], z["conv_w"], z["conv_b"], c0[n], dc[n],
                              act == "silu")
        ref.within(grads.dx[at], *g["dx"], f"dx {at}")
        ref.within(grads.dcache_in[n], *g["dcache_in"], f"dcache_in {n}")
        dw = [a + b for a, b in zip(dw, g["dconv_w"])]
        db = [a + b for a, b in zip(db, g["dconv_b"])]
    if grads is not None:
        ref.within(grads.dconv_w, *dw, "dconv_w")
        ref.within(grads.dconv_b, *db, "dconv_b")


UNIFORM = [
    # (B, L, E, act, activation, bias)
    (1, 1, 1, "f32", "silu", True), (2, 2, 3, "bf16", "none", True), (3, 3, 64, "f32", "silu", False),
    (1, 4, 65, "bf16", "silu", True), (2, 63, 130, "f32", "none", True),
    (1, 64, 8, "bf16", "silu", True), (2, 65, 256, "f32", "silu", True),
    (2, 66, 512, "bf16", "silu", True), (1, 67, 260, "f32", "silu", False),
    (2, 200, 1000, "bf16", "silu", True), (1, 1500, 24, "f32", "silu", True),
    (1, 300, 1026, "bf16", "none", True), (2, 130, 2048, "bf16", "silu", True),
]


@pytest.mark.parametrize("B,L,E,dtype,act,bias", UNIFORM)
def test_uniform_batch(B, L, E, dtype, act, bias):
    say(f"[conv] {B} x {L} x {E} {dtype} {act}")
    axon = _axon()
    z = make((B, L), E, dtype, seed=L + E, bias=bias)
    c0, dc, dy = caches(B, E), caches(B, E, 1), grad((B, L), E, dtype)
    y, c1 = axon.causal_conv(**z, activation=act, cache_in=c0)
    grads = axon.causal_conv_backward(dy, **z, activation=act, cache_in=c0, dcache_out=dc)
    torch.cuda.synchronize()
    compare(z, list(range(B)), c0, dc, dy, y, c1, grads, act)
    y, c1 = axon.causal_conv(**z, activation=act)
    grads = axon.causal_conv_backward(dy, **z, activation=act)
    torch.cuda.synchronize()
    zero = torch.zeros(B, 3, E)
    compare(z, list(range(B)), zero, zero, dy, y, c1, grads, act)


PACKED = [([5, 0, 64, 1, 130, 65, 0, 2, 63], 37), ([1] * 30 + [2] * 20 + [3, 4], 3), ([700], 0),
          ([0, 0, 3], 200), ([64, 128, 192, 1], 1)]


@pytest.mark.parametrize("E", [40, 71, 512])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lengths,spare", PACKED)
def test_packed(lengths, spare, dtype, E):
    say(f"[conv] packed {lengths} + {spare} {dtype} {E}")
    axon = _axon()
    total, N = sum(lengths) + spare, len(lengths)
    z = make((total,), E, dtype, seed=total)
    dy = grad((total,), E, dtype)
    end = total - spare
    z["x"][end:] = float("nan")
    dy[end:] = float("nan")
    n = torch.tensor(lengths, dtype=torch.int32).cuda()
    tables = axon.sequence_tables(n, total)
    c0, dc = caches(N, E), caches(N, E, 1)
    y, c1 = axon.causal_conv(**z, activation="silu", cache_in=c0, tables=tables)
    grads = axon.causal_conv_backward(dy, **z, activation="silu", cache_in=c0, dcache_out=dc,
                                      tables=tables)
    torch.cuda.synchronize()
    compare(z, parts_of(lengths), c0, dc, dy, y, c1, grads, "silu")
    assert not y[end:].any() and not grads.dx[end:].any()
    given = torch.full_like(y, 7.0)
    axon.causal_conv(**z, activation="silu", cache_in=c0, lengths=n, y=given)
    torch.cuda.synchronize()
    assert bool((given[end:] == 7).all()) and torch.equal(given[:end], y[:end])


@pytest.mark.parametrize("place", [True, False])
def test_pools(place):
    """Caches updated in place, among them of sequences shorter than the cache."""
    axon = _axon()
    lengths, E = [70, 0, 2, 300, 1, 64], 72
    z = make((sum(lengths),), E, seed=3)
    pool = caches(9, E)
    ins = torch.tensor([4, 2, 6, 8, -1, 100], dtype=torch.int32).cuda()
    outs = torch.tensor([4, 2, 6, 8, 0, -5], dtype=torch.int32).cuda()
    out = pool.clone() if place else torch.full((7, E), 5.0).cuda()[:, None].repeat(1, 3, 1)
    if not place:
        outs = torch.tensor([6, 2, 99, 5, 0, 1], dtype=torch.int32).cuda()
    before = out.clone()
    y, got = axon.causal_conv(**z, lengths=torch.tensor(lengths, dtype=torch.int32).cuda(),
                              cache_in=out if place else pool, in_slots=ins, cache_out=out,
                              out_slots=outs)
    torch.cuda.synchronize()
    assert got is out
    touched = set()
    for n, at in enumerate(parts_of(lengths)):
        slot, to = int(ins[n]), int(outs[n])
        c0 = pool[slot] if 0 <= slot < 9 else torch.zeros(3, E)
        want, off, cache = ref.conv(z["x"][at], z["conv_w"], z["conv_b"], c0, False)
        ref.within(y[at], want, off, f"y {n}")
        if 0 <= to < out.shape[0]:
            touched.add(to)
            assert torch.equal(out[to].cpu().double(), cache)
    for j in range(out.shape[0]):
        assert j in touched or torch.equal(out[j], before[j])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("E,first,width", [(64, 0, 200), (37, 1, 99), (256, 8, 1024), (256, 4, 516)])
def test_parts_of_one_projection(dtype, E, first, width):
    axon = _axon()
    B, L = 2, 90
    z = make((B, L), E, dtype, seed=6)
    z["x"] = make((B, L), width, dtype, seed=5)["x"][..., first:first + E]
    dy = grad((B, L), 2 * E, dtype)[..., E:]
    c0, dc = caches(B, E), caches(B, E, 1)
    y, c1 = axon.causal_conv(**z, activation="silu", cache_in=c0)
    grads = axon.causal_conv_backward(dy, **z, activation="silu", cache_in=c0, dcache_out=dc)
    torch.cuda.synchronize()
    compare(z, list(range(B)), c0, dc, dy, y, c1, grads, "silu")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_two_parts_and_steps(dtype):
    axon = _axon()
    B, L, E = 3, 100, 70
    z = make((B, L), E, dtype, seed=4)
    want, _ = axon.causal_conv(**z, activation="silu")
    x = z.pop("x")
    y1, c = axon.causal_conv(x[:, :1].contiguous(), **z, activation="silu")
    y2, c = axon.causal_conv(x[:, 1:95].contiguous(), **z, activation="silu", cache_in=c, cache_out=c)
    pool = torch.zeros(5, 3, E).cuda()
    slots = torch.tensor([3, 0, 4], dtype=torch.int32).cuda()
    pool[slots.long()] = c
    ys = [y1, y2]
    for t in range(95, L):
        ys.append(axon.causal_conv_step(x[:, t], **z, cache=pool, slots=slots,
                                        activation="silu")[:, None])
    torch.cuda.synchronize()
    assert torch.equal(torch.cat(ys, 1), want)
    assert torch.equal(pool[slots.long()], x[:, -3:].float())


@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("n,E,dtype", [(1, 1, "f32"), (3, 257, "bf16"), (70, 64, "f32"), (5, 1024, "bf16")])
def test_step(n, E, dtype, act):
    axon = _axon()
    z = make((n,), E, dtype, seed=n, bias=n != 3)
    pool = caches(n + 4, E)
    slots = torch.randperm(n + 4, generator=torch.Generator().manual_seed(n))[:n].int()
    if n > 4:
        slots[1], slots[3] = -1, n + 4
    before, given = pool.clone(), torch.full((n, E), 7.0, dtype=T[dtype]).cuda()
    y = axon.causal_conv_step(**z, cache=pool, slots=slots.cuda(), y=given, activation=act)
    torch.cuda.synchronize()
    live = set()
    for r in range(n):
        slot = int(slots[r])
        if not 0 <= slot < n + 4:
            assert bool((y[r] == 7).all())
            continue
        live.add(slot)
        want, off, cache = ref.conv(z["x"][r:r + 1], z["conv_w"], z["conv_b"], before[slot],
                                    act == "silu")
        ref.within(y[r:r + 1], want, off, f"y {r}")
        assert torch.equal(pool[slot].cpu().double(), cache)
    for j in range(n + 4):
        assert j in live or torch.equal(pool[j], before[j])
    y2 = axon.causal_conv_step(**z, cache=before.clone(), slots=slots.cuda(), activation=act)
    torch.cuda.synchronize()
    idle = torch.tensor([not 0 <= int(s) < n + 4 for s in slots])
    assert torch.equal(y2.cpu()[~idle], y.cpu()[~idle]) and not y2.cpu()[idle].any()


def test_as_in_the_prefill():
    """The convolution that prefill runs is this one: a scan whose decay forgets everything and whose
    readout is the skip alone shows u."""
    axon = _axon()
    B, L, E = 2, 70, 32
    z = make((B, L), E, seed=8)
    c0 = caches(B, E)
    zeros = torch.zeros(B, L, 16).cuda()
    gate = torch.full((B, L, E), 40.0).cuda()  # SiLU(40) = 40
    y, cache, _ = axon.prefill(z["x"], gate, torch.zeros(B, L, E).cuda(), zeros, zeros,
                               torch.zeros(E, 16).cuda(), torch.ones(E).cuda(), torch.zeros(E).cuda(),
                               z["conv_w"], z["conv_b"], conv_cache_in=c0, conv_activation="silu")
    mine, cache2 = axon.causal_conv(**z, cache_in=c0, activation="silu")
    torch.cuda.synchronize()
    assert torch.equal(cache, cache2)
    # both within the bound of one of them of the 64-bit value
    for b in range(B):
        want, off, _ = ref.conv(z["x"][b], z["conv_w"], z["conv_b"], c0[b], True)
        ref.within(y[b] / 40, want, off + 8 * ref.U * want.abs(), f"prefill {b}")
        ref.within(mine[b], want, off, f"conv {b}")


def test_no_tokens():
    axon = _axon()
    z = make((2, 0), 12)
    c0, dc = caches(2, 12), caches(2, 12, 1)
    y, c1 = axon.causal_conv(**z, cache_in=c0)
    g = axon.causal_conv_backward(y, **z, cache_in=c0, dcache_out=dc)
    torch.cuda.synchronize()
    assert y.shape == (2, 0, 12) and torch.equal(c0, c1) and torch.equal(g.dcache_in, dc)
    assert not g.dconv_w.any() and not g.dconv_b.any()


def test_captured_graph_and_other_stream():
    axon = _axon()
    total, E = 700, 264
    z = make((total,), E, "bf16", seed=1)
    dy = grad((total,), E, "bf16")
    n = torch.tensor([300, 0, 400], dtype=torch.int32).cuda()
    c0 = caches(3, E)

    def work(stream=None):
        tables = axon.sequence_tables(n, total, stream=stream)
        kw = dict(tables=tables, cache_in=c0, activation="silu", stream=stream)
        return [*axon.causal_conv(**z, **kw), *axon.causal_conv_backward(dy, **z, **kw)]

    work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = work()
    for lengths in ([300, 0, 400], [1, 2, 3], [0, 700, 0], [64, 128, 500]):
        n.copy_(torch.tensor(lengths, dtype=torch.int32))
        for t in out:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        want = work()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    got = work(side)
    junk = [torch.full((1 << 20,), float("nan"), device="cuda") for _ in range(8)]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    del junk


def test_buffer_beyond_32_bits():
    axon = _axon()
    E, total = 16384, 131072 + 500
    g = torch.Generator(device="cuda").manual_seed(0)
    z = make((1,), E, "bf16", seed=1)
    z["x"] = torch.empty(total, E, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    lengths = torch.tensor([131000, 72, 495], dtype=torch.int32).cuda()
    tables = axon.sequence_tables(lengths, total)
    y, c = axon.causal_conv(**z, tables=tables, activation="silu")
    d = axon.causal_conv_backward(z["x"], **z, tables=tables, activation="silu")
    lo = 131072
    x = z.pop("x")[None, lo:lo + 495].contiguous()
    ya, ca = axon.causal_conv(x, **z, activation="silu")
    da = axon.causal_conv_backward(x, x, **z, activation="silu")
    torch.cuda.synchronize()
    assert torch.equal(y[lo:lo + 495], ya[0]) and torch.equal(c[2], ca[0])
    assert torch.equal(d.dx[lo:lo + 495], da.dx[0])
    assert not y[lo + 495:].any() and not d.dx[lo + 495:].any()


def test_sums_over_many_tokens():
    """Sums of 200000 alike terms do not drift: x and dy are ones."""
    axon = _axon()
    L = 200_000
    x = torch.ones(1, L, 8, device="cuda")
    d = axon.causal_conv_backward(x, x, torch.ones(8, 4, device="cuda"))
    torch.cuda.synchronize()
    want = torch.tensor([L - 3.0, L - 2.0, L - 1.0, L]).expand(8, 4)
    assert torch.equal(d.dconv_w.cpu(), want) and bool((d.dconv_b == L).all())
