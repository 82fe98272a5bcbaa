"""The gated linear recurrence on the GPU against its plain 64-bit form, forward, backward and step:
one token to long sequences, odd widths, packed and empty sequences, pools of states, parts of one
projection, slow and strong decays, values that are not finite, streams, graphs, large buffers."""
from __future__ import annotations

import pytest

from gpu_util import say

torch = pytest.importorskip("torch")

import recurrent_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu
T = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import selective_state_space_depthwise_amd as axon

    axon.load()
    yield
    torch.cuda.synchronize()


def _axon():
    import selective_state_space_depthwise_amd as axon

    return axon


def make(lead, E, act="f32", seed=0, gated=True, rate=(-3.0, 0.0), bias=True):
    g = torch.Generator().manual_seed(seed)

    def n(*s):
        return torch.randn(*s, generator=g)

    z = dict(x=n(*lead, E), dt_raw=n(*lead, E), in_raw=n(*lead, E) if gated else None)
    z = {k: None if v is None else v.to(T[act]).cuda() for k, v in z.items()}
    z["A_log"] = (rate[0] + (rate[1] - rate[0]) * torch.rand(E, generator=g)).cuda()
    z["dt_bias"] = (0.3 * n(E)).cuda() if bias else None
    z["in_bias"] = (0.3 * n(E)).cuda() if bias and gated else None
    return z


def states(n, E, seed=0):
    return torch.randn(n, E, generator=torch.Generator().manual_seed(99 + seed)).cuda()


def grad(lead, E, act, seed=0):
    return torch.randn(*lead, E, generator=torch.Generator().manual_seed(7 + seed)).to(T[act]).cuda()


def sequence(z, s0, at, gate, scale):
    rows = {k: None if z[k] is None else z[k][at] for k in ("x", "dt_raw", "in_raw")}
    return ref.Linear(rows["x"], rows["dt_raw"], rows["in_raw"], s0, z["A_log"], z["dt_bias"],
                      z["in_bias"], gate, scale)


def compare(z, parts, s0, ds, dy, y, s1, grads, gate, scale, act_grads=True):
    """parts: the rows of each sequence."""
    E = y.shape[-1]
    sums = {k: [torch.zeros(E, dtype=torch.float64)] * 2 for k in ("dA_log", "ddt_bias", "din_bias")}
    for n, at in enumerate(parts):
        r = sequence(z, s0[n], at, gate, scale)
        ref.within(y[at], r.y, r.bound, f"y {at}")
        ref.within(s1[n], r.state, r.state_bound, f"state {n}")
        if grads is None:
            continue
        want = r.backward(dy[at], ds[n])
        for k in ("dx", "ddt_raw", "din_raw"):
            if k in want:
                ref.within(getattr(grads, k)[at], *want[k], f"{k} {at}")
        ref.within(grads.dstate_in[n], *want["dstate_in"], f"dstate_in {n}")
        for k in sums:
            if k in want:
                sums[k] = [a + b for a, b in zip(sums[k], want[k])]
    if grads is not None:
        for k in sums:
            if getattr(grads, k) is not None:
                ref.within(getattr(grads, k), *sums[k], k)


UNIFORM = [
    # (B, L, E, act, gate, scale, gated, bias)
    (1, 1, 1, "f32", "sigmoid", "sqrt", True, True),
    (2, 2, 3, "bf16", "softplus", "complement", False, True),
    (2, 31, 64, "f32", "softplus", "none", True, True),
    (1, 32, 65, "bf16", "sigmoid", "none", False, False),
    (2, 33, 128, "f32", "sigmoid", "complement", True, False),
    (3, 63, 5, "f32", "sigmoid", "sqrt", True, True),
    (1, 64, 130, "bf16", "softplus", "sqrt", True, True),
    (2, 65, 257, "f32", "softplus", "sqrt", False, True),
    (3, 127, 96, "bf16", "sigmoid", "sqrt", True, True),
    (2, 200, 200, "f32", "sigmoid", "sqrt", True, False),
    (1, 256, 66, "f32", "softplus", "complement", True, True),
    (2, 257, 70, "bf16", "softplus", "complement", False, True),
    (4, 300, 33, "f32", "sigmoid", "none", True, True),
    (1, 1025, 192, "bf16", "sigmoid", "sqrt", True, True),
    (1, 2500, 40, "f32", "sigmoid", "sqrt", True, True),
]


@pytest.mark.parametrize("B,L,E,act,gate,scale,gated,bias", UNIFORM)
def test_uniform_batch(B, L, E, act, gate, scale, gated, bias):
    say(f"[linear] {B} x {L} x {E} {act} {gate} {scale} gated={gated}")
    axon = _axon()
    z = make((B, L), E, act, seed=L + E, gated=gated, bias=bias)
    s0, ds, dy = states(B, E, 1), states(B, E, 2), grad((B, L), E, act)
    points = axon.linear_checkpoints(z["x"])
    y, s1 = axon.linear_scan(**z, gate=gate, input_scale=scale, state_in=s0, checkpoints=points)
    grads = axon.linear_scan_backward(dy, **z, gate=gate, input_scale=scale, checkpoints=points,
                                      dstate_out=ds)
    torch.cuda.synchronize()
    compare(z, list(range(B)), s0, ds, dy, y, s1, grads, gate, scale)
    # without states, checkpoints or biases given
    y0, _ = axon.linear_scan(**z, gate=gate, input_scale=scale)
    torch.cuda.synchronize()
    r = sequence(z, torch.zeros(E), 0, gate, scale)
    ref.within(y0[0], r.y, r.bound, "y from zeros")


PACKED = [
    # lengths, rows behind
    ([5, 0, 64, 1, 130, 65, 0, 63], 37),
    ([1] * 40, 3),
    ([700], 0),
    ([0, 0, 3], 200),
    ([64, 128, 192, 1], 1),
    ([2, 500, 3, 511, 1, 0], 0),
]


def parts_of(lengths):
    at, out = 0, []
    for n in lengths:
        out.append(slice(at, at + n))
        at += n
    return out


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("lengths,spare", PACKED)
def test_packed(lengths, spare, act):
    say(f"[linear] packed {lengths} + {spare} {act}")
    axon = _axon()
    total, E, N = sum(lengths) + spare, 71, len(lengths)
    z = make((total,), E, act, seed=total)
    for k in ("x", "dt_raw", "in_raw"):
        z[k][total - spare:] = float("nan")
    dy = grad((total,), E, act)
    dy[total - spare:] = float("nan")
    tables = axon.sequence_tables(torch.tensor(lengths, dtype=torch.int32).cuda(), total)
    s0, ds = states(N, E, 3), states(N, E, 4)
    points = axon.linear_checkpoints(z["x"], tables=tables)
    y, s1 = axon.linear_scan(**z, tables=tables, state_in=s0, checkpoints=points)
    grads = axon.linear_scan_backward(dy, **z, tables=tables, checkpoints=points, dstate_out=ds)
    torch.cuda.synchronize()
    compare(z, parts_of(lengths), s0, ds, dy, y, s1, grads, "sigmoid", "sqrt")
    end = total - spare
    for t in (y, grads.dx, grads.ddt_raw, grads.din_raw):
        assert bool((t[end:] == 0).all())
    given = torch.full_like(y, 7.0)
    y2, s2 = axon.linear_scan(**z, lengths=torch.tensor(lengths, dtype=torch.int32).cuda(), y=given,
                              state_in=s0)
    torch.cuda.synchronize()
    assert y2 is given and bool((y2[end:] == 7).all()) and torch.equal(y2[:end], y[:end])
    assert torch.equal(s1, s2)


def test_lengths_beyond_the_buffer_are_cut():
    axon = _axon()
    z = make((100,), 9, seed=1)
    n = torch.tensor([70, -3, 60, 50], dtype=torch.int32).cuda()
    s0 = states(4, 9)
    y, s1 = axon.linear_scan(**z, lengths=n, state_in=s0)
    y2, s2 = axon.linear_scan(**z, lengths=torch.tensor([70, 0, 30, 0], dtype=torch.int32).cuda(),
                              state_in=s0)
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and torch.equal(s1, s2) and torch.equal(s1[3], s0[3])


@pytest.mark.parametrize("place", [True, False])
def test_pools(place):
    """States in a pool, in place or not; slots outside it; a pool larger than the batch."""
    axon = _axon()
    lengths, E = [70, 0, 300, 1, 64], 50
    z = make((sum(lengths),), E, seed=3)
    pool = states(9, E)
    ins = torch.tensor([4, 2, 8, -1, 100], dtype=torch.int32).cuda()
    outs = torch.tensor([4, 2, 8, 0, -5], dtype=torch.int32).cuda()
    out = pool.clone() if place else torch.full((7, E), 5.0).cuda()
    if not place:
        outs = torch.tensor([6, 2, 99, 0, 1], dtype=torch.int32).cuda()
    before = out.clone()
    y, got = axon.linear_scan(**z, lengths=torch.tensor(lengths, dtype=torch.int32).cuda(),
                              state_in=out if place else pool, in_slots=ins, state_out=out,
                              out_slots=outs)
    torch.cuda.synchronize()
    assert got is out
    touched = set()
    for n, at in enumerate(parts_of(lengths)):
        slot, to = int(ins[n]), int(outs[n])
        r = sequence(z, pool[slot] if 0 <= slot < 9 else torch.zeros(E), at, "sigmoid", "sqrt")
        ref.within(y[at], r.y, r.bound, f"y {n}")
        if 0 <= to < out.shape[0]:
            ref.within(out[to], r.state, r.state_bound, f"state {n}")
            touched.add(to)
    for j in range(out.shape[0]):
        assert j in touched or torch.equal(out[j], before[j])


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_parts_of_one_projection(act):
    """Rows that lie apart, from any channel on."""
    axon = _axon()
    B, L, E = 2, 90, 37
    big = make((B, L), 4 * E + 1, act, seed=5, gated=False)["x"]
    z = make((B, L), E, act, seed=6)
    z.update(x=big[..., 1:1 + E], dt_raw=big[..., 1 + E:1 + 2 * E], in_raw=big[..., 1 + 3 * E:])
    dy = grad((B, L), 2 * E, act)[..., E:]
    points = axon.linear_checkpoints(z["x"])
    s0, ds = states(B, E), states(B, E, 1)
    y, s1 = axon.linear_scan(**z, state_in=s0, checkpoints=points)
    grads = axon.linear_scan_backward(dy, **z, checkpoints=points, dstate_out=ds)
    torch.cuda.synchronize()
    compare(z, list(range(B)), s0, ds, dy, y, s1, grads, "sigmoid", "sqrt")


@pytest.mark.parametrize("gate", ["sigmoid", "softplus"])
@pytest.mark.parametrize("scale", ["sqrt", "complement", "none"])
@pytest.mark.parametrize("rate", [(-15.0, -13.0), (3.0, 8.0), (-40.0, -35.0)])
def test_slow_and_strong_decays(rate, scale, gate):
    """Decays of 1e-6 a token over 3000 of them, decays that leave nothing, and decays below what 1 - a
    holds in fp32; large first states."""
    axon = _axon()
    L, E = 3000 if rate[0] == -15 else 150, 16
    z = make((1, L), E, seed=8, rate=rate)
    s0, ds, dy = 1e6 * states(1, E), 1e3 * states(1, E, 2), grad((1, L), E, "f32")
    points = axon.linear_checkpoints(z["x"])
    y, s1 = axon.linear_scan(**z, gate=gate, input_scale=scale, state_in=s0, checkpoints=points)
    grads = axon.linear_scan_backward(dy, **z, gate=gate, input_scale=scale, checkpoints=points,
                                      dstate_out=ds)
    torch.cuda.synchronize()
    compare(z, [0], s0, ds, dy, y, s1, grads, gate, scale)


@pytest.mark.parametrize("gate", ["sigmoid", "softplus"])
@pytest.mark.parametrize("scale", ["sqrt", "complement", "none"])
def test_gates_at_their_ends(scale, gate):
    """Gates of +-60 and +-90 saturate: finite results and gradients."""
    axon = _axon()
    E = 8
    z = make((1, 130), E, seed=9)
    z["dt_raw"][0, ::2] = torch.tensor([60.0, -60.0, 90.0, -90.0, 25.0, -25.0, 0.0, -110.0]).cuda()
    z["in_raw"][0, ::3] = torch.tensor([-60.0, 60.0, -90.0, 90.0, 3.0, 0.0, -110.0, 110.0]).cuda()
    s0, ds, dy = states(1, E), states(1, E, 2), grad((1, 130), E, "f32")
    points = axon.linear_checkpoints(z["x"])
    y, s1 = axon.linear_scan(**z, gate=gate, input_scale=scale, state_in=s0, checkpoints=points)
    grads = axon.linear_scan_backward(dy, **z, gate=gate, input_scale=scale, checkpoints=points,
                                      dstate_out=ds)
    torch.cuda.synchronize()
    compare(z, [0], s0, ds, dy, y, s1, grads, gate, scale)


def test_infinite_gates_are_their_limits():
    axon = _axon()
    inf = float("inf")
    for gate in ("sigmoid", "softplus"):
        z = make((1, 70), 3, seed=9)
        w = {k: v.clone() for k, v in z.items()}
        # -inf: the token keeps the state; in_raw -inf: nothing enters
        z["dt_raw"][0, 10], w["dt_raw"][0, 10] = -inf, -200.0
        z["in_raw"][0, 20], w["in_raw"][0, 20] = -inf, -200.0
        z["in_raw"][0, 21], w["in_raw"][0, 21] = inf, 200.0
        z["dt_raw"][0, 30], w["dt_raw"][0, 30] = inf, 200.0 if gate == "sigmoid" else 1e30
        a = [axon.linear_checkpoints(z["x"]) for _ in range(2)]
        got, state = axon.linear_scan(**z, gate=gate, checkpoints=a[0])
        want, state2 = axon.linear_scan(**w, gate=gate, checkpoints=a[1])
        dy = grad((1, 70), 3, "f32")
        g1 = axon.linear_scan_backward(dy, **z, gate=gate, checkpoints=a[0])
        g2 = axon.linear_scan_backward(dy, **w, gate=gate, checkpoints=a[1])
        torch.cuda.synchronize()
        assert torch.isfinite(got).all() and torch.allclose(got, want, rtol=1e-6, atol=1e-30)
        assert torch.equal(state, state2)
        for p, q in zip(g1, g2):
            assert torch.isfinite(p).all() and torch.allclose(p, q, rtol=1e-5, atol=1e-30)


@pytest.mark.parametrize("name", ["x", "dt_raw", "in_raw"])
def test_nan_stays_in_its_channel_and_sequence(name):
    axon = _axon()
    lengths, E = [100, 300, 64, 1, 200], 70
    total = sum(lengths)
    z = make((total,), E, seed=2)
    n = torch.tensor(lengths, dtype=torch.int32).cuda()
    want, s_want = axon.linear_scan(**z, lengths=n)
    z[name] = z[name].clone()
    z[name][250, 13] = float("nan")
    z[name][464, 69] = float("nan")
    y, s = axon.linear_scan(**z, lengths=n)
    torch.cuda.synchronize()
    bad = torch.zeros(total, E, dtype=torch.bool)
    bad[250:400, 13] = True
    bad[464, 69] = True
    assert torch.equal(torch.isnan(y).cpu(), bad)
    assert torch.equal(y.cpu()[~bad], want.cpu()[~bad])
    bad_s = torch.zeros(5, E, dtype=torch.bool)
    bad_s[1, 13] = bad_s[3, 69] = True
    assert torch.equal(torch.isnan(s).cpu(), bad_s)
    assert torch.equal(s.cpu()[~bad_s], s_want.cpu()[~bad_s])


def test_no_tokens():
    axon = _axon()
    z = make((2, 0), 12)
    s0 = states(2, 12)
    points = axon.linear_checkpoints(z["x"])
    y, s1 = axon.linear_scan(**z, state_in=s0, checkpoints=points)
    ds = states(2, 12, 1)
    g = axon.linear_scan_backward(y, **z, checkpoints=points, dstate_out=ds)
    torch.cuda.synchronize()
    assert y.shape == (2, 0, 12) and torch.equal(s1, s0) and torch.equal(g.dstate_in, ds)
    assert not g.dA_log.any() and not g.ddt_bias.any() and not g.din_bias.any()
    z = make((0,), 12)
    y, s1 = axon.linear_scan(**z, lengths=torch.zeros(3, dtype=torch.int32).cuda(),
                             state_in=states(3, 12))
    torch.cuda.synchronize()
    assert torch.equal(s1, states(3, 12))


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_scan_in_two_parts_and_steps(act):
    """A scan that continues another one, and steps behind it, are the whole scan."""
    axon = _axon()
    B, L, E = 3, 150, 66
    z = make((B, L), E, act, seed=4)
    whole = [sequence(z, torch.zeros(E), b, "sigmoid", "sqrt") for b in range(B)]

    def part(a, b):
        return {k: v[:, a:b].contiguous() if k in ("x", "dt_raw", "in_raw") else v
                for k, v in z.items()}

    y1, s = axon.linear_scan(**part(0, 70))
    y2, s = axon.linear_scan(**part(70, 140), state_in=s, state_out=s)
    pool = torch.zeros(5, E).cuda()
    slots = torch.tensor([3, 0, 4], dtype=torch.int32).cuda()
    pool[slots.long()] = s
    ys = [y1, y2]
    for t in range(140, L):
        step = {k: v[:, t] if k in ("x", "dt_raw", "in_raw") else v for k, v in z.items()}
        ys.append(axon.linear_step(**step, state=pool, slots=slots)[:, None])
    torch.cuda.synchronize()
    y = torch.cat(ys, 1)
    for b in range(B):
        ref.within(y[b], whole[b].y, whole[b].bound, f"y {b}")
        ref.within(pool[slots[b].long()], whole[b].state, whole[b].state_bound, f"state {b}")
    assert not pool[1].any() and not pool[2].any()


@pytest.mark.parametrize("gate", ["sigmoid", "softplus"])
@pytest.mark.parametrize("scale", ["sqrt", "complement", "none"])
@pytest.mark.parametrize("n,E,act", [(1, 1, "f32"), (3, 257, "bf16"), (70, 64, "f32"), (5, 1002, "bf16")])
def test_step(n, E, act, scale, gate):
    axon = _axon()
    z = make((n,), E, act, seed=n + E, gated=n != 3)
    pool = states(n + 4, E)
    slots = torch.randperm(n + 4, generator=torch.Generator().manual_seed(n))[:n].int()
    if n > 4:
        slots[1], slots[3] = -1, n + 4
    before, given = pool.clone(), torch.full((n, E), 7.0, dtype=T[act]).cuda()
    y = axon.linear_step(**z, state=pool, slots=slots.cuda(), y=given, gate=gate, input_scale=scale)
    torch.cuda.synchronize()
    live = set()
    for r in range(n):
        slot = int(slots[r])
        if not 0 <= slot < n + 4:
            assert bool((y[r] == 7).all())
            continue
        live.add(slot)
        want = sequence(z, before[slot], slice(r, r + 1), gate, scale)
        ref.within(y[r:r + 1], want.y, want.bound, f"y {r}")
        ref.within(pool[slot], want.state, want.state_bound, f"state {r}")
    for j in range(n + 4):
        assert j in live or torch.equal(pool[j], before[j])
    y2 = axon.linear_step(**z, state=before.clone(), slots=slots.cuda(), gate=gate, input_scale=scale)
    torch.cuda.synchronize()
    idle = torch.tensor([not 0 <= int(s) < n + 4 for s in slots])
    assert torch.equal(y2.cpu()[~idle], y.cpu()[~idle]) and not y2.cpu()[idle].any()


def test_same_results_every_time():
    """Twice the same call, alone and beside others on another stream."""
    axon = _axon()
    lengths = [1000, 3, 2000, 700]
    n = torch.tensor(lengths, dtype=torch.int32).cuda()
    z = make((sum(lengths),), 330, "bf16", seed=1)
    other = make((4, 900), 200, "f32", seed=2)
    dy = grad((sum(lengths),), 330, "bf16")
    tables = axon.sequence_tables(n, sum(lengths))
    side = torch.cuda.Stream()

    def once():
        p = axon.linear_checkpoints(z["x"], tables=tables)
        y, s = axon.linear_scan(**z, tables=tables, checkpoints=p)
        return [y, s, *axon.linear_scan_backward(dy, **z, tables=tables, checkpoints=p)]

    first = once()
    o1 = axon.linear_scan(**other)
    torch.cuda.synchronize()
    for _ in range(5):
        o2 = axon.linear_scan(**other, stream=side)
        again = once()
        o3 = axon.linear_scan(**other, stream=side)
        torch.cuda.synchronize()
        for a, b in zip(first, again):
            assert torch.equal(a, b)
        for o in (o2, o3):
            assert torch.equal(o[0], o1[0]) and torch.equal(o[1], o1[1])


def test_other_stream_keeps_memory():
    axon = _axon()
    z = make((2, 700), 256, "bf16", seed=3)
    dy = grad((2, 700), 256, "bf16")
    p0 = axon.linear_checkpoints(z["x"])
    want = axon.linear_scan(**z, checkpoints=p0)
    gw = axon.linear_scan_backward(dy, **z, checkpoints=p0)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    p = axon.linear_checkpoints(z["x"])
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    got = axon.linear_scan(**z, checkpoints=p, stream=side)
    grads = axon.linear_scan_backward(dy, **z, checkpoints=p, stream=side)
    junk = [torch.full((1 << 20,), float("nan"), device="cuda") for _ in range(8)]
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for a, b in zip(grads, gw):
        assert torch.equal(a, b)
    del junk


def test_captured_graph():
    """Forward and backward captured once, replayed with other lengths and inputs, with eager work of
    the same kind between the replays."""
    axon = _axon()
    total, E = 900, 130
    z = make((total,), E, "bf16", seed=1)
    dy = grad((total,), E, "bf16")
    n = torch.tensor([500, 0, 400], dtype=torch.int32).cuda()

    def work():
        tables = axon.sequence_tables(n, total)
        p = axon.linear_checkpoints(z["x"], tables=tables)
        y, s = axon.linear_scan(**z, tables=tables, checkpoints=p)
        return [y, s, *axon.linear_scan_backward(dy, **z, tables=tables, checkpoints=p)]

    work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = work()
    for lengths in ([500, 0, 400], [1, 1, 1], [0, 900, 0], [64, 128, 700]):
        n.copy_(torch.tensor(lengths, dtype=torch.int32))
        z["x"].copy_(make((total,), E, "bf16", seed=sum(lengths) + lengths[0])["x"])
        for t in out:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        want = work()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(out, want):
        assert torch.equal(a, b)


def test_many_sequences():
    axon = _axon()
    g = torch.Generator().manual_seed(0)
    lengths = torch.randint(0, 9, (3000,), generator=g)
    total, E = int(lengths.sum()) + 10, 20
    z = make((total,), E, seed=6)
    s0 = states(3000, E)
    dy = grad((total,), E, "f32")
    tables = axon.sequence_tables(lengths.int().cuda(), total)
    p = axon.linear_checkpoints(z["x"], tables=tables)
    y, s1 = axon.linear_scan(**z, tables=tables, state_in=s0, checkpoints=p)
    d = axon.linear_scan_backward(dy, **z, tables=tables, checkpoints=p)
    torch.cuda.synchronize()
    # the same sequences as a padded batch of 8 tokens, by the plain form in one go
    at = torch.cat([torch.zeros(1, dtype=torch.int64), lengths.cumsum(0)])
    pick = [0, 1, 2, 777, 1500, 2998, 2999]
    for j in pick:
        r = sequence(z, s0[j], slice(int(at[j]), int(at[j + 1])), "sigmoid", "sqrt")
        ref.within(y[at[j]:at[j + 1]], r.y, r.bound, f"y {j}")
        ref.within(s1[j], r.state, r.state_bound, f"state {j}")
        want = r.backward(dy[at[j]:at[j + 1]], torch.zeros(E))
        ref.within(d.dx[at[j]:at[j + 1]], *want["dx"], f"dx {j}")
        ref.within(d.dstate_in[j], *want["dstate_in"], f"dstate_in {j}")
    assert not y[total - 10:].any()


def test_buffer_beyond_32_bits():
    """2^31 elements and more: the last sequence of a packed buffer as if it were alone."""
    axon = _axon()
    E, total = 16384, 131072 + 900
    g = torch.Generator(device="cuda").manual_seed(0)
    z = make((1,), E, "bf16", seed=1, gated=False)
    for k in ("x", "dt_raw"):
        z[k] = torch.empty(total, E, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    lengths = torch.tensor([131000, 72, 895], dtype=torch.int32).cuda()
    tables = axon.sequence_tables(lengths, total)
    p = axon.linear_checkpoints(z["x"], tables=tables)
    y, s = axon.linear_scan(**z, tables=tables, checkpoints=p)
    d = axon.linear_scan_backward(z["x"], **z, tables=tables, checkpoints=p)
    lo = 131072
    alone = {k: v[None, lo:lo + 895].contiguous() if k in ("x", "dt_raw") else v for k, v in z.items()}
    pa = axon.linear_checkpoints(alone["x"])
    ya, sa = axon.linear_scan(**alone, checkpoints=pa)
    da = axon.linear_scan_backward(alone["x"], **alone, checkpoints=pa)
    torch.cuda.synchronize()
    # carries join other groups of blocks in the two calls: rounding apart, the same
    assert torch.allclose(y[lo:lo + 895].float(), ya[0].float(), rtol=2 ** -7, atol=1e-4)
    assert torch.allclose(s[2], sa[0], rtol=1e-4, atol=1e-5)
    assert torch.allclose(d.dx[lo:lo + 895].float(), da.dx[0].float(), rtol=2 ** -7, atol=1e-3)
    assert torch.allclose(d.ddt_raw[lo:lo + 895].float(), da.ddt_raw[0].float(), rtol=2 ** -7, atol=1e-3)
    assert not y[lo + 895:].any() and not d.dx[lo + 895:].any()
