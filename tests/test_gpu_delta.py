"""The gated delta rule on the GPU against its plain 64-bit recurrence: ragged and empty sequences,
packed buffers, pools of states, parts of one projection, keys that are all alike, strong decays,
streams, captured graphs, and prefill and steps together."""
from __future__ import annotations

import pytest

from gpu_util import say

torch = pytest.importorskip("torch")

import delta_ref as ref  # noqa: E402

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


def make(lead, hk, hv, K, V, act="f32", seed=0, alike=0.5):
    """Inputs on the GPU; keys and queries share a direction (`alike` of their size)."""
    g = torch.Generator().manual_seed(seed)

    def n(*s):
        return torch.randn(*s, generator=g)

    common = n(hk, K)
    d = dict(q=n(*lead, hk, K) + alike * common, k=n(*lead, hk, K) + alike * common,
             v=n(*lead, hv, V), dt_raw=n(*lead, hv), beta_raw=n(*lead, hv))
    d = {x: t.to(T[act]).cuda() for x, t in d.items()}
    u = torch.rand(2, hv, generator=g)
    d["A_log"] = torch.log(1 + 15 * u[0]).cuda()
    d["dt_bias"] = (torch.log(torch.expm1(1e-3 + 0.1 * u[1]))).cuda()
    return d


def state(n, hv, V, K, seed=0):
    g = torch.Generator().manual_seed(1000 + seed)
    return (torch.randn(n, hv, V, K, generator=g) * 0.3).cuda()


def rows(d, at):
    """The inputs of the tokens `at` (a slice of the packed axis, or an index of a batch)."""
    return {x: (t if x in ("A_log", "dt_bias") else t[at]) for x, t in d.items()}


def close(got, want, big, what):
    got = got.detach()
    bf = got.dtype == torch.bfloat16
    got = got.double().cpu()
    assert torch.isfinite(got).all(), f"{what}: not finite"
    bound = ref.F32 * (big + want.abs()) + (ref.BF16_HALF * want.abs() if bf else 0.0)
    off = (got - want).abs()
    assert bool((off <= bound).all()), (
        f"{what}: {float((off / bound).nan_to_num().max()):.2f} times the bound, largest error "
        f"{float(off.max()):.3e}")


UNIFORM = [
    # (B, L, hk, hv, K, V, act, carried)
    (1, 1, 1, 1, 64, 16, "f32", True),
    (2, 1, 2, 4, 128, 128, "bf16", True),
    (1, 63, 2, 2, 128, 64, "f32", False),
    (2, 64, 1, 2, 64, 64, "bf16", True),
    (1, 65, 2, 2, 128, 128, "f32", True),
    (3, 130, 1, 3, 128, 48, "bf16", False),
    (1, 333, 2, 4, 64, 256, "f32", True),
    (2, 200, 2, 4, 128, 128, "bf16", True),
    (1, 257, 1, 2, 128, 240, "bf16", True),
    (1, 700, 3, 3, 64, 80, "bf16", False),
]


@pytest.mark.parametrize("B,L,hk,hv,K,V,act,carried", UNIFORM)
def test_uniform_batch(B, L, hk, hv, K, V, act, carried):
    say(f"[delta] B={B} L={L} heads {hk}/{hv} K={K} V={V} {act} carried={carried}")
    d = make((B, L), hk, hv, K, V, act, seed=L + V)
    s0 = state(B, hv, V, K, L) if carried else None
    y, s1 = _axon().gated_delta_scan(**d, state_in=s0)
    torch.cuda.synchronize()
    for b in range(B):
        start = s0[b] if carried else torch.zeros(hv, V, K)
        yr, sr, big = ref.delta_tokens(start, **rows(d, b))
        close(y[b], yr, big, f"y[{b}]")
        close(s1[b], sr, big, f"state[{b}]")


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_packed_with_slots(act):
    """Lengths from none to several chunks, new and continued sequences, one not stored, one slot
    out of range; rows behind the last sequence hold NaN and stay as they were."""
    lengths = [5, 0, 64, 1, 130, 65, 0, 63]
    total = sum(lengths) + 37
    hk, hv, K, V = 2, 4, 128, 64
    say(f"[delta] packed {lengths} of {total} rows, {act}")
    d = make((total,), hk, hv, K, V, act, seed=3)
    end = sum(lengths)
    for x in ("q", "k", "v", "dt_raw", "beta_raw"):
        d[x][end:] = float("nan")
    pool = state(11, hv, V, K, 7)
    before = pool.clone()
    ins = torch.tensor([3, 4, -1, 0, 99, 7, -5, 10], dtype=torch.int32).cuda()
    outs = torch.tensor([3, 4, 5, 0, 6, -1, 8, 2 ** 30], dtype=torch.int32).cuda()
    y = torch.full((total, hv, V), 7.0, dtype=T[act]).cuda()
    _axon().gated_delta_scan(**d, lengths=torch.tensor(lengths, dtype=torch.int32).cuda(),
                             state_in=pool, in_slots=ins, y=y, state_out=pool, out_slots=outs)
    torch.cuda.synchronize()
    touched, at = set(), 0
    for n, length in enumerate(lengths):
        i, o = int(ins[n]), int(outs[n])
        start = before[i] if 0 <= i < 11 else torch.zeros(hv, V, K)
        yr, sr, big = ref.delta_tokens(start, **rows(d, slice(at, at + length)))
        close(y[at:at + length], yr, big, f"y of sequence {n}")
        if 0 <= o < 11:
            touched.add(o)
            close(pool[o], sr, big, f"state of sequence {n}")
        at += length
    assert bool((y[end:] == 7.0).all())
    for slot in set(range(11)) - touched:
        assert torch.equal(pool[slot], before[slot]), f"slot {slot} changed"


def test_packed_sequences_do_not_see_each_other():
    """One sequence of NaN and infinities between others: theirs are the same bits as without."""
    lengths = [70, 40, 100]
    d = make((210,), 1, 2, 128, 32, "bf16", seed=9)
    n = torch.tensor(lengths, dtype=torch.int32).cuda()
    y0, s0 = _axon().gated_delta_scan(**d, lengths=n)
    bad = {x: t.clone() for x, t in d.items()}
    for x in ("q", "k", "v", "dt_raw", "beta_raw"):
        bad[x][70:110] = float("nan")
        bad[x][71] = float("inf")
    y1, s1 = _axon().gated_delta_scan(**bad, lengths=n)
    torch.cuda.synchronize()
    for part in (slice(0, 70), slice(110, 210)):
        assert torch.equal(y0[part], y1[part])
    assert torch.equal(s0[0], s1[0]) and torch.equal(s0[2], s1[2])


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_tables_once_for_many_calls_and_cut_off(act):
    """Tables built once; lengths past the buffer are cut off at its end, negative ones are none."""
    axon = _axon()
    d = make((150,), 1, 1, 64, 16, act, seed=4)
    t = axon.sequence_tables(torch.tensor([40, -3, 90, 500, 9], dtype=torch.int32).cuda(), 150)
    y, s = axon.gated_delta_scan(**d, tables=t)
    y2, s2 = axon.gated_delta_scan(**d, tables=t)
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and torch.equal(s, s2)
    for n, (a, b) in enumerate([(0, 40), (40, 40), (40, 130), (130, 150), (150, 150)]):
        yr, sr, big = ref.delta_tokens(torch.zeros(1, 16, 64), **rows(d, slice(a, b)))
        close(y[a:b], yr, big, f"y of sequence {n}")
        close(s[n], sr, big, f"state of sequence {n}")


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["alike", "strong", "weak", "zero"])
def test_hard_values(kind, act):
    """Keys that are all alike and written with full strength (the chunk's system is as far from
    diagonal as it gets), decays that reach zero, no decay at all, keys of zeros."""
    say(f"[delta] {kind} {act}")
    B, L, hk, hv, K, V = 1, 150, 1, 2, 128, 32
    d = make((B, L), hk, hv, K, V, act, seed=11, alike=0.0)
    if kind == "alike":
        d["k"][:] = d["k"][:, :1]
        d["beta_raw"][:] = 30.0
        d["A_log"][:] = -12.0
    elif kind == "strong":
        d["dt_raw"][:, ::7] = 300.0
        d["dt_raw"][:, 1::5] = -80.0
    elif kind == "weak":
        d["A_log"][:] = -40.0
    else:
        d["k"][:, 20:90] = 0.0
        d["q"][:, 50:70] = 0.0
    s0 = state(B, hv, V, K, 5)
    y, s1 = _axon().gated_delta_scan(**d, state_in=s0)
    torch.cuda.synchronize()
    yr, sr, big = ref.delta_tokens(s0[0], **rows(d, 0))
    close(y[0], yr, big, "y")
    close(s1[0], sr, big, "state")


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_parts_of_one_projection(act):
    """q, k, v as slices of one buffer give the bits of contiguous ones, in the scan and the step."""
    hk, hv, K, V, total = 2, 4, 64, 32, 100
    d = make((total,), hk, hv, K, V, act, seed=6)
    whole = torch.randn(total, 2 * hk * K + hv * V + 8).to(T[act]).cuda()
    s = dict(d)
    for x, lo, h, w in (("q", 0, hk, K), ("k", hk * K, hk, K), ("v", 2 * hk * K, hv, V)):
        s[x] = whole[:, lo:lo + h * w].unflatten(-1, (h, w))
        s[x].copy_(d[x])
        assert not s[x].is_contiguous()
    n = torch.tensor([30, 70], dtype=torch.int32).cuda()
    for a, b in zip(_axon().gated_delta_scan(**d, lengths=n),
                    _axon().gated_delta_scan(**s, lengths=n)):
        assert torch.equal(a, b)
    # a uniform batch of the same rows
    u = {x: (t if x in ("A_log", "dt_bias") else t.unflatten(0, (4, 25))) for x, t in d.items()}
    us = {x: (t if x in ("A_log", "dt_bias") else t.unflatten(0, (4, 25))) for x, t in s.items()}
    for a, b in zip(_axon().gated_delta_scan(**u), _axon().gated_delta_scan(**us)):
        assert torch.equal(a, b)
    p0 = state(total, hv, V, K, 1)
    p1 = p0.clone()
    assert torch.equal(_axon().gated_delta_step(**d, state=p0), _axon().gated_delta_step(**s, state=p1))
    assert torch.equal(p0, p1)


@pytest.mark.parametrize("act,K,V", [("f32", 128, 128), ("bf16", 128, 128), ("bf16", 64, 48),
                                     ("f32", 64, 240), ("bf16", 128, 256)])
@pytest.mark.parametrize("slow", [3.0, 0.0, 1.5])
def test_long_sequences_in_segments(act, K, V, slow):
    """Few heads and long sequences are walked in segments at once: a uniform batch in place, and
    packed sequences of which some fill many segments and some none. Decays are such that states
    live through segments (slow), that they end within a few chunks, and between."""
    say(f"[delta] segments {act} K={K} V={V} slow={slow}")
    axon = _axon()
    hk, hv, L = 1, 2, 2200
    d = make((2, L), hk, hv, K, V, act, seed=31)
    d["A_log"] -= slow
    s = state(2, hv, V, K, 6)
    start = s.clone()
    y, _ = axon.gated_delta_scan(**d, state_in=s, state_out=s)
    torch.cuda.synchronize()
    for b in range(2):
        yr, sr, big = ref.delta_tokens(start[b], **rows(d, b))
        close(y[b], yr, 2 * big, f"y[{b}]")
        close(s[b], sr, 2 * big, f"state[{b}]")
    p = {x: (t if x in ("A_log", "dt_bias") else t.flatten(0, 1)) for x, t in d.items()}
    lengths = [3000, 0, 1, 1399]
    pool = state(6, hv, V, K, 7)
    before = pool.clone()
    slots = torch.tensor([5, 0, -1, 2], dtype=torch.int32).cuda()
    y, _ = axon.gated_delta_scan(**p, lengths=torch.tensor(lengths, dtype=torch.int32).cuda(),
                                 state_in=pool, in_slots=slots, state_out=pool, out_slots=slots)
    torch.cuda.synchronize()
    at = 0
    for n, length in enumerate(lengths):
        i = int(slots[n])
        yr, sr, big = ref.delta_tokens(before[i] if i >= 0 else torch.zeros(hv, V, K),
                                       **rows(p, slice(at, at + length)))
        close(y[at:at + length], yr, 2 * big, f"y of sequence {n}")
        if i >= 0:
            close(pool[i], sr, 2 * big, f"state of sequence {n}")
        at += length
    for i in (1, 3, 4):
        assert torch.equal(pool[i], before[i])


def test_continuation_in_place_and_empty():
    axon = _axon()
    d = make((2, 177), 1, 2, 128, 64, "f32", seed=8)
    s = state(2, 2, 64, 128, 2)
    start = s.clone()
    ys = []
    for a, b in ((0, 100), (100, 100), (100, 177)):
        part = {x: (t if x in ("A_log", "dt_bias") else t[:, a:b].contiguous()) for x, t in d.items()}
        y, out = axon.gated_delta_scan(**part, state_in=s, state_out=s)
        assert out is s
        ys.append(y)
    torch.cuda.synchronize()
    y = torch.cat(ys, 1)
    for b in range(2):
        yr, sr, big = ref.delta_tokens(start[b], **rows(d, b))
        close(y[b], yr, 2 * big, "y")
        close(s[b], sr, 2 * big, "state")
    empty = {x: (t if x in ("A_log", "dt_bias") else t[:, :0].contiguous()) for x, t in d.items()}
    y, out = axon.gated_delta_scan(**empty, state_in=start)
    assert y.shape == (2, 0, 2, 64) and torch.equal(out, start)
    _, out = axon.gated_delta_scan(**empty)
    assert torch.count_nonzero(out).item() == 0


STEPS = [
    # (rows, pool, hk, hv, K, V, act)
    (1, 1, 1, 1, 64, 16, "f32"),
    (3, 5, 2, 4, 128, 128, "bf16"),
    (5, 5, 1, 3, 64, 48, "bf16"),
    (9, 20, 2, 2, 128, 240, "f32"),
    (70, 80, 8, 16, 64, 64, "bf16"),     # enough rows for several passes a wave
    (40, 41, 16, 16, 128, 112, "f32"),
]


@pytest.mark.parametrize("B,pool,hk,hv,K,V,act", STEPS)
def test_step(B, pool, hk, hv, K, V, act):
    say(f"[delta] step rows={B} of {pool} heads {hk}/{hv} K={K} V={V} {act}")
    d = make((B,), hk, hv, K, V, act, seed=B)
    s = state(pool, hv, V, K, B)
    before = s.clone()
    g = torch.Generator().manual_seed(B)
    slots = torch.randperm(pool, generator=g)[:B].int()
    if B > 2:
        slots[1], slots[2] = -1, pool
    y = torch.full((B, hv, V), 3.0, dtype=T[act]).cuda()
    out = _axon().gated_delta_step(**d, state=s, slots=slots.cuda(), y=y)
    assert out is y
    torch.cuda.synchronize()
    live = [b for b in range(B) if 0 <= int(slots[b]) < pool]
    for b in live[:12] + live[-2:]:
        i = int(slots[b])
        yr, sr, big = ref.delta_tokens(before[i], **rows(d, slice(b, b + 1)))
        close(y[b], yr[0], big, f"y[{b}]")
        close(s[i], sr, big, f"state[{i}]")
    for b in set(range(B)) - set(live):
        assert bool((y[b] == 3.0).all())
    for i in set(range(pool)) - {int(slots[b]) for b in live}:
        assert torch.equal(s[i], before[i]), f"state {i} changed"


def test_steps_continue_a_scan():
    """Packed prefill into a pool, then steps, with the norm behind both: against the recurrence
    over the whole sequences."""
    axon = _axon()
    hk, hv, K, V = 1, 2, 128, 64
    lengths, steps = [70, 3, 128], 5
    whole = [make((n + steps,), hk, hv, K, V, "f32", seed=20 + j) for j, n in enumerate(lengths)]
    par = {x: whole[0][x] for x in ("A_log", "dt_bias")}
    acts = ("q", "k", "v", "dt_raw", "beta_raw")
    z = torch.randn(sum(lengths) + 3 * steps, hv * V, generator=torch.Generator().manual_seed(1)).cuda()
    w = (1 + 0.1 * torch.randn(V, generator=torch.Generator().manual_seed(2))).cuda()
    pool = torch.zeros(6, hv, V, K).cuda()
    slots = torch.tensor([4, 0, 2], dtype=torch.int32).cuda()
    packed = {x: torch.cat([whole[j][x][:n] for j, n in enumerate(lengths)]) for x in acts}
    fresh = torch.full((3,), -1, dtype=torch.int32).cuda()
    y, _ = axon.gated_delta_scan(**packed, **par, lengths=torch.tensor(lengths, dtype=torch.int32).cuda(),
                                 state_in=pool, in_slots=fresh, state_out=pool, out_slots=slots)
    outs = [y]
    for t in range(steps):
        one = {x: torch.stack([whole[j][x][n + t] for j, n in enumerate(lengths)]) for x in acts}
        outs.append(axon.gated_delta_step(**one, **par, state=pool, slots=slots))
    o = torch.cat(outs).flatten(1)
    normed = axon.group_norm(o, hv, w, z=z, centered=False, gate="after")
    torch.cuda.synchronize()
    at = 0
    for j, n in enumerate(lengths):
        yr, sr, big = ref.delta_tokens(torch.zeros(hv, V, K), **{**rows(whole[j], slice(None)), **par})
        got = torch.cat([outs[0][at:at + n]] + [x[j:j + 1] for x in outs[1:]])
        close(got, yr, 2 * big, f"y of request {j}")
        close(pool[int(slots[j])], sr, 2 * big, f"state of request {j}")
        at += n
    want = ref.group_norm(o, hv, w, None, z, 1e-5, False, "none", "after")
    assert float((normed.double().cpu() - want).abs().max()) <= 2e-6 * (1 + float(want.abs().max()))


def test_other_stream():
    axon = _axon()
    d = make((2, 100), 1, 2, 128, 64, "bf16", seed=12)
    s0 = state(2, 2, 64, 128, 1)
    y0, o0 = axon.gated_delta_scan(**d, state_in=s0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y1, o1 = axon.gated_delta_scan(**d, state_in=s0, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(y0, y1) and torch.equal(o0, o1)


def test_captured_serving_step():
    """A packed scan (tables built in the graph) and a decode step captured once and replayed with
    other lengths, inputs and slots, eager work between the replays; every replay equals the eager
    call bit for bit."""
    axon = _axon()
    hk, hv, K, V, total, n = 1, 2, 128, 64, 200, 3
    d = make((total,), hk, hv, K, V, "bf16", seed=13)
    one = make((n,), hk, hv, K, V, "bf16", seed=14)
    one.update({x: d[x] for x in ("A_log", "dt_bias")})
    lengths = torch.tensor([100, 50, 50], dtype=torch.int32).cuda()
    slots = torch.tensor([2, 0, 3], dtype=torch.int32).cuda()
    pool = state(4, hv, V, K, 3)
    y = torch.zeros(total, hv, V, dtype=torch.bfloat16).cuda()
    y1 = torch.zeros(n, hv, V, dtype=torch.bfloat16).cuda()

    def call():
        axon.gated_delta_scan(**d, lengths=lengths, state_in=pool, in_slots=slots, y=y,
                              state_out=pool, out_slots=slots)
        axon.gated_delta_step(**one, state=pool, slots=slots, y=y1)

    start = pool.clone()
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    pool.copy_(start)
    with torch.cuda.graph(graph):
        call()
    for rep, (ls, sl) in enumerate([([100, 50, 50], [2, 0, 3]), ([0, 199, 1], [1, 3, 2]),
                                    ([64, 0, 20], [0, -1, 1])]):
        lengths.copy_(torch.tensor(ls, dtype=torch.int32))
        slots.copy_(torch.tensor(sl, dtype=torch.int32))
        d["v"].copy_(torch.randn(total, hv, V))
        got = []
        for run in (graph.replay, call):
            pool.copy_(start)
            y.zero_()
            y1.zero_()
            torch.cuda.synchronize()
            run()
            torch.cuda.synchronize()
            got.append((y.clone(), y1.clone(), pool.clone()))
        for a, b, what in zip(*got, ("y", "step", "pool")):
            assert torch.equal(a, b), f"replay {rep}: {what} differs"


def test_refused_tensors():
    axon = _axon()
    d = make((2, 10), 1, 2, 64, 32, "f32", seed=1)
    cases = [
        dict(q=d["q"].to(torch.float16)), dict(k=d["k"].to(torch.bfloat16)), dict(v=d["v"].cpu()),
        dict(dt_raw=d["dt_raw"][:, :9]), dict(q=d["q"].transpose(0, 1)),
        dict(k=d["k"][:, :1].expand(2, 10, 1, 64)), dict(A_log=d["A_log"].double()),
        dict(state_in=torch.zeros(1, 2, 32, 64).cuda()), dict(state_in=torch.zeros(2, 2, 64, 32).cuda()),
        dict(in_slots=torch.zeros(3, dtype=torch.int32).cuda()),
        dict(in_slots=torch.zeros(2, dtype=torch.int64).cuda()),
        dict(out_slots=torch.zeros(2, dtype=torch.int32).cuda()), dict(eps=0.0), dict(dt_min=-1.0),
        dict(scale=float("nan")), dict(workspace=torch.empty(16, dtype=torch.uint8).cuda()),
        dict(y=d["v"]), dict(lengths=torch.tensor([5, 5], dtype=torch.int32).cuda()),
    ]
    for over in cases:
        with pytest.raises((TypeError, ValueError, axon.AxonError)):
            axon.gated_delta_scan(**{**d, **over})
    p = {x: (t if x in ("A_log", "dt_bias") else t.flatten(0, 1)) for x, t in d.items()}
    with pytest.raises(ValueError):
        axon.gated_delta_scan(**p, tables=axon.sequence_tables(
            torch.tensor([5, 5], dtype=torch.int32).cuda(), 20, block=32))
    with pytest.raises((ValueError, axon.AxonError)):
        axon.gated_delta_step(**p, state=torch.zeros(3, 2, 32, 64).cuda())
    with pytest.raises((ValueError, TypeError)):
        axon.gated_delta_step(**p, state=None)
    torch.cuda.synchronize()


def test_two_calls_at_once():
    """Two scans that share inputs and the pool, each with its own workspace and slots, on two
    streams: both as if alone. One is split into segments, the other packed."""
    axon = _axon()
    hk, hv, K, V, L = 1, 2, 128, 128, 4096
    d = make((1, L), hk, hv, K, V, "bf16", seed=31)
    p = {x: (t if x in ("A_log", "dt_bias") else t.flatten(0, 1)) for x, t in d.items()}
    lengths = torch.tensor([L // 2 + 5, 0, L // 4], dtype=torch.int32).cuda()
    pool = state(6, hv, V, K, 3)
    one = torch.tensor([2], dtype=torch.int32).cuda()
    three = torch.tensor([0, 5, 3], dtype=torch.int32).cuda()
    y = [torch.zeros(1, L, hv, V, dtype=torch.bfloat16).cuda(), torch.zeros(L, hv, V, dtype=torch.bfloat16).cuda()]

    def a(stream=None):
        axon.gated_delta_scan(**d, state_in=pool, in_slots=one, y=y[0], state_out=pool, out_slots=one,
                              stream=stream)

    def b(stream=None):
        axon.gated_delta_scan(**p, lengths=lengths, state_in=pool, in_slots=three, y=y[1], state_out=pool,
                              out_slots=three, stream=stream)

    start = pool.clone()
    a()
    b()
    torch.cuda.synchronize()
    want = [t.clone() for t in (*y, pool)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for rep in range(3):
        pool.copy_(start)
        for t in y:
            t.zero_()
        torch.cuda.synchronize()
        a(streams[0])
        b(streams[1])
        torch.cuda.synchronize()
        for got, w, what in zip((*y, pool), want, ("y", "packed y", "pool")):
            assert torch.equal(got, w), f"run {rep}: {what} differs"


@pytest.mark.parametrize("where", ["host", "spread"])
def test_refused_workspace(where):
    """A workspace that the kernels could not use is refused before any launch."""
    axon = _axon()
    d = make((2, 10), 1, 2, 64, 32, "f32", seed=1)
    need = axon.gated_delta_workspace_bytes(2, 20, 1, 2, 64, 32)
    ws = (torch.empty(need, dtype=torch.uint8) if where == "host"
          else torch.empty(2 * need, dtype=torch.uint8).cuda()[::2])
    with pytest.raises(ValueError):
        axon.gated_delta_scan(**d, workspace=ws)
