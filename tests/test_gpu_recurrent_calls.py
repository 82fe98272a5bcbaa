"""Calls of the gated linear recurrence, the causal convolution and the head norm on the GPU that the
tests of their numbers do not make: what is refused, long chains of few channels, workspaces that are
given and shared, tables with any contents, tables that are dropped while they are in use."""
from __future__ import annotations

import pytest

from gpu_util import say
from test_gpu_linear import compare, grad, make, parts_of, sequence, states

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


# ---- What is refused ----------------------------------------------------------------------------

def _linear():
    z = make((2, 70), 24, seed=1)
    return dict(**z, state_in=states(2, 24))


LINEAR_REFUSED = [
    ("x of the other type", lambda z: z.update(x=z["x"].bfloat16()), TypeError),
    ("half", lambda z: z.update({k: z[k].half() for k in ("x", "dt_raw", "in_raw")}), (TypeError, ValueError)),
    ("dt_raw shorter", lambda z: z.update(dt_raw=z["dt_raw"][:, :-1]), ValueError),
    ("in_raw on the host", lambda z: z.update(in_raw=z["in_raw"].cpu()), ValueError),
    ("x expanded", lambda z: z.update(x=z["x"][:1].expand(2, 70, 24)), ValueError),
    ("channels apart", lambda z: z.update(x=torch.zeros(2, 70, 48, device="cuda")[..., ::2]), ValueError),
    ("rows unevenly apart", lambda z: z.update(x=torch.zeros(2, 80, 24, device="cuda")[:, :70]), ValueError),
    ("A_log in bf16", lambda z: z.update(A_log=z["A_log"].bfloat16()), TypeError),
    ("A_log apart", lambda z: z.update(A_log=torch.zeros(48, device="cuda")[::2]), ValueError),
    ("dt_bias longer", lambda z: z.update(dt_bias=torch.zeros(25, device="cuda")), ValueError),
    ("in_bias alone", lambda z: z.update(in_raw=None), ValueError),
    ("gate", lambda z: z.update(gate="tanh"), ValueError),
    ("input scale", lambda z: z.update(input_scale=None), ValueError),
    ("lengths of a batch", lambda z: z.update(lengths=torch.tensor([70, 70], dtype=torch.int32).cuda()),
     ValueError),
    ("states of another width", lambda z: z.update(state_in=states(2, 25)), ValueError),
    ("states in bf16", lambda z: z.update(state_in=states(2, 24).bfloat16()), TypeError),
    ("too few states", lambda z: z.update(state_in=states(1, 24)), Exception),
    ("slots in 64 bits", lambda z: z.update(in_slots=torch.zeros(2, dtype=torch.int64).cuda()),
     (TypeError, ValueError)),
    ("too many slots", lambda z: z.update(in_slots=torch.zeros(3, dtype=torch.int32).cuda()), ValueError),
    ("slots without a pool", lambda z: z.update(out_slots=torch.zeros(2, dtype=torch.int32).cuda()),
     ValueError),
    ("y of another shape", lambda z: z.update(y=torch.zeros(140, 24, device="cuda")), ValueError),
    ("y over x", lambda z: z.update(y=z["x"]), Exception),
    ("checkpoints of another size", lambda z: z.update(checkpoints=torch.zeros(3, 24, device="cuda")),
     ValueError),
    ("workspace too small", lambda z: z.update(x=torch.zeros(2, 700, 24, device="cuda"),
                                               dt_raw=torch.zeros(2, 700, 24, device="cuda"),
                                               in_raw=torch.zeros(2, 700, 24, device="cuda"),
                                               workspace=torch.zeros(8, dtype=torch.uint8, device="cuda")),
     Exception),
    ("workspace on the host", lambda z: z.update(workspace=torch.zeros(1 << 16, dtype=torch.uint8)), ValueError),
]


@pytest.mark.parametrize("what,change,error", LINEAR_REFUSED, ids=[c[0] for c in LINEAR_REFUSED])
def test_linear_refuses(what, change, error):
    axon = _axon()
    z = _linear()
    axon.linear_scan(**z)
    change(z)
    with pytest.raises(error):
        axon.linear_scan(**z)


def test_linear_backward_and_step_refuse():
    axon = _axon()
    z = make((2, 70), 24, seed=1)
    p, dy = axon.linear_checkpoints(z["x"]), grad((2, 70), 24, "f32")
    axon.linear_scan_backward(dy, **z, checkpoints=p)
    for change in (dict(checkpoints=p[:-1]), dict(checkpoints=p.double()), dict(dstate_out=states(3, 24)),
                   dict(dstate_out=states(2, 24).cpu())):
        with pytest.raises((TypeError, ValueError)):
            axon.linear_scan_backward(dy, **z, **{**dict(checkpoints=p), **change})
    for bad in (dy[:, :-1], dy.bfloat16(), dy.cpu(), dy[:1].expand(2, 70, 24)):
        with pytest.raises((TypeError, ValueError)):
            axon.linear_scan_backward(bad, **z, checkpoints=p)
    one = {k: v[:, 0].contiguous() if v.dim() == 3 else v for k, v in z.items()}
    pool = states(5, 24)
    axon.linear_step(**one, state=pool)
    for change in (dict(state=pool[:1]), dict(state=pool.bfloat16()), dict(state=pool[:, :-1]),
                   dict(slots=torch.zeros(3, dtype=torch.int32).cuda()),
                   dict(y=torch.zeros(2, 24)), dict(x=z["x"]), dict(state=pool, y=pool[:2])):
        with pytest.raises(Exception):
            axon.linear_step(**{**one, **dict(state=pool), **change})


def test_tables_refuse():
    axon = _axon()
    z = make((100,), 24, seed=1)
    n = torch.tensor([40, 60], dtype=torch.int32).cuda()
    good = axon.sequence_tables(n, 100)
    axon.linear_scan(**z, tables=good)
    for tables in (axon.sequence_tables(n, 101), axon.sequence_tables(n, 100, block=128), good.buffer):
        with pytest.raises((TypeError, ValueError)):
            axon.linear_scan(**z, tables=tables)
        with pytest.raises((TypeError, ValueError)):
            axon.causal_conv(z["x"], torch.zeros(24, 4, device="cuda"), tables=tables)
    with pytest.raises(ValueError):
        axon.linear_scan(**z, tables=good, lengths=n)
    with pytest.raises(ValueError):
        axon.linear_scan(**z, lengths=n.cpu())
    with pytest.raises((TypeError, ValueError)):
        axon.linear_scan(**z, lengths=n.long())


def test_conv_refuses():
    axon = _axon()
    x, w = make((2, 30), 24, seed=1)["x"], torch.zeros(24, 4, device="cuda")
    b, cache = torch.zeros(24, device="cuda"), torch.zeros(2, 3, 24, device="cuda")
    axon.causal_conv(x, w, b, cache_in=cache)
    for change in (dict(conv_w=w[:, :3]), dict(conv_w=w.t()), dict(conv_w=w.bfloat16()), dict(conv_b=b[:-1]),
                   dict(activation="relu"), dict(cache_in=cache[:, :2]), dict(cache_in=cache[:1]),
                   dict(y=x), dict(cache_out=cache[:1]), dict(x=x.double()),
                   dict(out_slots=torch.zeros(2, dtype=torch.int32).cuda())):
        with pytest.raises(Exception):
            axon.causal_conv(**{**dict(x=x, conv_w=w, conv_b=b, cache_in=cache), **change})
    for change in (dict(dy=x[:, 1:]), dict(dy=x.bfloat16()), dict(cache_in=cache[:1]),
                   dict(dcache_out=cache[:1]), dict(workspace=torch.zeros(1, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(Exception):
            axon.causal_conv_backward(**{**dict(dy=x, x=x, conv_w=w, conv_b=b), **change})
    for change in (dict(cache=cache[:1]), dict(x=x), dict(slots=torch.zeros(1, dtype=torch.int32).cuda())):
        with pytest.raises(Exception):
            axon.causal_conv_step(**{**dict(x=x[:, 0].contiguous(), conv_w=w, conv_b=b, cache=cache), **change})


def test_rotate_refuses():
    axon = _axon()
    q, k = torch.zeros(9, 4, 16, device="cuda"), torch.zeros(9, 2, 16, device="cuda")
    z = dict(q=q, k=k, positions=torch.zeros(9, dtype=torch.int32).cuda(),
             freqs=torch.ones(8, dtype=torch.float64).cuda(), q_weight=torch.ones(16, device="cuda"))
    axon.norm_rotate(**z)
    for change in (dict(k=k[:8]), dict(k=k[..., :14]), dict(k=k.bfloat16()), dict(k=k[:, :0]),
                   dict(positions=z["positions"].long()), dict(positions=z["positions"][:8]),
                   dict(freqs=z["freqs"].float()), dict(freqs=torch.ones(9, dtype=torch.float64).cuda()),
                   dict(freqs=z["freqs"][:0]), dict(q_weight=torch.ones(15, device="cuda")), dict(eps=-1.0),
                   dict(eps=float("nan")), dict(k=None, k_weight=z["q_weight"]), dict(q_out=q[:8]),
                   dict(q_out=k), dict(k_out=q), dict(q=torch.zeros(9, 4, 15, device="cuda"), k=None),
                   dict(q=torch.zeros(9, 4, 258, device="cuda"), k=None, q_weight=None)):
        with pytest.raises(Exception):
            axon.norm_rotate(**{**z, **change})
    with pytest.raises(ValueError):
        axon.norm_rotate_backward(q, None, **z)
    with pytest.raises((TypeError, ValueError)):
        axon.norm_rotate_backward(q.bfloat16(), k, **z)
    with pytest.raises(Exception):
        axon.norm_rotate_backward(q, k, **z, workspace=torch.zeros(4, dtype=torch.uint8, device="cuda"))


# ---- Long chains of few channels ----------------------------------------------------------------

CHAINS = [
    # lengths of a packed buffer, or one of a uniform batch (B, L); channels
    ((1, 7001), 40),
    ((2, 6208), 130),
    ([3000, 1, 0, 64, 4500, 191], 8),
    ([7000], 71),
]


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("shape,E", CHAINS)
def test_long_chains(shape, E, act):
    """Enough tiles in a row, of few channels, that all waves of a tile look at the tiles in front."""
    say(f"[calls] chain {shape} x {E} {act}")
    axon = _axon()
    packed = isinstance(shape, list)
    lead, N = ((sum(shape),), len(shape)) if packed else (shape, shape[0])
    z = make(lead, E, act, seed=E, rate=(-8.0, 0.0))
    s0, ds, dy = states(N, E, 1), states(N, E, 2), grad(lead, E, act)
    tables = axon.sequence_tables(torch.tensor(shape, dtype=torch.int32).cuda(), lead[0]) if packed else None
    p = axon.linear_checkpoints(z["x"], tables=tables)
    y, s1 = axon.linear_scan(**z, tables=tables, state_in=s0, checkpoints=p)
    grads = axon.linear_scan_backward(dy, **z, tables=tables, checkpoints=p, dstate_out=ds)
    torch.cuda.synchronize()
    compare(z, parts_of(shape) if packed else list(range(N)), s0, ds, dy, y, s1, grads, "sigmoid", "sqrt")
    for _ in range(5):
        y2, s2 = axon.linear_scan(**z, tables=tables, state_in=s0)
        again = axon.linear_scan_backward(dy, **z, tables=tables, checkpoints=p, dstate_out=ds)
        torch.cuda.synchronize()
        assert torch.equal(y, y2) and torch.equal(s1, s2)
        for a, b in zip(grads, again):
            assert torch.equal(a, b)


def test_nan_in_a_long_chain():
    """A state that is not finite is handed on as such, to the end of its sequence and no further."""
    axon = _axon()
    lengths, E = [6000, 700], 24
    z = make((6700,), E, seed=2)
    z["x"][100, 3] = float("nan")
    z["x"][200, 5] = float("inf")
    y, s = axon.linear_scan(**z, lengths=torch.tensor(lengths, dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    assert bool(y[100:6000, 3].isnan().all()) and bool(torch.isfinite(y[:100, 3]).all())
    assert not bool(torch.isfinite(y[200:201, 5]).any())
    rest = [c for c in range(E) if c not in (3, 5)]
    assert bool(torch.isfinite(y[:, rest]).all()) and bool(torch.isfinite(y[6000:]).all())
    r = sequence(z, torch.zeros(E), slice(6000, 6700), "sigmoid", "sqrt")
    ref.within(y[6000:], r.y, r.bound, "y")


# ---- Workspaces, tables and streams -------------------------------------------------------------

def test_given_workspace():
    """One workspace for call after call of other sizes, whatever it holds."""
    axon = _axon()
    ws = torch.full((1 << 23,), 0xA5, dtype=torch.uint8, device="cuda")
    for B, L, E in ((1, 900, 70), (2, 7000, 33), (3, 65, 200), (1, 900, 70)):
        z, dy = make((B, L), E, seed=L), grad((B, L), E, "f32")
        p = axon.linear_checkpoints(z["x"])
        want = axon.linear_scan(**z, checkpoints=p)
        back = axon.linear_scan_backward(dy, **z, checkpoints=p)
        got = axon.linear_scan(**z, workspace=ws)
        gback = axon.linear_scan_backward(dy, **z, checkpoints=p, workspace=ws)
        torch.cuda.synchronize()
        for a, b in zip([*want, *back], [*got, *gback]):
            assert torch.equal(a, b)
    w = torch.ones(70, 4, device="cuda")
    x = make((1, 900), 70, seed=1)["x"]
    for a, b in zip(axon.causal_conv_backward(x, x, w), axon.causal_conv_backward(x, x, w, workspace=ws)):
        assert torch.equal(a, b)


def test_two_graphs_share_a_workspace():
    """Two captured graphs with one workspace, replayed one after the other, with eager calls between."""
    axon = _axon()
    ws = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    zs = [make((1, 2000), 64, "bf16", seed=1), make((2, 700), 200, "f32", seed=2)]
    want = [axon.linear_scan(**z) for z in zs]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for z in zs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(axon.linear_scan(**z, workspace=ws))
        graphs.append(g)
    for turn in range(4):
        for o in outs:
            for t in o:
                t.fill_(float("nan"))
        for j in (0, 1, 1, 0) if turn % 2 else (1, 0):
            graphs[j].replay()
            if turn > 1:
                axon.linear_scan(**zs[1 - j], workspace=ws)
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o[0], w[0]) and torch.equal(o[1], w[1])


@pytest.mark.parametrize("seed", range(3))
def test_tables_with_any_contents(seed):
    """Tables whose entries are not of sequence_tables: results mean nothing, but nothing outside the
    outputs is written, and rows of no sequence stay."""
    axon = _axon()
    total, E, N = 1500, 40, 5
    g = torch.Generator().manual_seed(seed)
    tables = axon.sequence_tables(torch.tensor([300] * 5, dtype=torch.int32).cuda(), total)
    reach = [1 << 31, 2000, 40][seed]
    tables.buffer.copy_(torch.randint(-reach, reach, tables.buffer.shape, generator=g).int())
    z = make((total,), E, seed=1)
    big = torch.full((total + 200, E), 9.0, device="cuda")
    y = big[100:100 + total]
    pool = torch.full((N + 8, E), 9.0, device="cuda")
    points = torch.full((total // 64 + N + 8, E), 9.0, device="cuda")
    axon.linear_scan(**z, tables=tables, y=y, state_out=pool[4:4 + N], checkpoints=points[4:-4])
    d = axon.linear_scan_backward(y, **z, tables=tables, checkpoints=points[4:-4])
    axon.causal_conv(z["x"], torch.ones(E, 4, device="cuda"), tables=tables, y=torch.zeros_like(y))
    axon.causal_conv_backward(z["x"], z["x"], torch.ones(E, 4, device="cuda"), tables=tables)
    torch.cuda.synchronize()
    assert d.dx.shape == y.shape
    for t in (big[:100], big[100 + total:], pool[:4], pool[4 + N:], points[:4], points[-4:]):
        assert bool((t == 9).all())


def test_tables_dropped_in_use():
    """Tables and inputs of a call on another stream that are dropped before it has run."""
    axon = _axon()
    z = make((900,), 64, "bf16", seed=1)
    n = torch.tensor([400, 500], dtype=torch.int32).cuda()
    w = torch.ones(64, 4, device="cuda")
    want, cwant = axon.linear_scan(**z, lengths=n), axon.causal_conv(z["x"], w, lengths=n)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    tables = axon.sequence_tables(n, 900)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    got = axon.linear_scan(**z, tables=tables, stream=side)
    cgot = axon.causal_conv(z["x"], w, tables=tables, stream=side)
    count = tables.buffer.numel()
    del tables
    junk = [torch.full((count,), 7, dtype=torch.int32, device="cuda") for _ in range(64)]
    torch.cuda.synchronize()
    for a, b in zip([*got, *cgot], [*want, *cwant]):
        assert torch.equal(a, b)
    del junk


def test_stream_of_the_wrong_kind():
    axon = _axon()
    z = make((1, 70), 24, seed=1)
    with pytest.raises(Exception):
        axon.linear_scan(**z, stream=7.5)


# ---- Wide convolutions --------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("E", [65540, 65538, 65537])
def test_conv_of_many_waves(E, dtype):
    """Enough waves that a lane takes four, two or one channels, as the rows' alignment allows."""
    import test_gpu_conv as conv

    say(f"[calls] convolution {E} {dtype}")
    axon = _axon()
    lengths, spare = [5, 0, 64, 1, 70, 2, 3, 65], 7
    total, N = sum(lengths) + spare, len(lengths)
    z, dy = conv.make((total,), E, dtype, seed=1), conv.grad((total,), E, dtype)
    z["x"][total - spare:] = float("nan")
    dy[total - spare:] = float("nan")
    tables = axon.sequence_tables(torch.tensor(lengths, dtype=torch.int32).cuda(), total)
    c0, dc = conv.caches(N, E), conv.caches(N, E, 1)
    y, c1 = axon.causal_conv(**z, activation="silu", cache_in=c0, tables=tables)
    grads = axon.causal_conv_backward(dy, **z, activation="silu", cache_in=c0, dcache_out=dc, tables=tables)
    torch.cuda.synchronize()
    conv.compare(z, parts_of(lengths), c0, dc, dy, y, c1, grads, "silu")
    assert not y[total - spare:].any() and not grads.dx[total - spare:].any()


# ---- Wide steps ---------------------------------------------------------------------------------

@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("E,apart", [(16388, 0), (16388, 4), (16388, 2), (16385, 0)])
def test_step_of_a_large_batch(E, apart, act):
    """Rows enough that a thread takes four channels, where their alignment allows it."""
    axon = _axon()
    n, slots = 65, 70
    z = make((n,), E + apart, act, seed=E)
    z = {k: v[..., :E] if v.dim() == 2 else v[:E].contiguous() for k, v in z.items()}
    pool = states(slots, E)
    at = torch.randperm(slots, generator=torch.Generator().manual_seed(1))[:n].int()
    at[7], at[20] = -1, slots
    before, y = pool.clone(), torch.full((n, E), 7.0, dtype=T[act], device="cuda")
    axon.linear_step(**z, state=pool, slots=at.cuda(), y=y)
    torch.cuda.synchronize()
    rows = [j for j in range(n) if 0 <= int(at[j]) < slots]
    for j in rows[::8]:
        r = sequence(z, before[int(at[j])], slice(j, j + 1), "sigmoid", "sqrt")
        ref.within(y[j:j + 1], r.y, r.bound, f"y {j}")
        ref.within(pool[int(at[j])], r.state, r.state_bound, f"state {j}")
    idle = [j for j in range(slots) if j not in [int(at[i]) for i in rows]]
    assert torch.equal(pool[idle], before[idle]) and bool((y[[7, 20]] == 7).all())


# ---- The most sequences, other ways to a stream, gradients recorded --------------------------------

@pytest.mark.parametrize("packed", [True, False])
def test_the_most_sequences(packed):
    """65535 sequences of one token: a scan is a step."""
    axon = _axon()
    N, E = 65535, 6
    z = make((N,), E, seed=1)
    s0 = states(N, E)
    lead = z if packed else {k: v[:, None] if v.dim() == 2 else v for k, v in z.items()}
    x = lead["x"]
    n = torch.ones(N, dtype=torch.int32, device="cuda") if packed else None
    tables = axon.sequence_tables(n, N) if packed else None
    p = axon.linear_checkpoints(x, tables=tables)
    y, s1 = axon.linear_scan(**lead, tables=tables, state_in=s0, checkpoints=p)
    d = axon.linear_scan_backward(x, **lead, tables=tables, checkpoints=p)
    c, c1 = axon.causal_conv(x, torch.ones(E, 4, device="cuda"), tables=tables)
    pool = s0.clone()
    y2 = axon.linear_step(**z, state=pool)
    torch.cuda.synchronize()
    assert torch.equal(y.reshape(N, E), s1) and torch.equal(c.reshape(N, E), z["x"])
    assert torch.equal(c1[:, 2], z["x"]) and not c1[:, :2].any()
    # one token by the step's and by the scan's form: the bounds of both
    for j in (0, 1, 191, 192, 32768, 65533, 65534):
        r = sequence(z, s0[j], slice(j, j + 1), "sigmoid", "sqrt")
        ref.within(y.reshape(N, E)[j:j + 1], r.y, r.bound, f"scan {j}")
        ref.within(y2[j:j + 1], r.y, r.bound, f"step {j}")
        want = r.backward(z["x"][j:j + 1], torch.zeros(E))
        ref.within(d.dx.reshape(N, E)[j:j + 1], *want["dx"], f"dx {j}")
    assert torch.equal(pool, y2)


def test_tables_of_another_stream():
    """Tables of one stream in calls on another, and in a captured graph, dropped while they run."""
    axon = _axon()
    z = make((900,), 64, "bf16", seed=1)
    n = torch.tensor([400, 500], dtype=torch.int32).cuda()
    want = axon.linear_scan(**z, lengths=n)
    tables = axon.sequence_tables(n, 900)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = axon.linear_scan(**z, tables=tables)
    for _ in range(3):
        captured[0].fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(captured[0], want[0]) and torch.equal(captured[1], want[1])
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        got = axon.linear_scan(**z, tables=tables)
    count = tables.buffer.numel()
    del graph, tables
    junk = [torch.full((count,), 7, dtype=torch.int32, device="cuda") for _ in range(64)]
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    del junk


def test_tensors_that_want_gradients():
    """The calls record no graph, whatever their inputs want, and give the same in inference mode."""
    axon = _axon()
    z = make((1, 300), 40, seed=1)
    want = axon.linear_scan(**z)
    grads = {k: v.clone().requires_grad_() for k, v in z.items()}
    got = axon.linear_scan(**grads)
    p = axon.linear_checkpoints(grads["x"])
    axon.linear_scan(**grads, checkpoints=p)
    back = axon.linear_scan_backward(got[0], **grads, checkpoints=p)
    with torch.inference_mode():
        other = axon.linear_scan(**z)
    torch.cuda.synchronize()
    for t in (*got, *back):
        assert not t.requires_grad and t.grad_fn is None
    for o in (got, other):
        assert torch.equal(o[0], want[0]) and torch.equal(o[1], want[1])
