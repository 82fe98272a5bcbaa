"""The head norm with position rotation on the GPU against its plain 64-bit form, forward and
backward: head sizes that are no power of two, parts of heads rotated, far and negative positions,
parts of one projection, in place, streams, graphs, and in front of the gated delta scan."""
from __future__ import annotations

import pytest

from gpu_util import say

torch = pytest.importorskip("torch")

import recurrent_ref as ref  # noqa: E402
from test_gpu_linear import T, _axon, _gpu  # noqa: E402,F401

pytestmark = pytest.mark.gpu


def make(rows, hq, hk, D, R, act="f32", seed=0, far=5000, weights=True):
    g = torch.Generator().manual_seed(seed)

    def n(*s):
        return torch.randn(*s, generator=g)

    z = dict(q=n(rows, hq, D).to(T[act]).cuda(), k=n(rows, hk, D).to(T[act]).cuda() if hk else None,
             positions=torch.randint(-far, far, (rows,), generator=g).int().cuda(),
             freqs=(10000.0 ** (-2 * torch.arange(R // 2, dtype=torch.float64) / R)).cuda())
    kw = dict(q_weight=(1 + 0.3 * n(D)).cuda() if weights else None,
              k_weight=(1 + 0.3 * n(D)).cuda() if weights and hk else None)
    return z, kw


def compare(z, kw, eps, inter, out, d=None, grads=None):
    for name, j in (("q", 0), ("k", 1)):
        if z[name] is None:
            assert out[j] is None
            continue
        args = (z["positions"], z["freqs"], kw[f"{name}_weight"], eps, inter)
        ref.within(out[j], *ref.norm_rotate(z[name], *args), name)
        if grads is not None:
            dx, dxb, dw, dwb = ref.norm_rotate_backward(d[j], z[name], *args)
            ref.within(grads[j], dx, dxb, f"d{name}")
            if kw[f"{name}_weight"] is not None:
                ref.within(grads[2 + j], dw, dwb, f"d{name}_weight")
            else:
                assert grads[2 + j] is None


CASES = [
    # (rows, hq, hk, D, R, act, interleaved, weights)
    (1, 1, 1, 2, 2, "f32", False, True), (3, 2, 1, 6, 4, "bf16", True, True),
    (5, 1, 0, 64, 64, "f32", False, True), (7, 8, 2, 128, 128, "bf16", False, True),
    (33, 3, 3, 96, 48, "f32", True, True), (40, 10, 2, 96, 96, "bf16", False, False),
    (17, 4, 1, 256, 64, "f32", False, True), (9, 5, 5, 254, 100, "bf16", True, True),
    (64, 32, 8, 128, 128, "bf16", True, True), (31, 2, 2, 130, 130, "f32", False, True),
    (50, 7, 1, 80, 40, "bf16", False, True), (2, 1, 1, 256, 256, "bf16", False, True),
    (130, 16, 4, 64, 16, "f32", False, False), (3, 33, 11, 32, 30, "f32", True, True),
    (6000, 2, 1, 16, 16, "bf16", False, True),
]


@pytest.mark.parametrize("rows,hq,hk,D,R,act,inter,weights", CASES)
def test_forward_and_backward(rows, hq, hk, D, R, act, inter, weights):
    say(f"[rotate] {rows} x {hq}+{hk} x {D}/{R} {act} interleaved={inter}")
    axon = _axon()
    z, kw = make(rows, hq, hk, D, R, act, seed=rows + D, weights=weights)
    g = torch.Generator().manual_seed(1)
    d = [torch.randn(rows, h, D, generator=g).to(T[act]).cuda() if h else None for h in (hq, hk)]
    out = axon.norm_rotate(**z, **kw, eps=1e-5, interleaved=inter)
    grads = axon.norm_rotate_backward(*d, **z, **kw, eps=1e-5, interleaved=inter)
    torch.cuda.synchronize()
    compare(z, kw, 1e-5, inter, out, d, grads)


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("D,extra", [(64, 0), (64, 8), (64, 3), (48, 0), (36, 2)])
def test_parts_of_one_projection(D, extra, act):
    axon = _axon()
    rows, hq, hk = 41, 6, 2
    big, kw = make(rows, 1, 0, (hq + 2 * hk) * D + extra, 2, act, seed=3)
    z, kw = make(rows, hq, hk, D, D // 2, act, seed=4)
    flat = big["q"][:, 0, extra:]
    z["q"] = flat[:, :hq * D].unflatten(1, (hq, D))
    z["k"] = flat[:, hq * D:(hq + hk) * D].unflatten(1, (hk, D))
    g = torch.Generator().manual_seed(1)
    wide = torch.randn(rows, hq + hk, D, generator=g).to(T[act]).cuda()
    d = [wide[:, :hq], wide[:, hq:]]
    out = axon.norm_rotate(**z, **kw)
    grads = axon.norm_rotate_backward(*d, **z, **kw)
    torch.cuda.synchronize()
    compare(z, kw, 1e-6, False, out, d, grads)


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_in_place_and_batches(act):
    """(B, L, heads, D) with positions (B, L); outputs over the inputs."""
    axon = _axon()
    z, kw = make(6 * 20, 4, 2, 64, 64, act, seed=2)
    out = axon.norm_rotate(**z, **kw)
    b = {k: v if k == "freqs" else v.unflatten(0, (6, 20)) for k, v in z.items()}
    again = axon.norm_rotate(**b, **kw)
    q, k = b["q"].clone(), b["k"].clone()
    got = axon.norm_rotate(q, k, b["positions"], b["freqs"], **kw, q_out=q, k_out=k)
    torch.cuda.synchronize()
    assert got[0] is q and got[1] is k and again[0].shape == (6, 20, 4, 64)
    for a, c, o in zip(out, again, got):
        assert torch.equal(a, c.flatten(0, 1)) and torch.equal(c, o)


def test_far_positions():
    """Positions up to the ends of int32: the angle is reduced before it is rounded."""
    axon = _axon()
    z, kw = make(8, 2, 1, 64, 64, seed=5)
    z["positions"] = torch.tensor([0, 1, -1, 1 << 20, (1 << 30) + 7, 2 ** 31 - 1, -2 ** 31, 12345678],
                                  dtype=torch.int32).cuda()
    out = axon.norm_rotate(**z, **kw)
    torch.cuda.synchronize()
    # p freqs / (2 pi) in 64 bits: off by 2^31 / (2 pi) 2^-52 turns = 8e-8 turns, 5e-7 radians at most
    for name, got in zip("qk", out):
        args = (z["positions"], z["freqs"], kw[f"{name}_weight"], 1e-6, False)
        want, off = ref.norm_rotate(z[name], *args)
        turned = ref.norm_rotate(z[name], torch.zeros_like(z["positions"]), *args[1:])[0]
        off = off + 5e-7 * ref.pair_size(turned, 64, False)
        ref.within(got, want, off, name)


def test_no_rows_and_zero_heads():
    axon = _axon()
    z, kw = make(0, 2, 1, 64, 64)
    out = axon.norm_rotate(**z, **kw)
    g = axon.norm_rotate_backward(out[0], out[1], **z, **kw)
    torch.cuda.synchronize()
    assert out[0].shape == (0, 2, 64) and not g.dq_weight.any() and not g.dk_weight.any()
    z, kw = make(3, 2, 1, 64, 64)
    z["q"] = torch.zeros_like(z["q"])
    out = axon.norm_rotate(**z, **kw)
    torch.cuda.synchronize()
    assert not out[0].any() and torch.isfinite(out[1]).all()


def test_nan_stays_in_its_head():
    axon = _axon()
    z, kw = make(9, 4, 2, 48, 48, seed=7)
    want = axon.norm_rotate(**z, **kw)
    z["q"][3, 1, 5] = float("nan")
    z["k"][8, 0, 40] = float("inf")
    out = axon.norm_rotate(**z, **kw)
    torch.cuda.synchronize()
    bad = torch.zeros(9, 4, dtype=torch.bool)
    bad[3, 1] = True
    assert bool(torch.isnan(out[0][3, 1]).all()) and torch.equal(out[0].cpu()[~bad], want[0].cpu()[~bad])
    bad = torch.zeros(9, 2, dtype=torch.bool)
    bad[8, 0] = True
    assert torch.equal(out[1].cpu()[~bad], want[1].cpu()[~bad])


def test_weight_sums_over_many_rows():
    """300000 alike rows: the weights' gradients are sums of equal terms and do not drift."""
    axon = _axon()
    rows, D = 300_000, 32
    q = torch.ones(rows, 1, D, device="cuda")
    pos = torch.zeros(rows, dtype=torch.int32, device="cuda")
    g = axon.norm_rotate_backward(q, None, q, None, pos, torch.ones(4, dtype=torch.float64).cuda(),
                                  q_weight=torch.ones(D).cuda(), eps=0.0)
    torch.cuda.synchronize()
    # terms of 1 within 24 u (the norm of 32 equal values), and one rounding
    assert bool(((g.dq_weight - rows).abs() <= rows * 26 * ref.U).all())


def test_streams_graphs_and_same_results():
    axon = _axon()
    z, kw = make(700, 8, 2, 128, 64, "bf16", seed=1)
    d = [torch.randn_like(z["q"]), torch.randn_like(z["k"])]

    def work(stream=None):
        return [*axon.norm_rotate(**z, **kw, stream=stream),
                *axon.norm_rotate_backward(*d, **z, **kw, stream=stream)]

    want = work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = work()
    for shift in (0, 1, 700):
        z["positions"].add_(shift)
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


def test_rows_beyond_32_bits():
    axon = _axon()
    rows, D = 140_000, 128
    g = torch.Generator(device="cuda").manual_seed(0)
    q = torch.empty(rows, 128, D, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    pos = torch.arange(rows, dtype=torch.int32, device="cuda")
    freqs = (10000.0 ** (-torch.arange(64, dtype=torch.float64) / 64)).cuda()
    w = torch.ones(D, device="cuda")
    out, _ = axon.norm_rotate(q, None, pos, freqs, q_weight=w)
    tail, _ = axon.norm_rotate(q[-50:].contiguous(), None, pos[-50:].contiguous(), freqs, q_weight=w)
    d = axon.norm_rotate_backward(q, None, q, None, pos, freqs, q_weight=w)
    dt = axon.norm_rotate_backward(q[-50:], None, q[-50:], None, pos[-50:].contiguous(), freqs,
                                   q_weight=w)
    torch.cuda.synchronize()
    assert torch.equal(out[-50:], tail) and torch.equal(d.dq[-50:], dt.dq)


def test_block_of_the_three():
    """The two recurrent blocks as they are used: convolution, gated recurrence and group norm; and
    convolution, head norm with rotation and gated delta scan, on one packed buffer."""
    axon = _axon()
    lengths = [100, 0, 30, 200]
    total, E = sum(lengths) + 6, 256
    g = torch.Generator().manual_seed(0)

    def n(*s):
        return torch.randn(*s, generator=g)

    x = n(total, E).cuda()
    w, b = n(E, 4).cuda(), n(E).cuda()
    raw, in_raw, A_log = n(total, E).cuda(), n(total, E).cuda(), (n(E) - 1).cuda()
    tables = axon.sequence_tables(torch.tensor(lengths, dtype=torch.int32).cuda(), total)
    u, _ = axon.causal_conv(x, w, b, activation="silu", tables=tables)
    h, _ = axon.linear_scan(u, raw, A_log, None, in_raw, tables=tables)
    o = axon.group_norm(h, 4, centered=False)
    starts = tables.starts.long()
    pos = (torch.arange(total).cuda() - starts[torch.searchsorted(
        starts[1:], torch.arange(total).cuda(), right=True).clamp(max=3)]).int()
    freqs = (10000.0 ** (-torch.arange(32, dtype=torch.float64) / 32)).cuda()
    q, k = axon.norm_rotate(u[:, :64].unflatten(1, (1, 64)), u[:, 64:128].unflatten(1, (1, 64)), pos,
                            freqs)
    v = u[:, 128:].unflatten(1, (2, 64))
    y, _ = axon.gated_delta_scan(q, k, v, raw[:, :2].contiguous(), raw[:, 2:4].contiguous(),
                                 A_log[:2].clone(), torch.zeros(2).cuda(), tables=tables)
    torch.cuda.synchronize()
    assert not o[total - 6:].any() and not y[total - 6:].any()
    import delta_ref

    at = 0
    for j, length in enumerate(lengths):
        rows = slice(at, at + length)
        at += length
        if not length:
            continue
        uu, ub, _ = ref.conv(x[rows], w, b, torch.zeros(3, E), True)
        ref.within(u[rows], uu, ub, "u")
        # each operator against the plain form of what it was given
        r = ref.Linear(u[rows], raw[rows], in_raw[rows], torch.zeros(E), A_log, None, None, "sigmoid",
                       "sqrt")
        ref.within(h[rows], r.y, r.bound, "h")
        want = delta_ref.group_norm(h[rows], 4, None, None, None, 1e-5, False, "none", "none")
        # 64 squares: 34 u in the root's reciprocal, and products
        ref.within(o[rows], want, 40 * ref.U * want.abs(), "norm")
        for t, src in ((q, u[rows, :64]), (k, u[rows, 64:128])):
            ref.within(t[rows], *ref.norm_rotate(src.unflatten(1, (1, 64)), pos[rows], freqs, None, 1e-6,
                                                 False), "rotated")
        yy, _, big = delta_ref.delta_tokens(torch.zeros(2, 64, 64), q[rows], k[rows], v[rows],
                                            raw[rows, :2], raw[rows, 2:4], A_log[:2], torch.zeros(2))
        ref.within(y[rows], yy, delta_ref.F32 * (big + yy.abs()), "delta")
