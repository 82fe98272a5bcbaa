"""Outputs of 64 MiB and more, which are stored past the caches: in both types, with everything that a call can
write, against the 64-bit forms in some channels over all rows; and the long sequence of a buffer of more than 2^32
bytes against the same channels by themselves."""
from __future__ import annotations

import pytest

from gpu_util import say

torch = pytest.importorskip("torch")

import recurrent_ref as ref  # noqa: E402
import test_gpu_conv as conv  # noqa: E402
import test_gpu_linear as linear  # noqa: E402
import test_gpu_rotate as rotate  # noqa: E402
from test_gpu_linear import T, _axon, _gpu  # noqa: E402,F401

pytestmark = pytest.mark.gpu
LARGE = 64 << 20


def size(t):
    return t.numel() * t.element_size()


@pytest.mark.parametrize("act,E", [("f32", 8000), ("f32", 8001), ("bf16", 16000)])
@pytest.mark.parametrize("gate,scale", [("sigmoid", "sqrt"), ("softplus", "complement")])
def test_linear(gate, scale, act, E):
    say(f"[large] linear {E} {act} {gate} {scale}")
    axon = _axon()
    B, L = 2, 1050
    z = linear.make((B, L), E, act, seed=1)
    s0, ds, dy = linear.states(B, E, 1), linear.states(B, E, 2), linear.grad((B, L), E, act)
    points = axon.linear_checkpoints(z["x"])
    y, s1 = axon.linear_scan(**z, gate=gate, input_scale=scale, state_in=s0, checkpoints=points)
    g = axon.linear_scan_backward(dy, **z, gate=gate, input_scale=scale, checkpoints=points, dstate_out=ds)
    torch.cuda.synchronize()
    assert size(y) >= LARGE
    some = torch.tensor([0, 1, 63, 64, 4567, E - 65, E - 1], device="cuda")
    part = {k: v.index_select(-1, some) for k, v in z.items()}
    grads = axon.LinearScanGrads(*[t.index_select(-1, some) for t in g])
    linear.compare(part, list(range(B)), s0[:, some], ds[:, some], dy[..., some], y[..., some], s1[:, some], grads,
                   gate, scale)


@pytest.mark.parametrize("act,E", [("f32", 8000), ("bf16", 8000)])
@pytest.mark.parametrize("activation", ["none", "silu"])
def test_conv(activation, act, E):
    """Rows enough that a lane takes four channels, the form that stores past the caches."""
    say(f"[large] convolution {E} {act} {activation}")
    axon = _axon()
    B, L = 4, 1100
    z, dy = conv.make((B, L), E, act, seed=1), conv.grad((B, L), E, act)
    c0, dc = conv.caches(B, E), conv.caches(B, E, 1)
    y, c1 = axon.causal_conv(**z, activation=activation, cache_in=c0)
    g = axon.causal_conv_backward(dy, **z, activation=activation, cache_in=c0, dcache_out=dc)
    torch.cuda.synchronize()
    assert size(y) >= LARGE
    some = torch.tensor([0, 1, 2, 3, 255, 256, 4567, E - 1], device="cuda")
    part = dict(x=z["x"][..., some], conv_w=z["conv_w"][some], conv_b=z["conv_b"][some])
    grads = axon.CausalConvGrads(g.dx[..., some], g.dconv_w[some], g.dconv_b[some], g.dcache_in[..., some])
    conv.compare(part, list(range(B)), c0[..., some], dc[..., some], dy[..., some], y[..., some], c1[..., some],
                 grads, activation)


ROTATE = [
    # (rows, hq, hk, D, R, act, interleaved): several rows a wave, one row a wave
    (180_000, 2, 1, 32, 32, "f32", True), (180_000, 2, 1, 32, 16, "f32", False),
    (3400, 32, 8, 128, 128, "f32", False), (3400, 32, 8, 128, 64, "f32", True),
    (360_000, 2, 1, 32, 32, "bf16", True), (360_000, 2, 1, 32, 32, "bf16", False),
    (6800, 32, 8, 128, 128, "bf16", True),
]


@pytest.mark.parametrize("rows,hq,hk,D,R,act,inter", ROTATE)
def test_rotate(rows, hq, hk, D, R, act, inter):
    say(f"[large] rotate {rows} x {hq}+{hk} x {D}/{R} {act} interleaved={inter}")
    axon = _axon()
    z, kw = rotate.make(rows, hq, hk, D, R, act, seed=rows)
    g = torch.Generator(device="cuda").manual_seed(1)
    d = [torch.empty(rows, h, D, device="cuda").normal_(generator=g).to(T[act]) for h in (hq, hk)]
    out = axon.norm_rotate(**z, **kw, interleaved=inter)
    grads = axon.norm_rotate_backward(*d, **z, **kw, interleaved=inter)
    torch.cuda.synchronize()
    assert size(out[0]) + size(out[1]) >= LARGE
    some = torch.arange(0, rows, max(1, rows // 3000), device="cuda")  # rows of every kind of place
    some = torch.cat([some, torch.arange(rows - 5, rows, device="cuda")])
    part = dict(q=z["q"][some], k=z["k"][some], positions=z["positions"][some], freqs=z["freqs"])
    for j, name in enumerate("qk"):
        args = (part["positions"], z["freqs"], kw[f"{name}_weight"], 1e-6, inter)
        ref.within(out[j][some], *ref.norm_rotate(part[name], *args), name)
        dx, dxb, _, _ = ref.norm_rotate_backward(d[j][some], part[name], *args)
        ref.within(grads[j][some], dx, dxb, f"d{name}")
    # the weights' gradients take all rows: those of k, which has fewer heads
    args = (z["positions"], z["freqs"], kw["k_weight"], 1e-6, inter)
    ref.within(grads[3], *ref.norm_rotate_backward(d[1], z["k"], *args)[2:], "dk_weight")


def test_the_long_sequence_of_a_buffer_beyond_32_bits():
    """Its last channels, by the wide call and by themselves: rounding of the carries apart, the same."""
    axon = _axon()
    E, total, long = 16384, 131072 + 900, 131000
    g = torch.Generator(device="cuda").manual_seed(0)
    z = linear.make((1,), E, "bf16", seed=1)
    for k in ("x", "dt_raw", "in_raw"):
        z[k] = torch.empty(total, E, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    lengths = torch.tensor([72, long, 895], dtype=torch.int32).cuda()
    tables = axon.sequence_tables(lengths, total)
    p = axon.linear_checkpoints(z["x"], tables=tables)
    y, s = axon.linear_scan(**z, tables=tables, checkpoints=p)
    d = axon.linear_scan_backward(z["x"], **z, tables=tables, checkpoints=p)
    rows, cols = slice(72, 72 + long), slice(E - 64, E)
    alone = {k: v[None, rows, cols].contiguous() if v.dim() == 2 else v[cols].contiguous() for k, v in z.items()}
    pa = axon.linear_checkpoints(alone["x"])
    ya, sa = axon.linear_scan(**alone, checkpoints=pa)
    da = axon.linear_scan_backward(alone["x"], **alone, checkpoints=pa)
    torch.cuda.synchronize()
    for got, want, what in ((y, ya, "y"), (d.dx, da.dx, "dx"), (d.ddt_raw, da.ddt_raw, "ddt_raw"),
                            (d.din_raw, da.din_raw, "din_raw")):
        assert torch.allclose(got[rows, cols].float(), want[0].float(), rtol=2 ** -7, atol=1e-3), what
    assert torch.allclose(s[1, cols], sa[0], rtol=1e-4, atol=1e-5)
    assert torch.allclose(d.dstate_in[1, cols], da.dstate_in[0], rtol=1e-4, atol=1e-5)
    del y, d, alone, ya, da
    x = z["x"]
    w, b = torch.randn(E, 4, device="cuda", generator=g), torch.randn(E, device="cuda", generator=g)
    y, c = axon.causal_conv(x, w, b, tables=tables, activation="silu")
    d = axon.causal_conv_backward(x, x, w, b, tables=tables, activation="silu")
    xa, wa, ba = x[None, rows, cols].contiguous(), w[cols].contiguous(), b[cols].contiguous()
    ya, ca = axon.causal_conv(xa, wa, ba, activation="silu")
    da = axon.causal_conv_backward(xa, xa, wa, ba, activation="silu")
    torch.cuda.synchronize()
    assert torch.equal(y[rows, cols], ya[0]) and torch.equal(c[1, :, cols], ca[0])
    assert torch.equal(d.dx[rows, cols], da.dx[0])
