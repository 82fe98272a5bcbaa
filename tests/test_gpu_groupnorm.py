"""The group norm against its plain 64-bit form.

Tolerance: the normalised value n has at most 3 roundings of the centred input, the sum of `width`
squares in up to 32 + log2(1024) sequential additions (their relative error, halved by the root, at
most 21 * 2^-24), and a reciprocal square root, weight, bias, SiLU and gate of at most 4 roundings
each (the hardware exponential and reciprocal): below 64 * 2^-24. Where the mean is taken off its
own error counts by the input's offset over its spread, at most 4 here: 4 * 64 * 2^-24 = 1.5e-5 of
the larger of 1 and |y|. A bf16 output adds its half step of 2^-8."""
from __future__ import annotations

import pytest

from gpu_util import say

torch = pytest.importorskip("torch")

import delta_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu
T = {"f32": torch.float32, "bf16": torch.bfloat16}
TOL = 64 * 2.0 ** -24


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


def _check(got, want, what):
    bf = got.dtype == torch.bfloat16
    got = got.double().cpu()
    assert torch.isfinite(got).all(), what
    size = want.abs().clamp(min=1.0)
    bound = 4 * TOL * size + (2.0 ** -8 * want.abs() if bf else 0.0)
    worst = float(((got - want).abs() / bound).max()) if got.numel() else 0.0
    assert worst <= 1.0, f"{what}: {worst:.2f} times the bound"


CASES = [
    # (rows, groups, width, act, centered, weight, bias, shared, activation, gate)
    (3, 1, 1, "f32", False, True, True, False, "none", "none"),
    (5, 3, 2, "bf16", True, True, True, False, "silu", "none"),
    (7, 2, 3, "f32", True, False, False, False, "none", "after"),
    (1, 5, 4, "f32", False, True, False, True, "silu", "after"),
    (9, 2, 8, "bf16", True, True, True, True, "none", "before"),
    (33, 32, 64, "bf16", False, True, False, True, "none", "after"),
    (2, 4, 100, "bf16", True, True, True, False, "silu", "before"),
    (65, 16, 128, "bf16", False, True, False, True, "none", "after"),
    (17, 8, 236, "f32", True, True, True, False, "silu", "none"),
    (4, 1, 511, "f32", True, True, True, False, "none", "none"),
    (4, 1, 513, "bf16", True, True, True, False, "none", "after"),
    (3, 2, 1024, "f32", True, True, True, False, "silu", "after"),
    (3, 1, 2048, "bf16", True, True, True, False, "none", "before"),
    (3, 1, 2052, "f32", True, True, True, False, "none", "before"),
    (2, 2, 2056, "bf16", False, True, False, False, "silu", "after"),
    (5, 1, 7680, "bf16", False, True, False, False, "none", "before"),
    (2, 1, 8191, "f32", True, True, True, False, "none", "none"),
    (2, 1, 8200, "bf16", True, True, True, False, "silu", "after"),
    (2, 2, 20001, "f32", True, True, True, True, "none", "before"),
    (0, 2, 64, "f32", True, True, True, False, "none", "none"),
]


def _inputs(rows, groups, width, act, weight, bias, shared, gate, seed=0):
    g = torch.Generator().manual_seed(seed)
    c = groups * width
    x = (torch.randn(rows, c, generator=g) * 1.5 + 0.5).to(T[act]).cuda()
    z = torch.randn(rows, c, generator=g).to(T[act]).cuda() if gate != "none" else None
    n = width if shared else c
    w = (1 + 0.2 * torch.randn(n, generator=g)).cuda() if weight else None
    b = (0.3 * torch.randn(n, generator=g)).cuda() if bias else None
    return x, w, b, z


@pytest.mark.parametrize("rows,groups,width,act,centered,weight,bias,shared,activation,gate", CASES)
def test_group_norm(rows, groups, width, act, centered, weight, bias, shared, activation, gate):
    say(f"[norm] {rows} x {groups} x {width} {act} {activation} {gate}")
    x, w, b, z = _inputs(rows, groups, width, act, weight, bias, shared, gate, seed=width)
    y = _axon().group_norm(x, groups, w, b, z, eps=1e-5, centered=centered, activation=activation,
                           gate=gate)
    torch.cuda.synchronize()
    assert y.shape == x.shape and y.dtype == x.dtype
    _check(y, ref.group_norm(x, groups, w, b, z, 1e-5, centered, activation, gate), "y")


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("offset,width", [(0, 128), (8, 128), (3, 128), (1, 50), (5, 20000)])
def test_parts_of_a_projection_and_in_place(act, offset, width):
    """x and z inside wider rows, at aligned and odd offsets; then in place."""
    say(f"[norm] part at {offset}, width {width}, {act}")
    x, w, b, z = _inputs(6, 2, width, act, True, True, False, "after", seed=3)
    wide = torch.randn(2, 3, 4 * width + 2 * offset + 8).to(T[act]).cuda()
    xs = wide[..., offset:offset + 2 * width]
    zs = wide[..., 2 * width + offset:4 * width + offset]
    xs.copy_(x.view(2, 3, -1))
    zs.copy_(z.view(2, 3, -1))
    want = ref.group_norm(x, 2, w, b, z, 1e-5, True, "silu", "after")
    y = _axon().group_norm(xs, 2, w, b, zs, activation="silu")
    _check(y.view(6, -1), want, "part")
    out = _axon().group_norm(x, 2, w, b, z, activation="silu", y=x)
    assert out is x
    _check(x, want, "in place")


def test_equal_values_and_not_finite():
    x = torch.full((3, 256), 2.5).cuda()
    y = _axon().group_norm(x, 2, bias=torch.full((256,), 0.25).cuda())
    assert bool((y == 0.25).all())
    x[1, 7] = float("nan")
    x[2, 200] = float("inf")
    y = _axon().group_norm(x, 2)
    torch.cuda.synchronize()
    assert bool((y[0] == 0).all()) and bool(y[1, :128].isnan().all()) and bool((y[1, 128:] == 0).all())
    assert bool((y[2, :128] == 0).all()) and bool(y[2, 128:].isnan().all())


def test_captured():
    x, w, b, z = _inputs(8, 4, 96, "bf16", True, True, False, "after", seed=5)
    y = torch.zeros_like(x)
    _axon().group_norm(x, 4, w, b, z, y=y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _axon().group_norm(x, 4, w, b, z, y=y)
    for _ in range(3):
        x.copy_(torch.randn(8, 384))
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, _axon().group_norm(x, 4, w, b, z))


def test_refused():
    axon = _axon()
    x, w, b, z = _inputs(4, 2, 64, "f32", True, True, False, "after")
    for args, kw in (((x, 3), {}), ((x, 0), {}), ((x.half(), 2), {}), ((x.cpu(), 2), {}),
                     ((x, 2, w.double()), {}), ((x, 2, w[:100]), {}), ((x, 2, w, b[:64]), {}),
                     ((x, 2, w, b, z[:3]), {}), ((x, 2, w, b, z.bfloat16()), {}),
                     ((x.t(), 2), {}), ((x[:1].expand(4, 128), 2), {}),
                     ((x, 2), dict(gate="after")), ((x, 2, w, b, z), dict(gate="none")),
                     ((x, 2, w, b, z), dict(gate="other")), ((x, 2), dict(activation="relu")),
                     ((x, 2), dict(eps=-1.0)), ((x, 2), dict(eps=float("nan"))),
                     ((x, 2, w, b, z), dict(y=z)), ((x, 2), dict(y=x[:2]))):
        with pytest.raises((TypeError, ValueError, axon.AxonError)):
            axon.group_norm(*args, **kw)
    with pytest.raises(axon.AxonError):  # y over part of x
        flat = torch.zeros(5 * 128).cuda()
        axon.group_norm(flat[:512].view(4, 128), 2, y=flat[128:].view(4, 128))
    torch.cuda.synchronize()
