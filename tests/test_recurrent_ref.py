"""The plain gradients that the GPU tests compare with, against central differences in 64 bits."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

import recurrent_ref as ref  # noqa: E402

STEP = 1e-5
# Central differences: h^2 / 6 of the third derivative (a few hundred at most here) and 2^-52 / h of the
# loss (about 10): 2e-8 + 2e-10, against gradients of about one.
TOL = 1e-6


def differences(loss, t):
    out = torch.zeros_like(t)
    flat, o = t.view(-1), out.view(-1)
    for j in range(flat.numel()):
        keep = float(flat[j])
        flat[j] = keep + STEP
        hi = loss()
        flat[j] = keep - STEP
        lo = loss()
        flat[j] = keep
        o[j] = (hi - lo) / (2 * STEP)
    return out


def near(got, want, what):
    assert torch.allclose(got, want, rtol=TOL, atol=TOL), f"{what}: {float((got - want).abs().max())}"


@pytest.mark.parametrize("gate", ["sigmoid", "softplus"])
@pytest.mark.parametrize("scale", ["sqrt", "complement", "none"])
@pytest.mark.parametrize("gated", [True, False])
def test_linear(gate, scale, gated):
    g = torch.Generator().manual_seed(1)
    L, E = 6, 3

    def n(*s):
        return torch.randn(*s, generator=g, dtype=torch.float64)

    z = dict(x=n(L, E), raw=n(L, E), in_raw=n(L, E) if gated else None, s0=n(E), A_log=n(E) - 1,
             dt_bias=n(E), in_bias=n(E) if gated else None)
    dy, ds = n(L, E), n(E)

    def loss():
        r = ref.Linear(*z.values(), gate, scale)
        return float((r.y * dy).sum() + (r.state * ds).sum())

    got = ref.Linear(*z.values(), gate, scale).backward(dy, ds)
    names = dict(x="dx", raw="ddt_raw", in_raw="din_raw", s0="dstate_in", A_log="dA_log",
                 dt_bias="ddt_bias", in_bias="din_bias")
    for k, name in names.items():
        if z[k] is not None:
            near(got[name][0], differences(loss, z[k]), name)


@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("L", [1, 2, 3, 7])
def test_conv(silu, L):
    g = torch.Generator().manual_seed(2)

    def n(*s):
        return torch.randn(*s, generator=g, dtype=torch.float64)

    z = dict(x=n(L, 3), w=n(3, 4), b=n(3), cache=n(3, 3))
    dy, dc = n(L, 3), n(3, 3)

    def loss():
        y, _, cache = ref.conv(*z.values(), silu)
        return float((y * dy).sum() + (cache * dc).sum())

    got = ref.conv_backward(dy, *z.values(), dc, silu)
    for k, name in dict(x="dx", w="dconv_w", b="dconv_b", cache="dcache_in").items():
        near(got[name][0], differences(loss, z[k]), name)


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("rotary", [2, 6, 8])
def test_norm_rotate(rotary, interleaved):
    g = torch.Generator().manual_seed(3)

    def n(*s):
        return torch.randn(*s, generator=g, dtype=torch.float64)

    x, w, dy = n(3, 2, 8), n(8), n(3, 2, 8)
    pos = torch.tensor([0, 5, 1000], dtype=torch.int32)
    freqs = 10.0 ** -torch.arange(rotary // 2, dtype=torch.float64)

    def loss():
        return float((ref.norm_rotate(x, pos, freqs, w, 1e-3, interleaved)[0] * dy).sum())

    dx, _, dw, _ = ref.norm_rotate_backward(dy, x, pos, freqs, w, 1e-3, interleaved)
    near(dx, differences(loss, x), "dx")
    near(dw, differences(loss, w), "dw")
