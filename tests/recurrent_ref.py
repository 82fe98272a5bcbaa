"""Plain 64-bit forms of the gated linear recurrence, the causal convolution and the head norm with
rotation on the CPU, for the GPU tests, each with a bound of what fp32 arithmetic may be off by.

With u = 2^-24 (half a step of fp32). A sigmoid or softplus of v is computed from a rounded sum and an
exponential of a rounded exponent: off by (4 |v| + 8) u, relative, where the framework's softplus adds
1e-6 < 17 u. log a = -exp(A_log) dt adds 4 u, and the sum of 64 of them that carries a state over a
block 64 roundings in the worst case: EL = (4 |v| + 96) u. An input b = m u(x) is off by EB = EL +
(4 |v_in| + 32) u. The recurrence then is off by at most

  N_t = a (N_{t-1} + EL |L| M_{t-1})     exponents, with M_t = a M_{t-1} + |b_t|
  E_t = a E_{t-1} + EB |b_t|             inputs
  R_t = a R_{t-1} + 6 u M_t              roundings of a, of two sums a token and of carried states

and likewise the gradient that runs backwards. What is formed from both takes the bounds of its factors
(first order) and 32 u + 4 EL (1 + |L|) of its size for its own products. Sums over tokens take the sum
of their terms' bounds and 64 u of their terms' sizes. The exponential's results below 2^-126, the least
normal fp32, are zeros: a is off by 2^-126 at most beside all that, which large factors (a state of
1e6, a gradient of 1e3, |L| of 100) bring up to 1e-27. Likewise dt, so that |L| is off by up to rate
2^-126 and m = sqrt(1 - a^2) = sqrt(2 |L|) by sqrt(2 rate 2^-126), about 1e-19; and the input's gate,
so that u is off by |x| 2^-126 (where the least reciprocal of a number below 2^126 stands for zero, by
1.001 times that: TINY). A bf16 result adds half a step, 2^-8 of its
size.
"""
from __future__ import annotations

import torch

U = 2.0 ** -24
TINY = 1.001 * 2.0 ** -126
BF16_HALF = 2.0 ** -8


def d(t):
    return None if t is None else t.detach().double().cpu()


def within(got, want, bound, what):
    """|got - want| <= bound, and half a step more for bf16."""
    bf = got.dtype == torch.bfloat16
    got = d(got)
    assert got.shape == want.shape, f"{what}: shape {tuple(got.shape)}, expected {tuple(want.shape)}"
    assert torch.isfinite(got).all(), f"{what}: not finite"
    bound = bound + 1e-37
    if bf:
        bound = bound + BF16_HALF * (want.abs() + bound)
    off = (got - want).abs()
    assert bool((off <= bound).all()), (
        f"{what}: {float((off / bound).max()):.2f} times the bound, largest error {float(off.max()):.3e}")


class Linear:
    """One sequence: x, raw, in_raw (L, E; in_raw may be None), s0 (E)."""

    def __init__(self, x, raw, in_raw, s0, A_log, dt_bias, in_bias, gate, input_scale):
        x, raw, in_raw, s0, A_log, dt_bias, in_bias = map(
            d, (x, raw, in_raw, s0, A_log, dt_bias, in_bias))
        v = raw if dt_bias is None else raw + dt_bias
        e = torch.exp(-v.abs())
        on = torch.where(v < 0, e / (1 + e), 1 / (1 + e))
        off = torch.where(v < 0, 1 / (1 + e), e / (1 + e))
        if gate == "sigmoid":
            dt, self.slope = on, off
        else:
            dt = torch.log1p(e) + v.clamp(min=0)
            self.slope = torch.where(v < -30, torch.ones_like(v), on / dt)
        self.L = L = -torch.exp(A_log) * dt
        self.a = torch.exp(L)
        self.scale = input_scale
        self.m = {"none": torch.ones_like(L), "complement": -torch.expm1(L),
                  "sqrt": torch.sqrt(-torch.expm1(2 * L))}[input_scale]
        rate = torch.exp(A_log)
        self.moff = (2 * rate * TINY).sqrt() if input_scale == "sqrt" else rate * TINY
        self.x, self.i = x, None
        vi = torch.zeros_like(x)
        if in_raw is not None:
            vi = in_raw if in_bias is None else in_raw + in_bias
            self.i = torch.sigmoid(vi)
            self.ioff = torch.sigmoid(-vi)
        self.u = x if self.i is None else x * self.i
        self.EL = (4 * v.abs() + 96) * U
        self.EB = self.EL + (4 * vi.abs() + 32) * U
        b = self.m * self.u
        self.uoff = TINY * x.abs() if self.i is not None else torch.zeros_like(x)
        n = x.shape[0]
        h, M = s0.clone(), s0.abs()
        N, E, R = torch.zeros_like(h), torch.zeros_like(h), torch.zeros_like(h)
        self.y, self.before = torch.zeros_like(x), torch.zeros_like(x)
        self.bound, self.size = torch.zeros_like(x), torch.zeros_like(x)
        self.before_bound = torch.zeros_like(x)
        for t in range(n):
            a = self.a[t]
            self.before[t], self.size[t], self.before_bound[t] = h, M, N + E + R
            N = a * (N + self.EL[t] * L[t].abs() * M) + TINY * M
            E = a * E + self.EB[t] * b[t].abs() + self.moff * self.u[t].abs() + self.uoff[t]
            h = a * h + b[t]
            M = a * M + b[t].abs()
            R = a * R + 6 * U * M
            self.y[t], self.bound[t] = h, N + E + R
        self.state, self.state_bound = h, N + E + R

    def backward(self, dy, dstate):
        """{name: (gradient, bound)}; sums over the tokens of this sequence."""
        dy, k = d(dy), d(dstate).clone()
        a, L, absL = self.a, self.L, self.L.abs()
        g, gb, Mg = torch.zeros_like(dy), torch.zeros_like(dy), torch.zeros_like(dy)
        M = k.abs()
        N, R = torch.zeros_like(k), torch.zeros_like(k)
        for t in range(dy.shape[0] - 1, -1, -1):
            g[t] = dy[t] + k
            size = dy[t].abs() + M
            Mg[t], gb[t] = size, N + R + 2 * U * size
            k = a[t] * g[t]
            N = a[t] * (N + self.EL[t] * absL[t] * size) + TINY * size
            M = a[t] * size
            R = a[t] * R + 6 * U * size * a[t]
        aL = torch.where(a == 0, torch.zeros_like(a), a * L)
        if self.scale == "sqrt":
            second = torch.where(self.m == 0, torch.zeros_like(a), -a * aL / self.m)
        elif self.scale == "complement":
            second = -aL
        else:
            second = torch.zeros_like(a)
        G = g * (aL * self.before + second * self.u)
        own = 4 * self.EL * (1 + absL) + 32 * U
        Gb = aL.abs() * (gb * self.size + Mg * self.before_bound) + second.abs() * self.u.abs() * gb
        Gb = Gb + (aL.abs() * self.size + second.abs() * self.u.abs()) * Mg * (own + self.EB)
        Gb = Gb + 2 * TINY * absL * Mg * (self.size + self.u.abs())
        Gb = Gb + Mg * (self.moff * self.u.abs() + self.moff ** 2 * self.size)
        Gb = Gb + Mg * second.abs() * self.uoff
        draw, drawb = G * self.slope, Gb * self.slope + G.abs() * self.slope * own
        du = g * self.m
        dub = gb * self.m + Mg * (self.m * self.EB + self.moff)
        out = {"ddt_raw": (draw, drawb)}
        if self.i is None:
            out["dx"] = (du, dub)
        else:
            out["dx"] = (du * self.i, dub * self.i + (du * self.i).abs() * self.EB + Mg * self.m * TINY)
            di = du * self.x * self.i * self.ioff
            dib = (dub * self.x * self.i * self.ioff).abs() + di.abs() * 2 * self.EB + Mg * self.m * self.uoff
            out["din_raw"] = (di, dib)
            out["din_bias"] = (di.sum(0), dib.sum(0) + 64 * U * di.abs().sum(0))
        out["dA_log"] = (G.sum(0), Gb.sum(0) + 64 * U * G.abs().sum(0))
        out["ddt_bias"] = (draw.sum(0), drawb.sum(0) + 64 * U * draw.abs().sum(0))
        out["dstate_in"] = (k, N + R)
        return out


def conv(x, w, b, cache, silu):
    """One sequence: x (L, E), cache (3, E). Returns y, its bound, the final cache."""
    x, w, b, cache = map(d, (x, w, b, cache))
    full = torch.cat([cache, x])
    n = x.shape[0]
    p = torch.zeros_like(x) if b is None else b.expand_as(x).clone()
    size = p.abs()
    for k in range(4):
        p = p + full[k:k + n] * w[:, k]
        size = size + (full[k:k + n] * w[:, k]).abs()
    # five roundings at most of partial sums, 2^-24 each
    off = 5 * U * size
    if silu:
        # |SiLU'| <= 1.1; the sigmoid's own error (4 |p| + 8) u of the result, and a product
        y = p * torch.sigmoid(p)
        off = 1.1 * off + (4 * p.abs() + 12) * U * y.abs()
    else:
        y = p
    return y, off, full[n:]


def conv_backward(dy, x, w, b, cache, dcache, silu):
    """{name: (gradient, bound)} of one sequence."""
    dy, x, w, b, cache, dcache = map(d, (dy, x, w, b, cache, dcache))
    full = torch.cat([cache, x])
    n = x.shape[0]
    p = torch.zeros_like(x) if b is None else b.expand_as(x).clone()
    size = p.abs()
    for k in range(4):
        p = p + full[k:k + n] * w[:, k]
        size = size + (full[k:k + n] * w[:, k]).abs()
    s, sb = dy, torch.zeros_like(dy)
    if silu:
        q = torch.sigmoid(p)
        s = dy * q * (1 + p * (1 - q))
        # |SiLU''| <= 1/2; q and 1 - q are off by (4 |p| + 8) u, the sum of 1 and p (1 - q) may cancel
        sb = dy.abs() * (0.5 * 5 * U * size + q * (1 + (p * (1 - q)).abs()) * (8 * p.abs() + 24) * U)
    dfull, db_ = torch.zeros_like(full), torch.zeros_like(full)
    dw, dwb = torch.zeros_like(w), torch.zeros_like(w)
    for k in range(4):
        dfull[k:k + n] += s * w[:, k]
        db_[k:k + n] += (sb + 5 * U * s.abs()) * w[:, k].abs()
        dw[:, k] = (s * full[k:k + n]).sum(0)
        dwb[:, k] = ((sb + 66 * U * s.abs()) * full[k:k + n].abs()).sum(0)
    dfull[n:] += dcache
    db_[n:] += 2 * U * dcache.abs()
    return {"dx": (dfull[3:], db_[3:]), "dcache_in": (dfull[:3], db_[:3]), "dconv_w": (dw, dwb),
            "dconv_b": (s.sum(0), (sb + 66 * U * s.abs()).sum(0))}


def angles(positions, freqs):
    return d(positions)[..., None] * d(freqs)


def turn(z, angle, interleaved):
    """z (rows, heads, D) with its first channels turned by angle (rows, R / 2)."""
    r = 2 * angle.shape[-1]
    c, s = angle.cos()[:, None], angle.sin()[:, None]
    z = z.clone()
    first = slice(0, r, 2) if interleaved else slice(0, r // 2)
    second = slice(1, r, 2) if interleaved else slice(r // 2, r)
    a, b = z[..., first].clone(), z[..., second].clone()
    z[..., first], z[..., second] = a * c - b * s, b * c + a * s
    return z


def pair_size(z, r, interleaved):
    """For every channel what the turned pair holds at most: |a| + |b|."""
    z = z.abs().clone()
    first = slice(0, r, 2) if interleaved else slice(0, r // 2)
    second = slice(1, r, 2) if interleaved else slice(r // 2, r)
    both = z[..., first] + z[..., second]
    z[..., first] = z[..., second] = both
    return z


def norm_rotate(x, positions, freqs, w, eps, interleaved):
    """x (rows, heads, D). The sum of D squares is off by (D + 2) u at most, its root's reciprocal by half
    of that and 4 u, products by 3 u; cosine and sine by 4 u and the reduced angle (a fraction of a
    turn in fp32, 2^-25 turns) by 2 pi 2^-25 < 4 u: 16 u + (D / 2) u of |a| + |b|."""
    x, w = d(x), d(w)
    z = x / (x.square().mean(-1, keepdim=True) + eps).sqrt()
    if w is not None:
        z = z * w
    angle = angles(positions, freqs)
    y = turn(z, angle, interleaved)
    return y, (20 + x.shape[-1] / 2) * U * pair_size(z, 2 * angle.shape[-1], interleaved)


def norm_rotate_backward(dout, x, positions, freqs, w, eps, interleaved):
    dout, x, w = d(dout), d(x), d(w)
    D = x.shape[-1]
    r = 1 / (x.square().mean(-1, keepdim=True) + eps).sqrt()
    n = x * r
    angle = angles(positions, freqs)
    back = turn(dout, -angle, interleaved)
    R = 2 * angle.shape[-1]
    backb = 14 * U * pair_size(dout, R, interleaved)
    dw = (back * n).sum((0, 1))
    # fp32 over 32 rows' heads in a lane and 64 lanes, then 64 bits
    count = min(32, x.shape[0]) * x.shape[1] + 64
    dwb = ((backb + (D / 2 + 8 + count) * U * back.abs()) * n.abs()).sum((0, 1))
    dn, dnb = back, backb
    if w is not None:
        dn, dnb = back * w, (backb + 2 * U * back.abs()) * w.abs()
    mean = (dn * n).mean(-1, keepdim=True)
    meanb = ((dnb + (D + D / 2 + 12) * U * dn.abs()) * n.abs()).mean(-1, keepdim=True)
    dx = r * (dn - n * mean)
    dxb = r * (dnb + n.abs() * meanb + (D / 2 + 12) * U * (dn.abs() + (n * mean).abs()))
    return dx, dxb, dw, dwb
