"""Plain 64-bit forms of the gated delta rule, of the tables of packed sequences and of the group
norm, token by token on the CPU, for the GPU tests.

Tolerances. A state, and an output before its rounding, is a sum of at most K + 64 fp32 products
(K <= 128 state entries, 64 writes of a chunk) of terms whose sizes the unit-length keys bound by
the size of the largest state row norm R; every product and sum rounds by at most 2^-24 relative.
Linear growth over those K + 64 < 200 roundings, twice (the writes D enter the states and the
outputs), gives 2 * 200 * 2^-24 R = 2.4e-5 R. The decays add 64 rounded exponents of size at most
e^-1 |g| e^g <= 2^-24 * 24 R, which is below a tenth of that. Later chunks forget no slower than
they add, so the bound is taken once more for what enters them: F32 = 5e-5 of (R + |ref|). A bf16
output adds its half step, 2^-8 of |ref|.
"""
from __future__ import annotations

import torch

F32 = 5e-5
BF16_HALF = 2.0 ** -8


def delta_tokens(S, q, k, v, dt_raw, beta_raw, A_log, dt_bias, *, dt_min=1e-4, dt_max=100.0,
                 scale=None, eps=1e-6):
    """The recurrence over the tokens of one sequence, in 64 bits: S (Hv, V, K), q, k (L, Hk, K),
    v (L, Hv, V). Returns (y (L, Hv, V), S after the last token, the largest row norm of S)."""
    q, k, v, dt_raw, beta_raw, A_log, dt_bias, S = (
        t.detach().double().cpu() for t in (q, k, v, dt_raw, beta_raw, A_log, dt_bias, S))
    ratio = v.shape[1] // q.shape[1]
    scale = q.shape[-1] ** -0.5 if scale is None else scale
    x = dt_raw + dt_bias
    dt = (x.clamp(min=0) + torch.log1p(torch.exp(-x.abs()))).clamp(dt_min, dt_max)
    a = torch.exp(-torch.exp(A_log) * dt)
    beta = torch.sigmoid(beta_raw)
    q = (q / (q.square().sum(-1, keepdim=True) + eps).sqrt()).repeat_interleave(ratio, 1)
    k = (k / (k.square().sum(-1, keepdim=True) + eps).sqrt()).repeat_interleave(ratio, 1)
    S = S.clone()
    big = float(S.norm(dim=-1).max())
    y = torch.zeros_like(v)
    for t in range(v.shape[0]):
        S = a[t][:, None, None] * S
        d = beta[t][:, None] * (v[t] - (S @ k[t][..., None])[..., 0])
        S = S + d[..., None] * k[t][:, None, :]
        y[t] = scale * (S @ q[t][..., None])[..., 0]
        big = max(big, float(S.norm(dim=-1).max()))
    return y, S, big


def tables(lengths, total, block):
    """(starts, block_starts, block_seq, block_first) as lists."""
    starts, blocks, seq, first = [0], [0], [], []
    for n, length in enumerate(lengths):
        end = min(total, starts[-1] + max(0, length))
        for at in range(starts[-1], end, block):
            seq.append(n)
            first.append(at)
        starts.append(end)
        blocks.append(len(seq))
    rows = total // block + len(lengths)
    pad = [-1] * (rows - len(seq))
    return starts, blocks, seq + pad, first + pad


def group_norm(x, groups, weight, bias, z, eps, centered, activation, gate):
    x = x.detach().double().cpu()
    s = None
    if z is not None:
        z = z.detach().double().cpu()
        s = z / (1 + torch.exp(-z))
    u = x * s if gate == "before" else x
    u = u.reshape(*x.shape[:-1], groups, x.shape[-1] // groups)
    if centered:
        u = u - u.mean(-1, keepdim=True)
    n = u / (u.square().mean(-1, keepdim=True) + eps).sqrt()
    if weight is not None:
        n = n * weight.detach().double().cpu().reshape(-1, u.shape[-1])
    if bias is not None:
        n = n + bias.detach().double().cpu().reshape(-1, u.shape[-1])
    if activation == "silu":
        n = n / (1 + torch.exp(-n))
    n = n.reshape(x.shape)
    return n * s if gate == "after" else n
