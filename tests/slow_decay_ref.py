"""States under decays so slow that the rounding of a counts: s0 exp(sum log a) in 64 bits, and what fp32
states that are handed on by h + expm1(log a) h may be off by.

With u = 2^-24 and no inputs (x = 0) such a hand-over rounds twice: the product, which is about |log a|
of the state, and the sum: u (1 + |log a|) of it. log a is a sum of up to 192 rounded terms and expm1's series
adds to their error: 100 u of |log a| at most on the way of 16 tokens, 250 u on that of 192. For 1e-6 a token
that is 0.05 u (192 tokens: |log a| 2e-4) and in all 1.06 u of |s0| a hand-over. The plain fp32 a instead is off by up to u / 2, by the same
in every token, and each product rounds the state once more."""
from __future__ import annotations

import numpy as np
import torch

U = 2.0 ** -24
HAND_OVER = 1.06 * U


def rates(E, lo=1e-7, hi=1e-6, seed=0):
    """A_log (E,) float32 for log a = -exp(A_log) / 2 between -hi and -lo (the gate's raw value is 0), and that
    log a of the float32 A_log in 64 bits."""
    g = torch.Generator().manual_seed(seed)
    target = torch.exp(np.log(lo) + (np.log(hi) - np.log(lo)) * torch.rand(E, generator=g, dtype=torch.float64))
    A_log = torch.log(2 * target).float()
    return A_log, -0.5 * torch.exp(A_log.double())


def hand_overs(tokens, wave, tile):
    """One a wave of a sequence's tokens; of more than a tile two more (the tile's front and the wave's)."""
    return -(-tokens // wave) + (2 if tokens > tile else 0)


def handed_on(s0, log_a, tokens, wave=16):
    """s0 (E,) after `tokens` by hand-overs of `wave` tokens, in float32."""
    h = s0.numpy().astype(np.float32)
    L = log_a.numpy()
    for first in range(0, tokens, wave):
        c = np.expm1(L * min(wave, tokens - first)).astype(np.float32)
        h = (c * h).astype(np.float32) + h
    return torch.from_numpy(h)


def multiplied(s0, log_a, tokens):
    """s0 (E,) after `tokens` products with the float32 a."""
    h = s0.numpy().astype(np.float32)
    a = np.exp(log_a.numpy()).astype(np.float32)
    for _ in range(tokens):
        h = (a * h).astype(np.float32)
    return torch.from_numpy(h)
