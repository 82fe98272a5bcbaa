"""Cases of the gated delta rule, of the tables of packed sequences and of the group norm.

``listed()`` names the cases, ``draw(rng)`` gives more of the same ranges, ``prepare`` makes what a
program has in hand before the call, ``run`` makes one pass: with ``own`` the package's entry
points, without it the same mathematics in elementary torch operations. ``exact`` is the
definition in 64 bits, token by token.
"""
from __future__ import annotations

import math

import torch

own = False

CHUNK = 64
EPS_QK = 1e-6


def listed():
    return [
        # A scheduler's step with a handful of new requests: latency only.
        dict(name="tables_few", op="tables", sequences=7, longest=300, block=64, spare=40),
        # A whole batch re-planned: thousands of requests, two million tokens.
        dict(name="tables_many", op="tables", sequences=4096, longest=1000, block=64, spare=1000),
        # One user decoding alone with a small fp32 layer.
        dict(name="step_one_f32", op="step", rows=1, slots=1, hk=4, hv=4, k=64, v=64, dtype="f32"),
        # An ordinary decode batch in a pool of states, padded to a captured size (some rows idle).
        dict(name="step_64", op="step", rows=64, slots=96, hk=16, hv=32, k=128, v=128,
             dtype="bf16"),
        # The largest decode batch: a gibibyte of states.
        dict(name="step_512", op="step", rows=512, slots=512, hk=16, hv=32, k=128, v=128,
             dtype="bf16"),
        # A short prompt: two chunks and a bit, latency.
        dict(name="scan_prompt", op="scan", sequences=1, tokens=150, hk=16, hv=32, k=128, v=128,
             dtype="bf16", packed=False, carried=False),
        # fp32 layer, a small uniform batch that continues from states.
        dict(name="scan_f32", op="scan", sequences=2, tokens=2048, hk=8, hv=16, k=128, v=128,
             dtype="f32", packed=False, carried=True),
        # One long document: few rows, a long axis.
        dict(name="scan_long", op="scan", sequences=1, tokens=16384, hk=16, hv=32, k=128, v=128,
             dtype="bf16", packed=False, carried=False),
        # A prefill batch of requests of unequal length, some continuing, packed in one buffer.
        dict(name="scan_packed", op="scan", sequences=24, tokens=32768, hk=16, hv=32, k=128,
             v=128, dtype="bf16", packed=True, carried=True),
        # The norm of one decode batch's heads, gated after (weights shared by the heads).
        dict(name="norm_decode", op="norm", rows=64, groups=32, width=128, dtype="bf16",
             centered=False, bias=False, shared=True, activation="none", gate="after"),
        # fp32, group width that is no power of two, centred with a bias and SiLU.
        dict(name="norm_f32", op="norm", rows=5001, groups=8, width=236, dtype="f32",
             centered=True, bias=True, shared=False, activation="silu", gate="none"),
        # Prefill activations, one wide group gated before.
        dict(name="norm_prefill", op="norm", rows=16384, groups=1, width=7680, dtype="bf16",
             centered=False, bias=False, shared=False, activation="none", gate="before"),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tables", "step", "scan", "scan", "norm"])
    dtype = rng.choice(["f32", "bf16"])
    if op == "tables":
        return dict(op=op, sequences=_spread(rng, 1, 4096), longest=_spread(rng, 1, 1000),
                    block=rng.choice([16, 64, 100, 256]), spare=rng.randrange(0, 500))
    hk = _spread(rng, 1, 16)
    heads = dict(hk=hk, hv=hk * rng.choice([1, 2]), k=rng.choice([64, 128]),
                 v=rng.choice([64, 128]), dtype=dtype)
    if op == "step":
        rows = _spread(rng, 1, 512)
        return dict(op=op, rows=rows, slots=rows + rng.randrange(0, 17), **heads)
    if op == "scan":
        n = _spread(rng, 1, 24)
        packed = rng.random() < 0.6
        tokens = _spread(rng, n, 32768 if dtype == "bf16" else 8192)
        if not packed:
            tokens = max(1, min(tokens, 16384) // n)
        elif tokens < n:
            tokens = n
        return dict(op=op, sequences=n, tokens=tokens, packed=packed, carried=rng.random() < 0.5,
                    **heads)
    groups = _spread(rng, 1, 64)
    return dict(op=op, rows=_spread(rng, 1, 16384), groups=groups,
                width=_spread(rng, 2, max(2, 7680 // groups)), dtype=dtype,
                centered=rng.random() < 0.5, bias=rng.random() < 0.5, shared=rng.random() < 0.5,
                activation=rng.choice(["none", "silu"]),
                gate=rng.choice(["none", "before", "after"]))


def _type(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _lengths(count, total, g):
    """Lengths of `count` requests that add up to `total`, from one token to long ones."""
    share = torch.rand(count, generator=g, device="cuda", dtype=torch.float64) ** 2 + 0.002
    cut = (share.cumsum(0) / share.sum() * (total - count)).long()
    cut[-1] = total - count
    return (torch.diff(cut, prepend=torch.zeros_like(cut[:1])) + 1).int()


def _parameters(heads, g):
    """Decay rates in [1, 16] and step sizes between 1e-3 and 1e-1, as the layers are set up."""
    u = torch.rand(2, heads, generator=g, device="cuda")
    dt = torch.exp(math.log(1e-3) + u[0] * (math.log(1e-1) - math.log(1e-3)))
    return torch.log(1 + 15 * u[1]), dt + torch.log(-torch.expm1(-dt))


def _rows(lead, case, g):
    """q, k, v and the raw step and write strengths of the tokens. Keys and queries share a common
    direction, as trained ones do, so that they are far from orthogonal; v comes out of a SiLU."""
    t = _type(case)

    def normal(*tail):
        return torch.randn(*lead, *tail, generator=g, device="cuda")

    common = torch.randn(case["hk"], case["k"], generator=g, device="cuda")
    q = (normal(case["hk"], case["k"]) + 0.7 * common).to(t)
    k = (normal(case["hk"], case["k"]) + 0.7 * common).to(t)
    v = torch.nn.functional.silu(normal(case["hv"], case["v"]) * 1.5).to(t)
    return q, k, v, normal(case["hv"]).to(t), normal(case["hv"]).to(t)


def prepare(case, seed):
    g = _generator(seed)
    s = dict(case=dict(case))
    if case["op"] == "tables":
        u = torch.rand(case["sequences"], generator=g, device="cuda")
        s["lengths"] = (u * (case["longest"] + 1)).int()
        # the packed buffer's rows, which the program knows from its own allocation
        s["total"] = case["sequences"] * case["longest"] + case["spare"]
        return s
    if case["op"] == "norm":
        t, c = _type(case), case["groups"] * case["width"]
        x = torch.randn(case["rows"], c, generator=g, device="cuda")
        # channels differ in scale and offset
        x = x * torch.exp(0.5 * torch.randn(c, generator=g, device="cuda")) + 0.3
        s["x"] = x.to(t)
        s["z"] = None
        if case["gate"] != "none":
            s["z"] = torch.randn(case["rows"], c, generator=g, device="cuda").to(t)
        w = case["width"] if case["shared"] else c
        s["weight"] = 1 + 0.2 * torch.randn(w, generator=g, device="cuda")
        s["bias"] = 0.2 * torch.randn(w, generator=g, device="cuda") if case["bias"] else None
        return s
    s["A_log"], s["dt_bias"] = _parameters(case["hv"], g)
    if case["op"] == "step":
        s["q"], s["k"], s["v"], s["dt_raw"], s["beta_raw"] = _rows((case["rows"],), case, g)
        # one state behind the pool's slots is spare
        s["state"] = torch.randn(case["slots"] + 1, case["hv"], case["v"], case["k"],
                                 generator=g, device="cuda") * 0.2
        slots = torch.randperm(case["slots"], generator=g, device="cuda")[:case["rows"]].int()
        if case["rows"] >= 8:  # a captured batch size with idle rows at its end
            slots[-(case["rows"] // 8):] = -1
        s["slots"] = slots
        s["y"] = torch.zeros_like(s["v"])
        return s
    n = case["sequences"]
    if case["packed"]:
        s["lengths"] = _lengths(n, case["tokens"], g)
        s["longest"] = int(s["lengths"].max())
        lead = (case["tokens"],)
    else:
        s["lengths"], s["longest"] = None, case["tokens"]
        lead = (n, case["tokens"])
    s["q"], s["k"], s["v"], s["dt_raw"], s["beta_raw"] = _rows(lead, case, g)
    s["state"] = None
    if case["carried"]:
        s["state"] = torch.randn(n, case["hv"], case["v"], case["k"], generator=g,
                                 device="cuda") * 0.2
    return s


def work(case):
    if case["op"] == "tables":
        n = case["sequences"]
        m = (n * case["longest"] + case["spare"]) // case["block"] + n
        return {"bytes": 4.0 * (n + 2 * (n + 1) + 2 * m), "flops": 0.0}
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "norm":
        c = case["groups"] * case["width"]
        tensors = 2 if case["gate"] == "none" else 3
        return {"bytes": float(e * tensors * case["rows"] * c), "flops": 10.0 * case["rows"] * c}
    kv = case["hv"] * case["k"] * case["v"]
    token = e * (2 * case["hk"] * case["k"] + 2 * case["hv"] * case["v"] + 2 * case["hv"])
    if case["op"] == "step":
        rows = case["rows"] - (case["rows"] // 8 if case["rows"] >= 8 else 0)
        return {"bytes": float(rows * (8 * kv + token)), "flops": 6.0 * rows * kv}
    n = case["sequences"]
    tokens = case["tokens"] if case["packed"] else n * case["tokens"]
    states = 2 if case["carried"] else 1
    return {"bytes": float(tokens * token + 4 * states * n * kv), "flops": 6.0 * tokens * kv}


# ---- the plain forms ---------------------------------------------------------------------------

def _tables(lengths, total, block, rows):
    """Starts of the packed sequences, starts of their blocks, and for each of `rows` blocks its
    sequence and first token (-1 behind the last)."""
    n = lengths.numel()
    zero = torch.zeros(1, dtype=torch.int64, device=lengths.device)
    starts = torch.cat([zero, lengths.long().clamp(min=0).cumsum(0)]).clamp(max=total)
    blocks = torch.cat([zero, ((torch.diff(starts) + block - 1) // block).cumsum(0)])
    at = torch.arange(rows, device=lengths.device)
    seq = torch.searchsorted(blocks[1:].contiguous(), at, right=True)
    live = seq < n
    i = seq.clamp(max=n - 1)
    first = starts[i] + (at - blocks[i]) * block
    minus = torch.full_like(at, -1)
    return (starts.int(), blocks.int(), torch.where(live, seq, minus).int(),
            torch.where(live, first, minus).int())


def _silu(x):
    return x / (1 + torch.exp(-x))


def _plain_norm(s):
    case = s["case"]
    x = s["x"].float()
    z = None if s["z"] is None else _silu(s["z"].float())
    if case["gate"] == "before":
        x = x * z
    u = x.view(case["rows"], case["groups"], case["width"])
    if case["centered"]:
        u = u - u.mean(-1, keepdim=True)
    u = u * torch.rsqrt((u * u).mean(-1, keepdim=True) + 1e-5)
    shape = (-1, case["width"])
    y = u * s["weight"].view(shape)
    if s["bias"] is not None:
        y = y + s["bias"].view(shape)
    if case["activation"] == "silu":
        y = _silu(y)
    y = y.reshape(case["rows"], -1)
    if case["gate"] == "after":
        y = y * z
    return y.to(s["x"].dtype)


def _unit(x):
    return x * torch.rsqrt((x * x).sum(-1, keepdim=True) + EPS_QK)


def _log_decay(dt_raw, s):
    """log a = -exp(A_log) dt, in 64 bits: it is summed over tokens."""
    v = dt_raw.double() + s["dt_bias"].double()
    dt = (torch.clamp(v, min=0) + torch.log1p(torch.exp(-v.abs()))).clamp(1e-4, 100.0)
    return -torch.exp(s["A_log"].double()) * dt


def _plain_step(s):
    case = s["case"]
    live = s["slots"] >= 0
    # idle rows read and write the spare state behind the pool
    slots = torch.where(live, s["slots"], case["slots"]).long()
    ratio = case["hv"] // case["hk"]
    q = _unit(s["q"].float()).repeat_interleave(ratio, 1) * case["k"] ** -0.5
    k = _unit(s["k"].float()).repeat_interleave(ratio, 1)
    a = torch.exp(_log_decay(s["dt_raw"], s)).float()
    beta = torch.sigmoid(s["beta_raw"].float())
    S = s["state"][slots] * a[..., None, None]
    d = beta[..., None] * (s["v"].float() - (S * k[:, :, None, :]).sum(-1))
    S = S + d[..., None] * k[:, :, None, :]
    y = (S * q[:, :, None, :]).sum(-1).to(s["y"].dtype)
    s["y"][:] = torch.where(live[:, None, None], y, s["y"])
    s["state"][slots] = S
    return s["y"], s["state"][:-1]


def _plain_scan(s):
    """The chunk form: everything inside the chunks at once, then the states chunk after chunk."""
    case = s["case"]
    n, hv, V, K = case["sequences"], case["hv"], case["v"], case["k"]
    ratio = hv // case["hk"]
    dev = s["q"].device
    tokens = s["q"].reshape(-1, case["hk"], K).shape[0]
    lengths = s["lengths"]
    if lengths is None:
        lengths = torch.full((n,), case["tokens"], dtype=torch.int32, device=dev)
    rows = tokens // CHUNK + n
    starts, chunk0, seq, first = (x.long() for x in _tables(lengths, tokens, CHUNK, rows))
    at = first[:, None] + torch.arange(CHUNK, device=dev)
    live = (seq[:, None] >= 0) & (at < starts[1:][seq.clamp(min=0)][:, None])
    at = torch.where(live, at, torch.zeros_like(at))

    def chunks(x, heads):  # (rows, heads, CHUNK, ...) in 32 bits, zero where there is no token
        x = x.reshape(tokens, heads, -1)[at] * 1.0
        x = torch.where(live[..., None, None], x.float(), torch.zeros((), device=dev))
        return x.transpose(1, 2)

    q = _unit(chunks(s["q"], case["hk"])).repeat_interleave(ratio, 1) * K ** -0.5
    k = _unit(chunks(s["k"], case["hk"])).repeat_interleave(ratio, 1)
    v = chunks(s["v"], hv)
    g = _log_decay(s["dt_raw"].reshape(tokens, hv)[at], s)
    g = torch.where(live[..., None], g, torch.zeros_like(g)).transpose(1, 2).cumsum(-1)
    beta = torch.sigmoid(s["beta_raw"].reshape(tokens, hv)[at].float())
    beta = torch.where(live[..., None], beta, torch.zeros_like(beta)).transpose(1, 2)
    i = torch.arange(CHUNK, device=dev)
    decay = torch.exp(torch.where(i[:, None] >= i, g[..., :, None] - g[..., None, :],
                                  torch.full((), -math.inf, dtype=g.dtype, device=dev)))
    # (I + M)^-1 = (I - M)(I + M^2)(I + M^4) ... for M strictly below the diagonal, in 64 bits:
    # the powers cancel where keys are alike
    M = (k @ k.transpose(-1, -2)).double() * decay * beta[..., None].double() * (i[:, None] > i)
    eye = torch.eye(CHUNK, dtype=torch.float64, device=dev)
    M2 = M @ M
    M4 = M2 @ M2
    M8 = M4 @ M4
    M16 = M8 @ M8
    T = (eye - M) @ (eye + M2) @ (eye + M4) @ (eye + M8) @ (eye + M16) @ (eye + M16 @ M16)
    T = (T * beta[..., None, :].double()).float()
    del M, M2, M4, M8, M16
    attend = (q @ k.transpose(-1, -2)) * decay.float()
    eg = torch.exp(g).float()
    to_end = torch.exp(g[..., -1:] - g).float()
    U, W = T @ v, T @ (k * eg[..., None])
    kd = k * to_end[..., None]
    end = eg[..., -1, None, None]
    S = s["state"]
    S = torch.zeros(n, hv, V, K, device=dev) if S is None else S
    entering = torch.empty(rows + 1, hv, V, K, device=dev)
    writes = torch.empty(rows + 1, hv, CHUNK, V, device=dev)
    for c in range((s["longest"] + CHUNK - 1) // CHUNK):
        here = chunk0[:-1] + c
        on = here < chunk0[1:]
        row = torch.where(on, here, torch.full_like(here, rows))
        here = here.clamp(max=rows - 1)
        d = U[here] - W[here] @ S.transpose(-1, -2)
        entering[row], writes[row] = S, d
        S = torch.where(on[:, None, None, None],
                        end[here] * S + d.transpose(-1, -2) @ kd[here], S)
    o = (q * eg[..., None]) @ entering[:-1].transpose(-1, -2) + attend @ writes[:-1]
    y = torch.empty(tokens + 1, hv, V, dtype=s["v"].dtype, device=dev)
    y[torch.where(live, at, torch.full_like(at, tokens))] = o.transpose(1, 2).to(y.dtype)
    return y[:-1].view(s["v"].shape), S


def run(s):
    case = s["case"]
    if own:
        import selective_state_space_depthwise_amd as axon

        if case["op"] == "tables":
            t = axon.sequence_tables(s["lengths"], s["total"], block=case["block"])
            return t.starts, t.block_starts, t.block_seq, t.block_first
        if case["op"] == "norm":
            return axon.group_norm(s["x"], case["groups"], s["weight"], s["bias"], s["z"],
                                   eps=1e-5, centered=case["centered"],
                                   activation=case["activation"], gate=case["gate"])
        if case["op"] == "step":
            y = axon.gated_delta_step(s["q"], s["k"], s["v"], s["dt_raw"], s["beta_raw"],
                                      s["A_log"], s["dt_bias"], s["state"], slots=s["slots"],
                                      y=s["y"])
            return y, s["state"][:-1]
        return axon.gated_delta_scan(s["q"], s["k"], s["v"], s["dt_raw"], s["beta_raw"],
                                     s["A_log"], s["dt_bias"], lengths=s["lengths"],
                                     state_in=s["state"])
    if case["op"] == "tables":
        rows = s["total"] // case["block"] + case["sequences"]
        return _tables(s["lengths"], s["total"], case["block"], rows)
    return {"norm": _plain_norm, "step": _plain_step, "scan": _plain_scan}[case["op"]](s)


# ---- the definition in 64 bits -----------------------------------------------------------------

def _token(S, q, k, v, a, beta, scale):
    """One token of the recurrence: S (..., V, K), q, k (..., K), v (..., V), a, beta (...)."""
    k = k / torch.sqrt((k * k).sum(-1, keepdim=True) + EPS_QK)
    q = q / torch.sqrt((q * q).sum(-1, keepdim=True) + EPS_QK)
    S = a[..., None, None] * S
    S = S + torch.einsum("...v,...k->...vk", beta[..., None]
                         * (v - torch.einsum("...vk,...k->...v", S, k)), k)
    return S, scale * torch.einsum("...vk,...k->...v", S, q)


def _gates(s):
    step = torch.nn.functional.softplus(s["dt_raw"].double() + s["dt_bias"].double(),
                                        threshold=1e9)
    a = torch.exp(-torch.exp(s["A_log"].double()) * step.clamp(1e-4, 100.0))
    return a, 1 / (1 + torch.exp(-s["beta_raw"].double()))


def exact(case, seed):
    if case["op"] == "tables":
        return None
    s = prepare(case, seed)
    if case["op"] == "norm":
        x = s["x"].double()
        gate = 1.0 if s["z"] is None else s["z"].double() * torch.sigmoid(s["z"].double())
        if case["gate"] == "before":
            x = x * gate
        x = x.unflatten(-1, (case["groups"], case["width"]))
        if case["centered"]:
            y = (x - x.mean(-1, keepdim=True)) / (x.var(-1, unbiased=False, keepdim=True)
                                                  + 1e-5).sqrt()
        else:
            y = x / ((x ** 2).mean(-1, keepdim=True) + 1e-5).sqrt()
        spread = (1, case["width"]) if case["shared"] else (case["groups"], case["width"])
        y = y * s["weight"].double().view(spread)
        if s["bias"] is not None:
            y = y + s["bias"].double().view(spread)
        y = (y * torch.sigmoid(y) if case["activation"] == "silu" else y).flatten(-2)
        return y * gate if case["gate"] == "after" else y
    a, beta = _gates(s)
    ratio, scale = case["hv"] // case["hk"], case["k"] ** -0.5
    if case["op"] == "step":
        y, pool = s["y"].double(), s["state"].double()
        for r, slot in enumerate(s["slots"].tolist()):
            if slot >= 0:
                pool[slot], y[r] = _token(
                    pool[slot], s["q"][r].double().repeat_interleave(ratio, 0),
                    s["k"][r].double().repeat_interleave(ratio, 0), s["v"][r].double(), a[r],
                    beta[r], scale)
        return y, pool[:-1]
    n, hv, V, K = case["sequences"], case["hv"], case["v"], case["k"]
    if s["lengths"] is None:
        lengths = [case["tokens"]] * n
    else:
        lengths = s["lengths"].tolist()
    flat = {x: s[x].flatten(0, -3) if x in "qkv" else None for x in ("q", "k", "v")}
    a, beta = a.reshape(-1, hv), beta.reshape(-1, hv)
    begin = [sum(lengths[:j]) for j in range(n)]
    S = torch.zeros(n, hv, V, K, dtype=torch.float64, device="cuda")
    if s["state"] is not None:
        S = s["state"].double()
    y = torch.zeros(flat["v"].shape, dtype=torch.float64, device="cuda")
    order = sorted(range(n), key=lambda j: -lengths[j])  # the longest first: rows fall away
    S = S[order]
    where = torch.tensor([begin[j] for j in order], device="cuda")
    for t in range(max(lengths)):
        m = sum(x > t for x in lengths)
        row = where[:m] + t
        S[:m], y[row] = _token(S[:m], flat["q"][row].double().repeat_interleave(ratio, 1),
                               flat["k"][row].double().repeat_interleave(ratio, 1),
                               flat["v"][row].double(), a[row], beta[row], scale)
    out = torch.empty_like(S)
    out[order] = S
    return y.view(s["v"].shape), out
