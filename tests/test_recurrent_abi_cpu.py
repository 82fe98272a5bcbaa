"""The C ABI of the linear recurrence, the causal convolution and the head norm with rotation on the
CPU: sizes and refusals. No call here passes the checks, so nothing reaches the GPU (fake pointers are
never dereferenced)."""
import ctypes

import pytest

from selective_state_space_depthwise_amd import _abi as A

P = 0x7F0000000000
G = 1 << 34
BAD, UNS, SMALL = A.AXON_ERR_INVALID_ARGUMENT, A.AXON_ERR_UNSUPPORTED, A.AXON_ERR_WORKSPACE_TOO_SMALL


def struct(cls, base, over):
    f = dict(base)
    assert set(over) <= set(f), over
    f.update(over)
    return cls(*[f[n] for n, _ in cls._fields_])


def call(name, structs, names, ws, over, unset=(), tail=(None,)):
    b = {n: P + (j + 1) * G for j, n in enumerate(names)}
    for n in unset:
        b[n] = None
    assert set(over) <= set(b), over
    b.update(over)
    size = () if ws is None else (ws,)
    return getattr(A.load(), name)(*structs, *[b[n] for n in names], *size, *tail)


def at(names, name):
    return P + (names.index(name) + 1) * G


# ---- linear --------------------------------------------------------------------------------------

LINEAR = dict(sequences=2, tokens=128, channels=40, x_stride=0, dt_stride=0, in_stride=0, dy_stride=0,
              state_slots=2, out_slots=2, act_dtype=0, gate=0, input_scale=2, clear_behind=0)
SCAN = ["x", "dt_raw", "in_raw", "tables", "state_in", "in_slots", "y", "state_out", "out_slots",
        "checkpoints", "workspace"]
BACK = ["dy", "x", "dt_raw", "in_raw", "tables", "checkpoints", "dstate_out", "dx", "ddt_raw",
        "din_raw", "dA_log", "ddt_bias", "din_bias", "dstate_in", "workspace"]
STEP = ["x", "dt_raw", "in_raw", "state", "slots", "y"]
PRM = dict(A_log=P, dt_bias=P + (1 << 28), in_bias=P + (2 << 28))


def lshape(**over):
    return struct(A.LinearShape, LINEAR, over)


def lparams(**over):
    return struct(A.LinearParams, PRM, over)


def scan(shape=None, params=None, ws=1 << 33, **over):
    return call("axon_linear_scan", (shape or lshape(), params or lparams()), SCAN, ws, over,
                unset=("tables", "in_slots", "out_slots"))


def back(shape=None, params=None, ws=1 << 33, **over):
    return call("axon_linear_scan_backward", (shape or lshape(), params or lparams()), BACK, ws, over,
                unset=("tables",))


def step(shape=None, params=None, **over):
    return call("axon_linear_step", (shape or lshape(tokens=2), params or lparams()), STEP, None, over,
                unset=("slots",))


@pytest.mark.parametrize("over,status", [
    (dict(sequences=0), BAD), (dict(tokens=-1), BAD), (dict(channels=0), BAD), (dict(x_stride=-1), BAD),
    (dict(dt_stride=39), BAD), (dict(in_stride=1), BAD), (dict(act_dtype=2), UNS), (dict(gate=2), UNS),
    (dict(gate=-1), UNS), (dict(input_scale=3), UNS), (dict(clear_behind=2), UNS),
    (dict(sequences=65536, tokens=65536), UNS), (dict(tokens=1 << 29), UNS),
    (dict(channels=(1 << 22) + 1), UNS), (dict(x_stride=(1 << 22) + 1), UNS),
    (dict(tokens=1 << 28, channels=1 << 20), UNS),
])
def test_linear_shapes(over, status):
    assert scan(lshape(**over)) == status
    assert back(lshape(**over)) == status
    assert step(lshape(**{"tokens": over.get("sequences", 2), **over})) == status
    assert A.load().axon_linear_scan_backward_workspace_bytes(lshape(**over)) == 0
    assert A.load().axon_linear_scan_workspace_bytes(lshape(**over)) == 0


def test_linear_slots_and_strides_of_one_direction():
    for over in (dict(state_slots=-1), dict(out_slots=-1)):
        assert scan(lshape(**over)) == BAD
    for over in (dict(state_slots=1 << 40), dict(out_slots=1 << 40)):
        assert scan(lshape(**over)) == UNS
    assert back(lshape(dy_stride=39)) == BAD and back(lshape(dy_stride=-1)) == BAD
    assert scan(lshape(state_slots=1)) == BAD and scan(lshape(out_slots=1)) == BAD
    assert scan(lshape(out_slots=3), state_out=at(SCAN, "state_in")) == BAD
    assert scan(lshape(tokens=127)) == BAD and back(lshape(tokens=127)) == BAD
    assert step(lshape(tokens=3)) == BAD and step(lshape(tokens=2, state_slots=1)) == BAD


@pytest.mark.parametrize("over", [dict(A_log=None), dict(A_log=P + 2), dict(dt_bias=P + 1),
                                  dict(in_bias=P + 3)])
def test_linear_params(over):
    for f in (scan, back, step):
        assert f(params=lparams(**over)) == BAD


def test_linear_pointers():
    for n in ("x", "dt_raw", "y"):
        assert scan(**{n: None}) == BAD and step(**{n: None}) == BAD
    for n in ("x", "dt_raw", "in_raw", "y"):
        assert scan(**{n: P + 2}) == BAD and step(**{n: P + 2}) == BAD
        assert scan(lshape(act_dtype=1), **{n: P + 1}) == BAD
    for n in ("tables", "state_in", "in_slots", "state_out", "out_slots", "checkpoints"):
        assert scan(**{n: at(SCAN, n) + 2}) == BAD
    for n in ("state", "slots"):
        assert step(**{n: at(STEP, n) + 2}) == BAD
    assert step(state=None) == BAD
    for n in ("dy", "x", "dt_raw", "checkpoints", "dx", "ddt_raw", "dA_log", "ddt_bias"):
        assert back(**{n: None}) == BAD and back(**{n: at(BACK, n) + 2}) == BAD
    for n in ("in_raw", "din_raw", "din_bias"):  # all or none
        assert back(**{n: None}) == BAD and back(**{n: at(BACK, n) + 2}) == BAD
    for n in ("tables", "dstate_out", "dstate_in"):
        assert back(**{n: at(BACK, n) + 2}) == BAD
    need = A.load().axon_linear_scan_backward_workspace_bytes(lshape())
    assert need > 0 and back(ws=need - 1) == SMALL
    assert back(workspace=None) == BAD and back(workspace=P + 8) == BAD
    lib = A.load()
    assert lib.axon_linear_scan(None, lparams(), *[None] * 11, 0, None) == BAD
    assert lib.axon_linear_scan(lshape(), None, *[None] * 11, 0, None) == BAD
    assert lib.axon_linear_step(None, None, *[None] * 7) == BAD
    assert lib.axon_linear_scan_backward(None, None, *[None] * 15, 0, None) == BAD


def test_linear_overlaps():
    outs = ("y", "state_out", "checkpoints")
    for o in outs:
        for r in ("x", "dt_raw", "in_raw", "tables", "state_in", "in_slots", "out_slots") + outs:
            if r == o or (o, r) == ("state_out", "state_in"):
                continue
            kw = {r: at(SCAN, r), o: at(SCAN, r)}
            assert scan(**kw) == BAD, (o, r)
        assert scan(**{o: P}) == BAD
    assert scan(state_out=at(SCAN, "state_in") + 4) == BAD
    assert scan(lshape(x_stride=100), y=at(SCAN, "x") + 4 * 50) == BAD  # between its rows
    outs = ("dx", "ddt_raw", "din_raw", "dA_log", "ddt_bias", "din_bias", "dstate_in", "workspace")
    for o in outs:
        for r in ("dy", "x", "dt_raw", "in_raw", "tables", "checkpoints", "dstate_out") + outs:
            if r != o:
                assert back(**{r: at(BACK, r), o: at(BACK, r)}) == BAD, (o, r)
        assert back(**{o: P}) == BAD
    for o in ("y", "state"):
        for r in ("x", "dt_raw", "in_raw", "slots", "y", "state"):
            if r != o:
                assert step(**{r: at(STEP, r), o: at(STEP, r)}) == BAD, (o, r)


@pytest.mark.parametrize("args,rows", [
    ((2, 128, 0), 2), ((2, 130, 0), 4), ((3, 0, 0), 0), ((3, 0, 1), 3), ((3, 100, 1), 4),
    ((1, 64, 1), 2), ((0, 10, 0), 0), ((65536, 65536, 0), 0), ((2, -1, 1), 0), ((2, 127, 0), 0),
    ((1, 1 << 29, 0), 0), ((1, 64, 2), 0),
])
def test_checkpoint_rows(args, rows):
    assert A.load().axon_linear_checkpoint_rows(*args) == rows


# ---- convolution ---------------------------------------------------------------------------------

CONV = dict(sequences=2, tokens=128, channels=40, x_stride=0, dy_stride=0, cache_slots=2, out_slots=2,
            act_dtype=0, activation=1, clear_behind=0)
CSCAN = ["x", "conv_w", "conv_b", "tables", "cache_in", "in_slots", "y", "cache_out", "out_slots"]
CBACK = ["dy", "x", "conv_w", "conv_b", "tables", "cache_in", "dcache_out", "dx", "dconv_w", "dconv_b",
         "dcache_in", "workspace"]
CSTEP = ["x", "conv_w", "conv_b", "cache", "slots", "y"]


def cshape(**over):
    return struct(A.ConvShape, CONV, over)


def conv(shape=None, **over):
    return call("axon_causal_conv", (shape or cshape(),), CSCAN, None, over,
                unset=("tables", "in_slots", "out_slots"))


def cback(shape=None, ws=1 << 33, **over):
    return call("axon_causal_conv_backward", (shape or cshape(),), CBACK, ws, over, unset=("tables",))


def cstep(shape=None, **over):
    return call("axon_causal_conv_step", (shape or cshape(tokens=2),), CSTEP, None, over,
                unset=("slots",))


@pytest.mark.parametrize("over,status", [
    (dict(sequences=0), BAD), (dict(tokens=-1), BAD), (dict(channels=0), BAD), (dict(x_stride=39), BAD),
    (dict(act_dtype=2), UNS), (dict(activation=2), UNS), (dict(clear_behind=-1), UNS),
    (dict(sequences=65536, tokens=65536), UNS), (dict(tokens=1 << 29), UNS),
    (dict(channels=(1 << 22) + 1), UNS), (dict(x_stride=(1 << 22) + 1), UNS),
    (dict(tokens=1 << 28, channels=1 << 20), UNS),
])
def test_conv_shapes(over, status):
    assert conv(cshape(**over)) == status
    assert cback(cshape(**over)) == status
    assert cstep(cshape(**{"tokens": over.get("sequences", 2), **over})) == status
    assert A.load().axon_causal_conv_backward_workspace_bytes(cshape(**over)) == 0


def test_conv_arguments():
    assert conv(cshape(cache_slots=1)) == BAD and conv(cshape(out_slots=1)) == BAD
    assert conv(cshape(cache_slots=-1)) == BAD and conv(cshape(out_slots=1 << 40)) == UNS
    assert conv(cshape(out_slots=3), cache_out=at(CSCAN, "cache_in")) == BAD
    assert conv(cshape(tokens=127)) == BAD and cback(cshape(tokens=127)) == BAD
    assert cback(cshape(dy_stride=20)) == BAD
    assert cstep(cshape(tokens=3)) == BAD and cstep(cshape(tokens=2, cache_slots=1)) == BAD
    for n in ("x", "conv_w", "y"):
        assert conv(**{n: None}) == BAD and cstep(**{n: None}) == BAD
    for n in CSCAN:
        assert conv(**{n: at(CSCAN, n) + 2}) == BAD
    for n in CSTEP:
        assert cstep(**{n: at(CSTEP, n) + 2}) == BAD
    assert cstep(cache=None) == BAD
    for n in ("dy", "x", "conv_w", "dx", "dconv_w", "dconv_b", "workspace"):
        assert cback(**{n: None}) == BAD
    for n in CBACK:
        assert cback(**{n: at(CBACK, n) + 2}) == BAD
    need = A.load().axon_causal_conv_backward_workspace_bytes(cshape())
    assert need > 0 and cback(ws=need - 1) == SMALL
    lib = A.load()
    assert lib.axon_causal_conv(None, *[None] * 10) == BAD
    assert lib.axon_causal_conv_backward(None, *[None] * 12, 0, None) == BAD
    assert lib.axon_causal_conv_step(None, *[None] * 7) == BAD


def test_conv_overlaps():
    for o in ("y", "cache_out"):
        for r in CSCAN:
            if r != o and (o, r) != ("cache_out", "cache_in"):
                assert conv(**{r: at(CSCAN, r), o: at(CSCAN, r)}) == BAD, (o, r)
    assert conv(cache_out=at(CSCAN, "cache_in") + 4) == BAD
    for o in ("dx", "dconv_w", "dconv_b", "dcache_in", "workspace"):
        for r in CBACK:
            if r != o:
                assert cback(**{r: at(CBACK, r), o: at(CBACK, r)}) == BAD, (o, r)
    for o in ("y", "cache"):
        for r in CSTEP:
            if r != o:
                assert cstep(**{r: at(CSTEP, r), o: at(CSTEP, r)}) == BAD, (o, r)


# ---- norm and rotation ---------------------------------------------------------------------------

ROT = dict(rows=10, q_heads=4, k_heads=2, head_dim=64, rotary_dim=32, q_stride=0, k_stride=0,
           dq_stride=0, dk_stride=0, eps=1e-6, act_dtype=0, interleaved=0)
RF = ["q", "k", "positions", "freqs", "q_weight", "k_weight", "q_out", "k_out"]
RB = ["dq_out", "dk_out", "q", "k", "positions", "freqs", "q_weight", "k_weight", "dq", "dk",
      "dq_weight", "dk_weight", "workspace"]


def desc(**over):
    return struct(A.NormRotateDesc, ROT, over)


def rot(d=None, **over):
    return call("axon_norm_rotate", (d or desc(),), RF, None, over)


def rback(d=None, ws=1 << 33, **over):
    return call("axon_norm_rotate_backward", (d or desc(),), RB, ws, over)


@pytest.mark.parametrize("over,status", [
    (dict(rows=-1), BAD), (dict(q_heads=0), BAD), (dict(k_heads=-1), BAD), (dict(head_dim=0), BAD),
    (dict(rotary_dim=0), BAD), (dict(rotary_dim=66), BAD), (dict(q_stride=255), BAD),
    (dict(k_stride=-1), BAD), (dict(eps=-1.0), BAD), (dict(eps=float("nan")), BAD),
    (dict(eps=float("inf")), BAD), (dict(head_dim=65), UNS), (dict(rotary_dim=31), UNS),
    (dict(head_dim=258), UNS), (dict(act_dtype=3), UNS), (dict(interleaved=2), UNS),
    (dict(q_heads=65536), UNS), (dict(k_heads=65536), UNS), (dict(rows=1 << 31), UNS),
    (dict(q_stride=(1 << 31) + 1), UNS), (dict(rows=1 << 30, q_stride=1 << 20), UNS),
])
def test_rotate_descs(over, status):
    assert rot(desc(**over)) == status
    assert rback(desc(**over)) == status
    assert A.load().axon_norm_rotate_backward_workspace_bytes(desc(**over)) == 0


def test_rotate_arguments():
    assert rback(desc(dq_stride=1)) == BAD and rback(desc(dk_stride=-1)) == BAD
    for n in ("q", "k", "positions", "freqs", "q_out", "k_out"):
        assert rot(**{n: None}) == BAD
    for n in RF:
        assert rot(**{n: at(RF, n) + 2}) == BAD
    assert rot(freqs=at(RF, "freqs") + 4) == BAD
    for n in ("dq_out", "dk_out", "q", "k", "positions", "freqs", "dq", "dk", "workspace"):
        assert rback(**{n: None}) == BAD
    for n in RB:
        assert rback(**{n: at(RB, n) + 2}) == BAD
    assert rback(desc(k_heads=0)) == BAD  # dk_weight without k
    need = A.load().axon_norm_rotate_backward_workspace_bytes(desc())
    assert need > 0 and rback(ws=need - 1) == SMALL
    assert A.load().axon_norm_rotate_backward_workspace_bytes(desc(rows=0)) == 0
    assert rot(desc(rows=0), **dict.fromkeys(RF)) == A.AXON_OK
    lib = A.load()
    assert lib.axon_norm_rotate(None, *[None] * 9) == BAD
    assert lib.axon_norm_rotate_backward(None, *[None] * 13, 0, None) == BAD


def test_rotate_overlaps():
    for o in ("q_out", "k_out"):
        for r in RF:
            if r != o and (o, r) not in (("q_out", "q"), ("k_out", "k")):
                assert rot(**{r: at(RF, r), o: at(RF, r)}) == BAD, (o, r)
    assert rot(q_out=at(RF, "q") + 4) == BAD
    assert rot(desc(q_stride=512), q_out=at(RF, "q")) == BAD
    for o in ("dq", "dk", "dq_weight", "dk_weight", "workspace"):
        for r in RB:
            if r != o and (o, r) not in (("dq", "dq_out"), ("dk", "dk_out")):
                assert rback(**{r: at(RB, r), o: at(RB, r)}) == BAD, (o, r)
    assert rback(dq=at(RB, "dq_out") + 4) == BAD
    assert rback(desc(dk_stride=512), dk=at(RB, "dk_out")) == BAD


# ---- the Python entry points, before anything reaches the library ---------------------------------

def test_python_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    import selective_state_space_depthwise_amd as axon

    x = torch.zeros(2, 3, 4)
    A_log = torch.zeros(4)
    with pytest.raises(ValueError):
        axon.linear_scan(x, x, A_log)
    with pytest.raises(ValueError):
        axon.linear_scan_backward(x, x, x, A_log, checkpoints=x)
    with pytest.raises(ValueError):
        axon.linear_checkpoints(x)
    with pytest.raises(ValueError):
        axon.linear_step(x[0], x[0], A_log, None, None, None, x[0])
    with pytest.raises(ValueError):
        axon.causal_conv(x, torch.zeros(4, 4))
    with pytest.raises(ValueError):
        axon.causal_conv_backward(x, x, torch.zeros(4, 4))
    with pytest.raises(ValueError):
        axon.causal_conv_step(x[0], torch.zeros(4, 4), None, x)
    with pytest.raises(ValueError):
        axon.norm_rotate(x, None, x, x)
    with pytest.raises(ValueError):
        axon.norm_rotate_backward(x, None, x, None, x, x)
    with pytest.raises(TypeError):
        axon.linear_scan([1.0], x, A_log)
