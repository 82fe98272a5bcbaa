"""The C ABI of the gated delta rule, the packed-sequence tables and the group norm on the CPU:
sizes and refusals. No call here passes the checks, so nothing reaches the GPU (fake pointers are
never dereferenced)."""
import ctypes

import pytest

from selective_state_space_depthwise_amd import _abi as A

P = 0x7F0000000000
MB = 1 << 20


def _shape(**over):
    f = dict(sequences=2, tokens=128, key_heads=2, value_heads=4, key_dim=128, value_dim=128,
             q_stride=0, k_stride=0, v_stride=0, state_slots=2, out_slots=2, act_dtype=A.AXON_F32)
    f.update(over)
    return A.GatedDeltaShape(*[f[n] for n, _ in A.GatedDeltaShape._fields_])


def _params(**over):
    f = dict(A_log=P, dt_bias=P + MB, dt_min=1e-4, dt_max=100.0, scale=0.1, eps=1e-6)
    f.update(over)
    return A.GatedDeltaParams(*[f[n] for n, _ in A.GatedDeltaParams._fields_])


NAMES = ["q", "k", "v", "dt_raw", "beta_raw", "tables", "state_in", "in_slots", "y", "state_out",
         "out_slots", "workspace"]


def _scan(shape=None, params=None, ws=1 << 40, **over):
    b = {n: P + (j + 1) * (1 << 30) for j, n in enumerate(NAMES)}
    b.update(tables=None, in_slots=None, out_slots=None)
    b.update(over)
    return A.raw_gated_delta_scan(shape or _shape(), params or _params(), *[b[n] for n in NAMES[:-1]],
                                  b["workspace"], ws, None)


def _step(shape=None, params=None, **over):
    names = ["q", "k", "v", "dt_raw", "beta_raw", "state", "slots", "y"]
    b = {n: P + (j + 1) * (1 << 30) for j, n in enumerate(names)}
    b.update(slots=None)
    b.update(over)
    return A.raw_gated_delta_step(shape or _shape(tokens=2), params or _params(),
                                  *[b[n] for n in names], None)


BAD, UNS, SMALL = A.AXON_ERR_INVALID_ARGUMENT, A.AXON_ERR_UNSUPPORTED, A.AXON_ERR_WORKSPACE_TOO_SMALL


@pytest.mark.parametrize("over,status", [
    (dict(sequences=0), BAD), (dict(tokens=-1), BAD), (dict(key_heads=0), BAD),
    (dict(value_heads=0), BAD), (dict(key_dim=0), BAD), (dict(value_dim=0), BAD),
    (dict(state_slots=-1), BAD), (dict(out_slots=-1), BAD), (dict(q_stride=-8), BAD),
    (dict(q_stride=128), BAD), (dict(k_stride=257), BAD), (dict(v_stride=504), BAD),
    (dict(value_heads=3), UNS), (dict(key_dim=96), UNS), (dict(key_dim=256), UNS),
    (dict(value_dim=24), UNS), (dict(value_dim=272), UNS), (dict(act_dtype=2), UNS),
    (dict(sequences=65536, tokens=65536), UNS), (dict(tokens=1 << 29), UNS),
    (dict(sequences=60000, tokens=60000, key_heads=20, value_heads=20), UNS),
    (dict(q_stride=1 << 40), UNS), (dict(state_slots=1 << 40), UNS), (dict(out_slots=1 << 40), UNS),
])
def test_shapes_refused(over, status):
    assert _scan(shape=_shape(**over)) == status
    if "act_dtype" in over or status == UNS:
        assert A.gated_delta_workspace_bytes(_shape(**over)) == 0
    if "out_slots" not in over or over["out_slots"] < 0:
        assert _step(shape=_shape(**{"tokens": over.get("sequences", 2), **over})) == status


@pytest.mark.parametrize("over", [
    dict(A_log=None), dict(dt_bias=None), dict(A_log=P + 4), dict(dt_min=-1.0), dict(dt_min=2.0, dt_max=1.0),
    dict(dt_max=float("inf")), dict(dt_min=float("nan")), dict(scale=float("nan")), dict(eps=0.0),
    dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
])
def test_params_refused(over):
    assert _scan(params=_params(**over)) == BAD
    assert _step(params=_params(**over)) == BAD


@pytest.mark.parametrize("name", ["q", "k", "v", "dt_raw", "beta_raw", "y"])
def test_null_and_misaligned(name):
    for p in (None, P + 8):
        assert _scan(**{name: p}) == BAD
        assert _step(**{name: p}) == BAD


def test_scan_refusals():
    assert _scan(shape=_shape(tokens=127)) == BAD          # not a multiple of sequences
    assert _scan(tables=P + 2) == BAD
    assert _scan(in_slots=P + 2) == BAD
    assert _scan(out_slots=P + 2) == BAD
    assert _scan(state_in=P + 4) == BAD
    assert _scan(state_out=P + 4) == BAD
    assert _scan(shape=_shape(state_slots=1)) == BAD       # fewer states than sequences, no slots
    assert _scan(shape=_shape(out_slots=1)) == BAD
    assert _scan(state_in=P + (7 << 30), state_out=P + (7 << 30),
                 shape=_shape(out_slots=3)) == BAD         # in place with two sizes
    assert _scan(workspace=None) == BAD
    assert _scan(workspace=P + 8) == BAD
    need = A.gated_delta_workspace_bytes(_shape())
    assert need > 0
    assert _scan(ws=need - 1) == SMALL
    assert A.gated_delta_workspace_bytes(_shape(tokens=0)) == 0
    assert A.load().axon_gated_delta_scan(None, ctypes.byref(_params()), *[None] * 12, 0, None) == BAD
    assert A.load().axon_gated_delta_scan(ctypes.byref(_shape()), None, *[None] * 12, 0, None) == BAD


def test_scan_overlaps_refused():
    at = {n: P + (j + 1) * (1 << 30) for j, n in enumerate(NAMES)}
    for out in ("y", "state_out", "workspace"):
        for other in ("q", "k", "v", "dt_raw", "beta_raw", "state_in", "y", "state_out", "workspace"):
            if out == other or (out == "state_out" and other == "state_in"):
                continue
            assert _scan(**{out: at[other]}) == BAD, (out, other)
        assert _scan(**{out: P}) == BAD
        assert _scan(tables=at["tables"], **{out: at["tables"]}) == BAD
        assert _scan(in_slots=at["in_slots"], **{out: at["in_slots"]}) == BAD
        assert _scan(out_slots=at["out_slots"], **{out: at["out_slots"]}) == BAD
    assert _scan(state_out=at["state_in"] + 16) == BAD
    # the rows of a strided input cover what lies between them
    assert _scan(shape=_shape(v_stride=1024), y=at["v"] + 2048) == BAD


def test_step_refusals():
    assert _step(shape=_shape(tokens=3)) == BAD            # one token a row
    assert _step(shape=_shape(tokens=2, state_slots=1)) == BAD
    assert _step(state=None) == BAD
    assert _step(state=P + 4) == BAD
    assert _step(slots=P + 1) == BAD
    at = {n: P + (j + 1) * (1 << 30) for j, n in
          enumerate(["q", "k", "v", "dt_raw", "beta_raw", "state", "slots", "y"])}
    for out in ("y", "state"):
        for other in ("q", "k", "v", "dt_raw", "beta_raw"):
            assert _step(**{out: at[other]}) == BAD, (out, other)
    assert _step(y=at["state"]) == BAD
    assert _step(slots=at["slots"], state=at["slots"]) == BAD


@pytest.mark.parametrize("n,total,block,status", [
    (0, 10, 64, BAD), (2, -1, 64, BAD), (2, 10, 0, BAD), (65536, 10, 64, UNS),
    (2, 1 << 31, 64, UNS), (2, (1 << 31) - 1, 1, UNS),
])
def test_tables_refused(n, total, block, status):
    assert A.sequence_tables_count(n, total, block) == 0
    assert A.raw_sequence_tables(n, total, block, P, P + MB, None) == status


def test_tables_pointers():
    assert A.sequence_tables_count(3, 100, 64) == 2 * 4 + 2 * (1 + 3)
    for a, b in ((None, P), (P, None), (P + 2, P + MB), (P, P + MB + 1), (P, P), (P + 4, P)):
        assert A.raw_sequence_tables(4, 100, 64, a, b, None) == BAD


def _desc(**over):
    f = dict(rows=4, groups=2, width=64, x_stride=0, z_stride=0, eps=1e-5, act_dtype=0, centered=1,
             activation=0, gate=0, shared_weights=0)
    f.update(over)
    return A.GroupNormDesc(*[f[n] for n, _ in A.GroupNormDesc._fields_])


@pytest.mark.parametrize("over,status", [
    (dict(rows=-1), BAD), (dict(groups=0), BAD), (dict(width=0), BAD), (dict(x_stride=-1), BAD),
    (dict(x_stride=127), BAD), (dict(gate=1, z_stride=100), BAD), (dict(eps=-1.0), BAD),
    (dict(eps=float("nan")), BAD), (dict(act_dtype=5), UNS), (dict(centered=2), UNS),
    (dict(activation=2), UNS), (dict(gate=3), UNS), (dict(shared_weights=7), UNS),
    (dict(width=1 << 30), UNS), (dict(rows=1 << 31), UNS), (dict(rows=1 << 30, width=1 << 12), UNS),
    (dict(x_stride=1 << 32), UNS),
])
def test_norm_shapes_refused(over, status):
    assert A.raw_group_norm(_desc(**over), P, P + MB, None, None, P + 2 * MB, None) == status


def test_norm_pointers():
    y = P + 8 * MB
    assert A.raw_group_norm(_desc(), None, None, None, None, y, None) == BAD
    assert A.raw_group_norm(_desc(), P, None, None, None, None, None) == BAD
    assert A.raw_group_norm(_desc(gate=2), P, None, None, None, y, None) == BAD
    assert A.raw_group_norm(_desc(), P + 2, None, None, None, y, None) == BAD
    assert A.raw_group_norm(_desc(), P, None, P + MB + 1, None, y, None) == BAD
    assert A.raw_group_norm(_desc(), P, None, None, P + MB + 2, y, None) == BAD
    assert A.raw_group_norm(_desc(gate=1), P, y, None, None, y, None) == BAD   # y over z
    assert A.raw_group_norm(_desc(), P, None, y, None, y, None) == BAD         # y over weight
    assert A.raw_group_norm(_desc(), P, None, None, y, y, None) == BAD
    assert A.raw_group_norm(_desc(), P, None, None, None, P + 4, None) == BAD  # partly over x
    assert A.raw_group_norm(_desc(x_stride=256), P, None, None, None, P, None) == BAD
    assert A.load().axon_group_norm(None, P, None, None, None, y, None) == BAD
