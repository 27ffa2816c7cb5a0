"""Host-side checks of the C ABI of the gated delta rule and the block norms (no
GPU needed): the library exports every function the headers declare, and invalid
arguments and empty problems come back as the documented status codes before
anything touches a device."""
import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x7F0000000000  # 16-byte aligned, never dereferenced by these calls
GB = 1 << 30


@pytest.fixture(scope="module")
def libs():
    from linear_rnn_state_gb300 import _build, blocknorm, gdr

    _build.build()
    gdr.load(), blocknorm.load()
    return gdr, blocknorm


@pytest.mark.parametrize("header,which", [("gdr.h", 0), ("blocknorm.h", 1)])
def test_exports_every_declared_function(libs, header, which):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", header)).read(), flags=re.S)
    prefix = header[:-2]
    declared = sorted(set(re.findall(r"\b(%s_\w+)\s*\(" % prefix, text)))
    assert declared and sorted(libs[which].EXPORTS) == declared
    lib = libs[which].load()
    for name in declared:
        assert len(getattr(lib, name).argtypes) == libs[which].EXPORTS[name], name


def test_buffer_sizes(libs):
    gdr = libs[0]
    full = gdr.saved_bytes(4, 4096, 32, 32, 64, 64, bf16=True, for_backward=True)
    # 8192 chunks of a head: q, k of 8 KB, T, P of 10 KB, states and u of 16 KB each
    assert 8192 * (16 + 20 + 32) * 1024 < full < 8192 * 76 * 1024
    assert gdr.saved_bytes(4, 4096, 32, 32, 64, 64, bf16=True, for_backward=False) < full
    assert gdr.saved_bytes(1, 64, 1, 1, 12, 64, bf16=True, for_backward=True) == 0
    assert gdr.saved_bytes(2, 64, 1, 1, 64, 64, 3, bf16=True, for_backward=True) == 0  # packed: one batch row
    # packed sequences get slots of their own
    assert gdr.saved_bytes(1, 64, 1, 1, 64, 64, 3, bf16=True, for_backward=False) > gdr.saved_bytes(
        1, 64, 1, 1, 64, 64, bf16=True, for_backward=False)


FWD = ("q", "k", "v", "g", "beta", "s_init", "seq_starts", "o", "s_final", "saved")
BWD = ("q", "k", "v", "g", "beta", "d_o", "dS_final", "seq_starts", "saved", "workspace", "dq", "dk", "dv", "dg", "dbeta", "dS_init")
STEP = ("q", "k", "v", "g", "beta", "state", "slots", "o")


def _call(lib, fn, names, tail, over):
    over = dict(over)
    strides = over.pop("strides", None)
    dims = {"B": 1, "T": 8, "Hk": 2, "Hv": 4, "K": 64, "V": 64, "nseq": -1, "n_slots": 4}
    dims.update({n: over.pop(n) for n in list(over) if n in dims})
    ptr = {n: FAKE + i * GB for i, n in enumerate(names)}
    ptr["seq_starts"] = None
    ptr.update(over)
    st = None if strides is None else (ctypes.c_longlong * 6)(*strides)
    return getattr(lib, fn)(*(ptr[n] for n in names), st, 1.0, *[dims.get(t, t) for t in tail], None)


def _forward(lib, over):
    return _call(lib, "gdr_forward_bf16", FWD, (0, 0, "B", "T", "Hk", "Hv", "K", "V", "nseq"), over)


def _backward(lib, over):
    return _call(lib, "gdr_backward", BWD, (0, "B", "T", "Hk", "Hv", "K", "V", "nseq"), over)


def _step(lib, over):
    return _call(lib, "gdr_step", STEP, (0, "B", "T", "Hk", "Hv", "K", "V", "n_slots"), over)


COMMON = [
    ("q_null", {"q": None}),
    ("beta_null", {"beta": None}),
    ("misaligned_v", {"v": FAKE + 8}),
    ("misaligned_g", {"g": FAKE + 2}),
    ("K_not_a_multiple_of_8", {"K": 60}),
    ("K_too_large", {"K": 136}),
    ("V_zero", {"V": 0}),
    ("heads", {"Hk": 3}),
    ("more_key_heads", {"Hk": 8}),
    ("negative_T", {"T": -1}),
    ("negative_B", {"B": -1}),
    ("stride_below_the_heads", {"strides": (0, 120, 0, 128, 0, 256)}),
    ("stride_not_a_multiple_of_8", {"strides": (0, 132, 0, 128, 0, 256)}),
    ("too_large", {"B": 1 << 20, "T": 1 << 20, "Hk": 1 << 10, "Hv": 1 << 10}),
]
BAD_FWD = COMMON + [
    ("o_null", {"o": None}),
    ("saved_null", {"saved": None}),
    ("o_overlaps_q", {"o": FAKE + 16}),
    ("saved_overlaps_v", {"saved": FAKE + 2 * GB - 64}),
    ("packed_batches", {"seq_starts": FAKE + 100 * GB, "B": 2, "nseq": 2}),
    ("packed_without_a_count", {"seq_starts": FAKE + 100 * GB, "nseq": -1}),
]
BAD_BWD = COMMON + [
    ("d_o_null", {"d_o": None}),
    ("dg_null", {"dg": None}),
    ("workspace_null", {"workspace": None}),
    ("dq_overlaps_d_o", {"dq": FAKE + 5 * GB + 16}),
    ("dk_overlaps_dq", {"dk": FAKE + 10 * GB + 16}),
    ("dS_init_overlaps_dS_final", {"dS_init": FAKE + 6 * GB}),
]
BAD_STEP = COMMON + [
    ("state_null", {"state": None}),
    ("fewer_states_than_requests", {"B": 5, "slots": None}),
    ("negative_slots", {"n_slots": -1}),
    ("o_overlaps_state", {"o": FAKE + 5 * GB + 64}),
    ("state_overlaps_k", {"state": FAKE + GB + 64}),
]


@pytest.mark.parametrize("case,over", BAD_FWD, ids=[c for c, _ in BAD_FWD])
def test_forward_rejects_invalid_arguments(libs, case, over):
    assert _forward(libs[0].load(), over) == -2
    assert libs[0].wkv7.last_error()


@pytest.mark.parametrize("case,over", BAD_BWD, ids=[c for c, _ in BAD_BWD])
def test_backward_rejects_invalid_arguments(libs, case, over):
    assert _backward(libs[0].load(), over) == -2


@pytest.mark.parametrize("case,over", BAD_STEP, ids=[c for c, _ in BAD_STEP])
def test_step_rejects_invalid_arguments(libs, case, over):
    assert _step(libs[0].load(), over) == -2


def test_empty_problems_need_no_device(libs):
    lib = libs[0].load()
    none = {n: None for n in FWD}
    for dims in ({"B": 0}, {"Hk": 0, "Hv": 0}, {"T": 0}):
        assert _forward(lib, {**none, **dims}) == 0
        assert _backward(lib, {**{n: None for n in BWD}, **dims}) == 0
        assert _step(lib, {**{n: None for n in STEP}, **dims, "n_slots": 1}) == 0


ADD_F = ("x", "residual", "weight", "scale", "h", "n", "rstd")
ADD_B = ("x", "residual", "weight", "scale", "rstd", "dn", "dh", "dresidual", "dx", "dweight", "dscale", "part")
GATED_F = ("o", "z", "weight", "y", "rstd")
GATED_B = ("o", "z", "weight", "rstd", "dy", "d_o", "dz", "dweight", "part")


def _norm(lib, fn, names, over, *, eps, gated):
    over = dict(over)
    d = {"s0": 64, "s1": 64, "rows": 10, "H": 2, "D": 32, "bf16": 1, "rbf16": 1}
    d.update({n: over.pop(n) for n in list(over) if n in d})
    ptr = {n: FAKE + i * GB for i, n in enumerate(names)}
    ptr.update(over)
    tail = [d["s0"], d["s1"], d["rows"]] + ([d["H"]] if gated else []) + [d["D"]] + ([1e-6] if eps else []) + [d["bf16"]]
    return getattr(lib, fn)(*(ptr[n] for n in names), *tail, *([] if gated else [d["rbf16"]]), None)


BAD_NORM = [
    ("rows_negative", {"rows": -1}),
    ("D_zero", {"D": 0}),
    ("D_too_large", {"D": 8200, "s0": 16400, "s1": 16400}),
    ("stride_below_the_row", {"s0": 16}),
    ("weight_null", {"weight": None}),
    ("too_many_rows", {"rows": 1 << 40}),
]


@pytest.mark.parametrize("case,over", BAD_NORM, ids=[c for c, _ in BAD_NORM])
def test_norms_reject_invalid_arguments(libs, case, over):
    lib = libs[1].load()
    assert _norm(lib, "blocknorm_add_forward", ADD_F, over, eps=True, gated=False) == -2
    assert _norm(lib, "blocknorm_add_backward", ADD_B, over, eps=False, gated=False) == -2
    assert _norm(lib, "blocknorm_gated_forward", GATED_F, over, eps=True, gated=True) == -2
    assert _norm(lib, "blocknorm_gated_backward", GATED_B, over, eps=False, gated=True) == -2


def test_norms_reject_mismatched_arguments(libs):
    lib = libs[1].load()

    def add(over):
        return _norm(lib, "blocknorm_add_forward", ADD_F, over, eps=True, gated=False)

    assert add({"bf16": 0, "rbf16": 1}) == -2  # fp32 x, bfloat16 residual
    assert add({"x": None}) == -2  # scale and h without x
    assert add({"h": None}) == -2
    assert add({"n": FAKE + GB}) == -2  # over residual
    assert add({"h": FAKE + GB + 16}) == -2  # near residual, but not it
    assert add({"h": FAKE + GB}) == -2  # residual with rows apart
    bad = {"scale": None}
    assert _norm(lib, "blocknorm_add_backward", ADD_B, bad, eps=False, gated=False) == -2  # dscale without scale
    assert _norm(lib, "blocknorm_add_backward", ADD_B, {"dx": None}, eps=False, gated=False) == -2
    assert _norm(lib, "blocknorm_gated_backward", GATED_B, {"part": None}, eps=False, gated=True) == -2


def test_norms_of_no_rows_need_no_device(libs):
    lib = libs[1].load()
    assert _norm(lib, "blocknorm_add_forward", ADD_F, {"rows": 0}, eps=True, gated=False) == 0
    assert _norm(lib, "blocknorm_gated_forward", GATED_F, {"rows": 0}, eps=True, gated=True) == 0
    assert libs[1].load().blocknorm_part_bytes(0, 64, 2) > 0
    assert libs[1].load().blocknorm_part_bytes(1 << 20, 64, 1) == 152 * 4 * 64 * 4
    assert libs[1].load().blocknorm_part_bytes(5, 0, 1) == 0
