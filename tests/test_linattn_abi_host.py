"""Host-side checks of the C ABI of linear attention with a decay and of the norms
of queries and keys with the rotation (no GPU needed): the library exports every
function the headers declare, and invalid arguments and empty problems come back as
the documented status codes before anything touches a device."""
import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x7F0000000000  # 16-byte aligned, never dereferenced by these calls
GB = 1 << 30


@pytest.fixture(scope="module")
def libs():
    from linear_rnn_state_gb300 import _build, linattn, qkrope

    _build.build()
    linattn.load(), qkrope.load()
    return linattn, qkrope


@pytest.mark.parametrize("header,which", [("linattn.h", 0), ("qkrope.h", 1)])
def test_exports_every_declared_function(libs, header, which):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", header)).read(), flags=re.S)
    declared = sorted(set(re.findall(r"\b(%s_\w+)\s*\(" % header[:-2], text)))
    assert declared and sorted(libs[which].EXPORTS) == declared
    lib = libs[which].load()
    for name in declared:
        assert len(getattr(lib, name).argtypes) == libs[which].EXPORTS[name], name


def test_buffer_sizes(libs):
    la = libs[0]
    full = la.saved_bytes(4, 4096, 32, 32, 64, 64, bf16=True, for_backward=True)
    assert full == 4096 * 24 * 1024  # 4 x 32 chunks x 32 heads of 64 x 64 numbers in three 16-bit parts
    assert la.saved_bytes(4, 4096, 32, 32, 64, 64, bf16=True, for_backward=False) == 0
    # a long sequence of few heads goes in segments, with states of their own
    assert la.saved_bytes(1, 65536, 2, 2, 64, 64, bf16=True, for_backward=False) > 0
    assert la.saved_bytes(1, 64, 1, 1, 12, 64, bf16=True, for_backward=True) == 0
    assert la.saved_bytes(2, 64, 1, 1, 64, 64, 3, bf16=True, for_backward=True) == 0  # packed: one batch row
    # packed sequences get slots of their own
    assert la.saved_bytes(1, 128, 1, 1, 64, 64, 3, bf16=True, for_backward=True) > la.saved_bytes(
        1, 128, 1, 1, 64, 64, bf16=True, for_backward=True)
    lib = la.load()
    per_token = lib.linattn_backward_bytes(1, 128, 1, 1, 64, 64, -1, 0, 1)
    assert lib.linattn_backward_bytes(1, 128, 1, 1, 64, 64, -1, 1, 1) > per_token > 0  # fixed decays: dg of the tokens


@pytest.mark.parametrize("bf16,K,V", [(True, 64, 64), (True, 128, 128), (True, 16, 72), (False, 64, 64), (False, 32, 16)])
def test_one_packed_sequence_is_planned_as_a_dense_one(libs, bf16, K, V):
    """In segments, which need states of their own, or whole: no more than the sequence is taken for its length. (Were it three
    times that, 96 heads of 64 and 8192 tokens would go in segments: 100 steps after one another for 66.)"""
    size = lambda T, H, nseq: libs[0].saved_bytes(1, T, H, H, K, V, nseq, bf16=bf16, for_backward=False)
    ways = set()
    for T in (100, 1024, 2100, 4096, 8192, 20000, 65536):
        for H in (1, 2, 8, 17, 32, 40, 64, 76, 80, 96, 128, 152, 160, 300):
            dense, packed = size(T, H, -1), size(T, H, 1)
            assert (dense == 0) == (packed == 0), (T, H)
            ways.add(dense == 0)
    assert ways == {True, False}


def test_packed_sequences_are_not_longer_than_all_tokens(libs):
    """Two and three sequences: at most as in one, beside the others."""
    size = lambda H, nseq: libs[0].saved_bytes(1, 8192, H, H, 64, 64, nseq, bf16=True, for_backward=False)
    assert all(size(H, n) == 0 for H in (96, 128) for n in (1, 2, 3))
    assert all(size(4, n) > 0 for n in (1, 2, 3))


FWD = ("q", "k", "v", "g", "s_init", "seq_starts", "o", "s_final", "saved")
BWD = ("q", "k", "v", "g", "d_o", "dS_final", "seq_starts", "saved", "workspace", "dq", "dk", "dv", "dg", "dS_init")
STEP = ("q", "k", "v", "g", "state", "slots", "o")


def _call(lib, fn, names, tail, over):
    over = dict(over)
    strides = over.pop("strides", None)
    # long enough for segments, so that `saved` is needed in every call
    dims = {"B": 1, "T": 2048, "Hk": 2, "Hv": 4, "K": 64, "V": 64, "nseq": -1, "n_slots": 4, "fixed": 0, "bf16": 1}
    dims.update({n: over.pop(n) for n in list(over) if n in dims})
    ptr = {n: FAKE + i * GB for i, n in enumerate(names)}
    ptr["seq_starts"] = None
    ptr.update(over)
    st = None if strides is None else (ctypes.c_longlong * 6)(*strides)
    return getattr(lib, fn)(*(ptr[n] for n in names), st, 1.0, *[dims.get(t, t) for t in tail], None)


def _forward(lib, over):
    return _call(lib, "linattn_forward", FWD, ("fixed", 1, "B", "T", "Hk", "Hv", "K", "V", "nseq", "bf16"), over)


def _backward(lib, over):
    return _call(lib, "linattn_backward", BWD, ("fixed", "B", "T", "Hk", "Hv", "K", "V", "nseq", "bf16"), {"bf16": 0, **over})


def _step(lib, over):
    return _call(lib, "linattn_step", STEP, ("fixed", "B", "T", "Hk", "Hv", "K", "V", "n_slots", "bf16"), {"T": 1, **over})


COMMON = [
    ("q_null", {"q": None}),
    ("g_null", {"g": None}),
    ("misaligned_v", {"v": FAKE + 8}),
    ("misaligned_g", {"g": FAKE + 2}),
    ("K_not_a_multiple_of_8", {"K": 60}),
    ("K_too_large", {"K": 136}),
    ("V_zero", {"V": 0}),
    ("heads", {"Hk": 3}),
    ("more_key_heads", {"Hk": 8}),
    ("negative_T", {"T": -1}),
    ("T_too_large", {"T": (1 << 30) + 1}),
    ("negative_B", {"B": -1}),
    ("stride_below_the_heads", {"T": 8, "strides": (0, 120, 0, 128, 0, 256)}),
    ("stride_not_a_multiple_of_8", {"T": 8, "strides": (0, 132, 0, 128, 0, 256)}),
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
    ("workspace_null", {"workspace": None}),
    ("dq_overlaps_d_o", {"dq": FAKE + 4 * GB + 16}),
    ("dk_overlaps_dq", {"dk": FAKE + 9 * GB + 16}),
    ("dg_overlaps_g", {"dg": FAKE + 3 * GB + 12, "fixed": 1}),  # (g: four numbers)
    ("dS_init_overlaps_dS_final", {"dS_init": FAKE + 5 * GB}),
]
BAD_STEP = [c for c in COMMON if c[0] not in ("stride_below_the_heads", "stride_not_a_multiple_of_8")] + [
    ("state_null", {"state": None}),
    ("fewer_states_than_requests", {"B": 5, "slots": None}),
    ("negative_slots", {"n_slots": -1}),
    ("o_overlaps_state", {"o": FAKE + 4 * GB + 64}),
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
    for dims in ({"B": 0}, {"Hk": 0, "Hv": 0}, {"T": 0}):
        assert _forward(lib, {**{n: None for n in FWD}, **dims}) == 0
        assert _backward(lib, {**{n: None for n in BWD}, **dims}) == 0
        assert _step(lib, {**{n: None for n in STEP}, **dims, "n_slots": 1}) == 0


ROPE_F = ("q", "k", "q_weight", "k_weight", "freq", "positions", "q_out", "k_out")
ROPE_B = ("q", "k", "q_weight", "k_weight", "freq", "positions", "dq_out", "dk_out", "dq", "dk", "dq_weight", "dk_weight", "part")


def _rope(lib, fn, names, over):
    over = dict(over)
    d = {"qs": 4 * 64, "ks": 2 * 64, "tokens": 10, "T": 10, "Hq": 4, "Hk": 2, "D": 64, "half": 32}
    d.update({n: over.pop(n) for n in list(over) if n in d})
    ptr = {n: FAKE + i * GB for i, n in enumerate(names)}
    ptr.update(over)
    return getattr(lib, fn)(*(ptr[n] for n in names), *d.values(), 0, 1e-6, 1, None)


BAD_ROPE = [
    ("tokens_negative", {"tokens": -1}),
    ("D_not_a_multiple_of_8", {"D": 60}),
    ("D_too_large", {"D": 264, "qs": 4 * 264, "ks": 2 * 264}),
    ("more_pairs_than_half", {"half": 33}),
    ("half_negative", {"half": -1}),
    ("stride_below_the_heads", {"qs": 248}),
    ("stride_not_a_multiple_of_8", {"ks": 132}),
    ("weight_null", {"k_weight": None}),
    ("freq_null", {"freq": None}),
    ("q_null", {"q": None}),
    ("misaligned_k", {"k": FAKE + GB + 8}),
    ("no_positions_and_no_T", {"positions": None, "T": 0}),
    ("too_many_rows", {"tokens": 1 << 30, "Hq": 1 << 10, "qs": 1 << 16}),
]


@pytest.mark.parametrize("case,over", BAD_ROPE, ids=[c for c, _ in BAD_ROPE])
def test_rotation_rejects_invalid_arguments(libs, case, over):
    lib = libs[1].load()
    assert _rope(lib, "qkrope_forward", ROPE_F, over) == -2
    assert _rope(lib, "qkrope_backward", ROPE_B, over) == -2


@pytest.mark.parametrize("half", [(1 << 31) - 1, 1 << 30, (1 << 30) + 5])
def test_rotation_rejects_counts_of_pairs_past_32_bits(libs, half):
    """Twice the number is below 0 or small in 32 bits."""
    lib = libs[1].load()
    assert _rope(lib, "qkrope_forward", ROPE_F, {"half": half, "freq": FAKE + 1000 * GB}) == -2
    assert _rope(lib, "qkrope_backward", ROPE_B, {"half": half, "freq": FAKE + 1000 * GB}) == -2
    assert "half" in libs[1].wkv7.last_error()


def test_rotation_rejects_mismatched_buffers(libs):
    lib = libs[1].load()
    assert _rope(lib, "qkrope_forward", ROPE_F, {"q_out": FAKE}) == -2  # over q
    assert _rope(lib, "qkrope_forward", ROPE_F, {"k_out": FAKE + 6 * GB + 16}) == -2  # over q_out
    assert _rope(lib, "qkrope_backward", ROPE_B, {"part": None}) == -2
    assert _rope(lib, "qkrope_backward", ROPE_B, {"dk": FAKE + 7 * GB}) == -2


def test_rotation_of_nothing_needs_no_device(libs):
    lib = libs[1].load()
    assert _rope(lib, "qkrope_forward", ROPE_F, {"tokens": 0}) == 0
    assert _rope(lib, "qkrope_forward", ROPE_F, {"Hq": 0, "Hk": 0, **{n: None for n in ROPE_F}}) == 0
    assert lib.qkrope_part_bytes(0, 4, 2, 64) > 0
    assert lib.qkrope_part_bytes(5, 4, 2, 60) == 0
