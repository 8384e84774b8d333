"""Outputs of the key-value cache operators that overlap other tensors of the call are refused on the
host, before any device call; what only lies near another tensor is not."""
import ctypes
import os

import pytest

import fp4_mqa_scoring_amd as mqa

P = ctypes.c_void_p
OVERLAP = -10


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(mqa.LIB_PATH):
        from fp4_mqa_scoring_amd import build
        build.build()
    return mqa.lib()


def test_the_code_has_a_name(lib):
    assert mqa.ERRORS[OVERLAP] == "MQA_ERR_OVERLAP" and b"overlaps" in lib.mqa_fp4_error_string(OVERLAP)


# acc: 3 rows of 20,000 floats every 30,000; the rest apart from it and each other
EVICT = dict(acc=0x10000000, lens=0x20000000, keep=0x30000000, kept=0x40000000, kept_acc=0x50000000, ws=0x60000000)
PITCH = 30000 * 4


@pytest.mark.parametrize("over,refused", [
    ({}, False),
    (dict(kept=EVICT["lens"]), False),              # in the lengths' place
    (dict(kept=EVICT["lens"] + 4), True), (dict(kept=EVICT["lens"] - 8), True), (dict(kept=EVICT["lens"] + 12), False),
    (dict(kept=EVICT["lens"] - 12), False),
    (dict(keep=EVICT["lens"]), True), (dict(keep=EVICT["lens"] - 1200), False), (dict(keep=EVICT["lens"] - 1196), True),
    (dict(kept_acc=EVICT["lens"]), True), (dict(ws=EVICT["lens"]), True),
    (dict(kept_acc=EVICT["acc"]), True), (dict(kept_acc=EVICT["acc"] - 1200), False), (dict(kept_acc=EVICT["acc"] - 1196), True),
    (dict(kept_acc=EVICT["acc"] + 80000), False),   # between the first row and the second
    (dict(kept_acc=EVICT["acc"] + 79996), True),
    (dict(kept_acc=EVICT["acc"] + PITCH - 1200), False), (dict(kept_acc=EVICT["acc"] + PITCH - 1196), True),
    (dict(kept_acc=EVICT["acc"] + 2 * PITCH + 79996), True), (dict(kept_acc=EVICT["acc"] + 2 * PITCH + 80000), False),
    (dict(keep=EVICT["acc"] + PITCH), True), (dict(kept=EVICT["acc"] + 4), True), (dict(ws=EVICT["acc"]), True),
    (dict(keep=EVICT["kept_acc"]), True), (dict(keep=EVICT["kept"]), True), (dict(kept=EVICT["kept_acc"] + 4), True),
    (dict(ws=EVICT["keep"]), True), (dict(ws=EVICT["kept_acc"]), True), (dict(kept_acc=None), False),
])
def test_eviction_s_choice(lib, over, refused):
    a = {k: None if x is None else P(x) for k, x in {**EVICT, **over}.items()}
    rc = lib.mqa_kv_evict_select(a["acc"], 30000, a["lens"], 3, 20000, 100, 10, a["keep"], a["kept"], a["kept_acc"], a["ws"],
                                 1 << 30, None)
    assert (rc == OVERLAP) == refused, rc


class Cache(ctypes.Structure):
    _fields_ = [("k", P), ("v", P), ("k_stride", ctypes.c_int64 * 3), ("v_stride", ctypes.c_int64 * 3),
                ("num_phys_pages", ctypes.c_int64), ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("type", ctypes.c_int32), ("k_scale", ctypes.c_float), ("v_scale", ctypes.c_float)]


class Query(ctypes.Structure):
    _fields_ = [("q", P), ("row_stride", ctypes.c_int64), ("num_rows", ctypes.c_int64), ("num_heads", ctypes.c_int32),
                ("type", ctypes.c_int32), ("scale", ctypes.c_float)]


ROWS, H, D = 4, 8, 128
ROW = H * D * 2         # bytes of a row of queries
ATTN = dict(q=0x10000000, out=0x20000000, lse=0x30000000, ws=0x40000000, table=0x50000000, seq=0x51000000,
            start=0x52000000, end=0x53000000, slots=0x54000000, count=0x55000000, acc=0x56000000)


def attention(lib, call, stride=H * D, rows=ROWS, acc_stride=320, **over):
    a = {k: None if x is None else P(x) for k, x in {**ATTN, **over}.items()}
    q = Query(a["q"], stride, rows, H, 0, 0.1)
    c = Cache(0x60000000, 0x61000000, (64 * 256, 256, 128), (64 * 256, 256, 128), 10, 2, D, 0, 1.0, 1.0)
    q, c = ctypes.byref(q), ctypes.byref(c)
    if call == "decode":
        return lib.mqa_kv_attention_decode(q, c, a["table"], 2, 5, a["seq"], a["start"], a["end"], a["out"], a["lse"], a["ws"],
                                           1 << 40, None)
    if call == "selected":
        return lib.mqa_kv_attention_selected(q, c, a["slots"], a["count"], 512, a["out"], a["lse"], a["ws"], 1 << 40, None)
    return lib.mqa_kv_weights_accumulate(q, a["lse"], c, a["table"], 2, 5, a["seq"], a["start"], a["end"], a["acc"], acc_stride,
                                         None)


Q0, O0 = ATTN["q"], ATTN["out"]


@pytest.mark.parametrize("call", ["decode", "selected"])
@pytest.mark.parametrize("over,refused", [
    ({}, False), (dict(out=Q0), False),                                          # in place
    (dict(out=Q0, stride=H * D + 8), True), (dict(out=Q0, stride=H * D + 8, rows=1), False), (dict(out=Q0 + 16), True),
    (dict(out=Q0 - 4 * ROW), False), (dict(out=Q0 - 4 * ROW + 16), True), (dict(out=Q0 + 4 * ROW), False),
    # one row of queries every six: out (four rows) fits behind one of them
    (dict(out=Q0 + ROW, stride=6 * H * D), False), (dict(out=Q0 + 2 * ROW, stride=6 * H * D), False),
    (dict(out=Q0 + 2 * ROW + 16, stride=6 * H * D), True), (dict(out=Q0 + 7 * ROW, stride=6 * H * D), False),
    (dict(out=Q0 + 19 * ROW - 16, stride=6 * H * D), True), (dict(out=Q0 + 19 * ROW, stride=6 * H * D), False),
    (dict(lse=Q0), True), (dict(lse=Q0 - 4 * 4 * H), False), (dict(lse=None), False), (dict(lse=O0 + 4), True),
    (dict(lse=O0 + 4 * ROW), False), (dict(ws=Q0), True), (dict(ws=O0), True), (dict(ws=ATTN["lse"]), True),
])
def test_attention(lib, call, over, refused):
    rc = attention(lib, call, **over)
    assert (rc == OVERLAP) == refused, rc


@pytest.mark.parametrize("call,names", [("decode", ["table", "seq", "start", "end"]), ("selected", ["slots", "count"])])
def test_attention_s_tables_and_lists(lib, call, names):
    for name in names:
        size = dict(table=2 * 5 * 4, slots=4 * 512 * 4).get(name, 16)
        for out in ("out", "lse", "ws"):
            assert attention(lib, call, **{out: ATTN[name]}) == OVERLAP, (name, out)
            assert attention(lib, call, **{name: ATTN[out] - size}) != OVERLAP, (name, out)
            assert attention(lib, call, **{name: ATTN[out] - size + 4}) == OVERLAP, (name, out)


def test_accumulated_weights(lib):
    call = lambda **over: attention(lib, "weights", **over)
    assert call() != OVERLAP
    for name, size in (("q", 4 * ROW), ("lse", 4 * 4 * H), ("table", 2 * 5 * 4), ("seq", 16), ("start", 16), ("end", 16)):
        assert call(**{name: ATTN["acc"] + 16}) == OVERLAP, name
        assert call(**{name: ATTN["acc"] - size}) != OVERLAP, name
        assert call(**{name: ATTN["acc"] - size + 16}) == OVERLAP, name
        # behind the first row's 320 sums, before the second's
        assert call(acc_stride=320 + size // 4, **{name: ATTN["acc"] + 1280}) != OVERLAP, name
        assert call(acc_stride=320 + size // 4, **{name: ATTN["acc"] + 1296}) == OVERLAP, name
    # records of 320 sums and one row of queries: nothing of them overlaps
    assert call(acc_stride=320 + ROW // 4, stride=320 * 2 + H * D, q=ATTN["acc"] + 1280, rows=2) != OVERLAP
    assert call(acc_stride=320 + ROW // 4, stride=320 * 2 + H * D, q=ATTN["acc"] + 1264, rows=2) == OVERLAP
