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
