"""CPU checks of the C ABI and binding of norm, rotation, appending and attention over caches in 4 bits: what the host
refuses before any device call."""
import ctypes
import os
import re

import pytest
import torch

import fp4_mqa_scoring_amd as mqa

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P, I64, I32, F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float
NULL, MISALIGNED, SIZE, DEVICE, HIP, UNSUPPORTED, OVERLAP = -2, -3, -4, -5, -7, -9, -10
INF, NAN = float("inf"), float("nan")


class Rows(ctypes.Structure):
    _fields_ = [("x", P), ("row_stride", I64), ("out", P), ("out_stride", I64), ("weight", P), ("weight_offset", F), ("num_heads", I32)]


class Turn(ctypes.Structure):
    _fields_ = [("inv_freq", P), ("position", P), ("rotary_dim", I32), ("rotary_offset", I32), ("interleaved", I32), ("eps", F)]


class New(ctypes.Structure):
    _fields_ = [("k", Rows), ("v", Rows), ("num_rows", I64), ("type", I32), ("block_table", P), ("num_seqs", I64), ("max_pages", I64),
                ("seq_of_row", P), ("position", P), ("turn", Turn)]


class Cache(ctypes.Structure):
    _fields_ = [("k", P), ("v", P), ("k_stride", I64 * 3), ("v_stride", I64 * 3), ("num_phys_pages", I64), ("num_kv_heads", I32),
                ("head_dim", I32), ("type", I32), ("k_scale", F), ("v_scale", F)]


class Fp4(ctypes.Structure):
    _fields_ = [("k", P), ("v", P), ("k_scale", P), ("v_scale", P), ("k_stride", I64 * 3), ("v_stride", I64 * 3),
                ("k_scale_stride", I64 * 3), ("v_scale_stride", I64 * 3), ("num_phys_pages", I64), ("num_kv_heads", I32), ("head_dim", I32)]


class Query(ctypes.Structure):
    _fields_ = [("q", P), ("row_stride", I64), ("num_rows", I64), ("num_heads", I32), ("type", I32), ("scale", F)]


def test_packed_structures_have_the_header_s_layout():
    assert mqa._KV_ROWS.size == ctypes.sizeof(Rows) and mqa._KV_TURN.size == ctypes.sizeof(Turn)
    assert 2 * mqa._KV_ROWS.size + mqa._KV_NEW.size + mqa._KV_TURN.size == ctypes.sizeof(New)
    assert mqa._KV_CACHE_FP4.size == ctypes.sizeof(Fp4)
    r = Rows.from_buffer_copy(mqa._KV_ROWS.pack(1, 2, 3, 4, 5, 0.5, 6))
    assert (r.x, r.row_stride, r.out, r.out_stride, r.weight, r.weight_offset, r.num_heads) == (1, 2, 3, 4, 5, 0.5, 6)
    n = New.from_buffer_copy(bytes(96) + mqa._KV_NEW.pack(1, 2, 3, 4, 5, 6, 7) + mqa._KV_TURN.pack(8, 9, 10, 11, 12, 0.25))
    assert (n.num_rows, n.type, n.block_table, n.num_seqs, n.max_pages, n.seq_of_row, n.position) == (1, 2, 3, 4, 5, 6, 7)
    t = n.turn
    assert (t.inv_freq, t.position, t.rotary_dim, t.rotary_offset, t.interleaved, t.eps) == (8, 9, 10, 11, 12, 0.25)
    c = Fp4.from_buffer_copy(mqa._KV_CACHE_FP4.pack(*range(1, 20)))
    assert (c.k, c.v, c.k_scale, c.v_scale, list(c.k_stride), list(c.v_scale_stride), c.num_phys_pages, c.num_kv_heads,
            c.head_dim) == (1, 2, 3, 4, [5, 6, 7], [14, 15, 16], 17, 18, 19)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(mqa.LIB_PATH):
        from fp4_mqa_scoring_amd import build
        build.build()
    return mqa.lib()


def test_library_exports_every_declared_symbol(lib):
    names = set()
    for header in ("mqa_kv_append.h", "mqa_kv_fp4.h"):
        text = open(os.path.join(ROOT, "include", header)).read()
        names |= set(re.findall(r"^\s*(?:int32_t|int64_t)\s+(mqa_kv_\w+)\s*\(", text, re.M))
    assert names == {"mqa_kv_norm_rotate", "mqa_kv_append", "mqa_kv_append_fp4", "mqa_kv_attention_decode_fp4",
                     "mqa_kv_attention_selected_fp4"}
    for n in names:
        assert hasattr(lib, n) and hasattr(mqa, n), n


# 5 rows, 4 query and 2 key heads of 128 dims, every tensor far from the others
Q, QO, K, KO, V, POS, TPOS, SEQ, TABLE, FREQ, W, CK, CV, KS, VS, OUT, WS = (0x10000000 * (i + 1) for i in range(17))


def rows(at, to=None, heads=2, **over):
    a = dict(x=at, row_stride=1024, out=to, out_stride=1024, weight=None, weight_offset=0.0, num_heads=heads)
    a.update(over)
    return Rows(**a)


def turn(**over):
    a = dict(inv_freq=FREQ, position=TPOS, rotary_dim=64, rotary_offset=0, interleaved=0, eps=1e-6)
    a.update(over)
    return Turn(**a)


def rotate(lib, q={}, k=None, t={}, n=5, D=128, type=0):
    q = rows(Q, QO, 4, **q)
    k = None if k is None else ctypes.byref(rows(K, KO, 2, **k))
    return lib.mqa_kv_norm_rotate(ctypes.byref(q), k, ctypes.byref(turn(**t)), n, D, type, None)


def append(lib, k={}, v={}, q=None, t={}, c={}, fp4=False, **over):
    a = dict(num_rows=5, type=0, block_table=TABLE, num_seqs=3, max_pages=7, seq_of_row=SEQ, position=POS)
    a.update(over)
    new = New(k=rows(K, **k), v=rows(V, **v), turn=turn(**t), **a)
    q = None if q is None else ctypes.byref(rows(Q, QO, 4, **q))
    call = lib.mqa_kv_append_fp4 if fp4 else lib.mqa_kv_append
    return call(ctypes.byref(new), q, ctypes.byref((fp4_cache if fp4 else cache)(**c)), None)


def strided(cls, defaults, over):
    strides = {n: over.pop(n, defaults.pop(n)) for n in [n for n in defaults if n.endswith("stride")]}
    c = cls(**{**defaults, **over})
    for n, s in strides.items():
        getattr(c, n)[:] = s
    return c


def cache(**over):
    return strided(Cache, dict(k=CK, v=CV, k_stride=(64 * 256, 256, 128), v_stride=(64 * 256, 256, 128), num_phys_pages=10, num_kv_heads=2,
                               head_dim=128, type=0, k_scale=1.0, v_scale=1.0), over)


def fp4_cache(**over):
    codes, scales = (64 * 128, 128, 64), (64 * 8, 8, 4)
    return strided(Fp4, dict(k=CK, v=CV, k_scale=KS, v_scale=VS, k_stride=codes, v_stride=codes, k_scale_stride=scales,
                             v_scale_stride=scales, num_phys_pages=10, num_kv_heads=2, head_dim=128), over)


def passes(rc):
    """Nothing on the host refuses: what fails is the device."""
    return rc in (DEVICE, HIP)


def test_good_calls_reach_the_device(lib):
    assert passes(rotate(lib)) and passes(rotate(lib, k={})) and passes(rotate(lib, t=dict(inv_freq=None, position=None)))
    assert passes(rotate(lib, q=dict(out=Q))) and passes(rotate(lib, q=dict(weight=W), k=dict(weight=W)))
    for fp4 in (False, True):
        assert passes(append(lib, fp4=fp4)) and passes(append(lib, fp4=fp4, q={})) and passes(append(lib, fp4=fp4, v=dict(x=None)))
        assert passes(append(lib, fp4=fp4, t=dict(position=None))) and passes(append(lib, fp4=fp4, c=dict(num_phys_pages=0, k=None, v=None)))
        assert passes(append(lib, fp4=fp4, v=dict(x=None), c=dict(v=None)))
    assert passes(append(lib, c=dict(type=2, k_scale=0.5, v_scale=3.0)))
    # the page stride of one page and the head stride of one head are not looked at
    one = dict(num_phys_pages=1, num_kv_heads=1)
    assert passes(append(lib, k=dict(num_heads=1), v=dict(num_heads=1), c=dict(k_stride=(-5, 128, -7), v_stride=(3, 128, 1), **one)))
    assert passes(append(lib, fp4=True, k=dict(num_heads=1), v=dict(num_heads=1), c=dict(k_stride=(-5, 64, -7), k_scale_stride=(3, 4, 1), **one)))
    assert passes(rotate(lib, q=dict(row_stride=7, out_stride=-3), n=1))


@pytest.mark.parametrize("code,over", [
    (UNSUPPORTED, dict(type=2)), (UNSUPPORTED, dict(type=-1)), (UNSUPPORTED, dict(D=96)), (UNSUPPORTED, dict(D=0)),
    (SIZE, dict(n=-1)), (SIZE, dict(n=1 << 24)), (SIZE, dict(q=dict(num_heads=0))), (SIZE, dict(q=dict(num_heads=65537))),
    (SIZE, dict(q=dict(row_stride=511))), (SIZE, dict(q=dict(out_stride=504))), (SIZE, dict(k=dict(row_stride=(1 << 32) + 8))),
    (SIZE, dict(q=dict(weight_offset=INF))), (SIZE, dict(k=dict(weight_offset=NAN))),
    (MISALIGNED, dict(q=dict(row_stride=516))), (MISALIGNED, dict(q=dict(x=Q + 8))), (MISALIGNED, dict(q=dict(out=QO + 2))),
    (MISALIGNED, dict(q=dict(weight=W + 8))), (MISALIGNED, dict(t=dict(inv_freq=FREQ + 2))), (MISALIGNED, dict(t=dict(position=TPOS + 1))),
    (NULL, dict(q=dict(x=None))), (NULL, dict(q=dict(out=None))), (NULL, dict(k=dict(out=None))), (NULL, dict(t=dict(position=None))),
    (SIZE, dict(t=dict(eps=-1e-6))), (SIZE, dict(t=dict(eps=NAN))), (SIZE, dict(t=dict(eps=INF, inv_freq=None))),
    (SIZE, dict(t=dict(rotary_dim=0))), (SIZE, dict(t=dict(rotary_dim=24))), (SIZE, dict(t=dict(rotary_dim=144))),
    (SIZE, dict(t=dict(rotary_offset=4))), (SIZE, dict(t=dict(rotary_offset=-8))), (SIZE, dict(t=dict(rotary_offset=72))),
    (SIZE, dict(t=dict(interleaved=2))), (SIZE, dict(t=dict(interleaved=-1))),
])
def test_norm_and_rotation_are_checked_on_the_host(lib, code, over):
    assert rotate(lib, **over) == code


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("code,over", [
    (UNSUPPORTED, dict(type=2)), (SIZE, dict(num_rows=-1)), (SIZE, dict(num_rows=1 << 24)), (SIZE, dict(num_seqs=-1)),
    (SIZE, dict(max_pages=-1)), (SIZE, dict(max_pages=(1 << 31) // 64)), (SIZE, dict(num_seqs=1 << 20, max_pages=1 << 12)),
    (SIZE, dict(k=dict(num_heads=3))), (SIZE, dict(v=dict(num_heads=1))), (SIZE, dict(v=dict(row_stride=248))),
    (SIZE, dict(t=dict(rotary_dim=160))), (SIZE, dict(q=dict(num_heads=0))), (SIZE, dict(c=dict(num_kv_heads=0))),
    (SIZE, dict(c=dict(num_phys_pages=-1))), (SIZE, dict(c=dict(num_phys_pages=(1 << 31) // 64))),
    (UNSUPPORTED, dict(c=dict(head_dim=32))),
    (NULL, dict(k=dict(x=None))), (NULL, dict(block_table=None)), (NULL, dict(seq_of_row=None)), (NULL, dict(position=None)),
    (NULL, dict(c=dict(k=None))), (NULL, dict(c=dict(v=None))), (NULL, dict(q=dict(out=None))),
    (MISALIGNED, dict(k=dict(x=K + 4))), (MISALIGNED, dict(c=dict(k=CK + 8))), (MISALIGNED, dict(position=POS + 2)),
    (MISALIGNED, dict(k=dict(weight=W + 2))), (MISALIGNED, dict(v=dict(row_stride=260))),
])
def test_appending_is_checked_on_the_host(lib, fp4, code, over):
    assert append(lib, fp4=fp4, **over) == code


@pytest.mark.parametrize("code,over", [
    (UNSUPPORTED, dict(type=1)), (UNSUPPORTED, dict(type=3)), (SIZE, dict(k_scale=0.5)), (SIZE, dict(v_scale=0.0)),
    (SIZE, dict(type=2, k_scale=0.0)), (SIZE, dict(type=2, v_scale=-1.0)), (SIZE, dict(type=2, k_scale=NAN)), (SIZE, dict(type=2, v_scale=INF)),
    (SIZE, dict(k_stride=(-64, 256, 128))), (SIZE, dict(k_stride=(1 << 30, 1 << 25, 128))), (SIZE, dict(v_stride=(1 << 35, 256, 128))),
    (MISALIGNED, dict(v_stride=(64 * 256, 256, 132))), (MISALIGNED, dict(k_stride=(64 * 256, 257, 128))),
])
def test_caches_to_write_are_checked_on_the_host(lib, code, over):
    assert append(lib, c=over) == code


FP4_REFUSED = [
    (SIZE, dict(k_stride=(-16, 128, 64))), (SIZE, dict(v_stride=(1 << 36, 128, 64))), (SIZE, dict(k_stride=(1 << 30, 1 << 26, 64))),
    (SIZE, dict(k_scale_stride=(512, 1 << 26, 4))), (SIZE, dict(v_scale_stride=(512, 8, 1 << 31))), (SIZE, dict(k_scale_stride=(512, -8, 4))),
    (MISALIGNED, dict(k_stride=(64 * 128, 128, 72))), (MISALIGNED, dict(v_stride=(64 * 128 + 8, 128, 64))),
    (MISALIGNED, dict(k_scale_stride=(512, 8, 2))), (MISALIGNED, dict(v_scale_stride=(513, 8, 4))), (MISALIGNED, dict(k_scale=KS + 2)),
    (MISALIGNED, dict(v_scale=VS + 1)), (MISALIGNED, dict(v=CV + 8)), (NULL, dict(k_scale=None)), (NULL, dict(v_scale=None)),
]


@pytest.mark.parametrize("code,over", FP4_REFUSED)
def test_caches_in_4_bits_are_checked_on_the_host(lib, code, over):
    for call in (lambda c: append(lib, fp4=True, c=c), lambda c: decode(lib, c=c), lambda c: selected(lib, c=c)):
        assert call(dict(over)) == code


def query(**over):
    a = dict(q=Q, row_stride=1024, num_rows=5, num_heads=8, type=0, scale=0.1)
    a.update(over)
    return Query(**a)


def decode(lib, q={}, c={}, n_seq=3, pages=7, ws=WS, size=1 << 40, out=OUT, lse=None, seq=SEQ, table=TABLE):
    return lib.mqa_kv_attention_decode_fp4(ctypes.byref(query(**q)), ctypes.byref(fp4_cache(**c)), table, n_seq, pages, seq, POS, TPOS,
                                           out, lse, ws, size, None)


def selected(lib, q={}, c={}, K=512, ws=WS, size=1 << 40, out=OUT, lse=None, slots=TABLE, count=SEQ):
    return lib.mqa_kv_attention_selected_fp4(ctypes.byref(query(**q)), ctypes.byref(fp4_cache(**c)), slots, count, K, out, lse, ws, size, None)


@pytest.mark.parametrize("call", [decode, selected])
@pytest.mark.parametrize("code,over", [
    (UNSUPPORTED, dict(q=dict(type=2))), (UNSUPPORTED, dict(c=dict(head_dim=96))), (UNSUPPORTED, dict(c=dict(head_dim=0))),
    (SIZE, dict(q=dict(num_heads=7))), (SIZE, dict(c=dict(num_kv_heads=0))), (SIZE, dict(q=dict(num_rows=-1))), (SIZE, dict(q=dict(scale=NAN))),
    (SIZE, dict(q=dict(row_stride=1016))), (SIZE, dict(size=255)), (MISALIGNED, dict(q=dict(row_stride=1028))), (MISALIGNED, dict(ws=WS + 128)),
    (MISALIGNED, dict(out=OUT + 8)), (NULL, dict(q=dict(q=None))), (NULL, dict(out=None)), (NULL, dict(ws=None)), (NULL, dict(c=dict(k=None))),
    (OVERLAP, dict(out=WS)), (OVERLAP, dict(out=Q + 16)), (OVERLAP, dict(lse=OUT)), (OVERLAP, dict(out=TABLE)), (OVERLAP, dict(lse=SEQ)),
])
def test_attention_over_4_bits_is_checked_on_the_host(lib, call, code, over):
    assert call(lib, **over) == code


def test_good_attention_calls_reach_the_device(lib):
    for call in (decode, selected):
        assert passes(call(lib)) and passes(call(lib, c=dict(num_phys_pages=0, k=None, v=None, k_scale=None, v_scale=None)))
    assert decode(lib, n_seq=-1) == SIZE and decode(lib, pages=1 << 26) == SIZE and selected(lib, K=-1) == SIZE


@pytest.mark.parametrize("over,refused", [
    ({}, False), (dict(q=dict(out=Q)), False),                                      # in place
    (dict(q=dict(out=Q, out_stride=2048)), True), (dict(q=dict(out=Q + 16)), True),
    (dict(q=dict(out=Q + 1024)), False), (dict(q=dict(out=Q + 1008)), True),        # beside x in one row of 1,024 numbers
    (dict(k=dict(x=Q + 1024, out=Q + 1024)), False), (dict(q=dict(out=Q), k=dict(x=Q + 1024, out=Q + 1024)), False),
    (dict(q=dict(out=Q + 1024), k=dict(x=Q + 1024)), True), (dict(k=dict(out=QO)), True), (dict(k=dict(out=QO + 1024)), False),
    (dict(q=dict(out=K)), False), (dict(k=dict(x=K), q=dict(out=K)), True), (dict(q=dict(out=FREQ - 16)), True),
    (dict(q=dict(out=TPOS)), True), (dict(q=dict(weight=QO)), True), (dict(k=dict(weight=QO + 512)), True),
])
def test_overlapping_rows_are_refused(lib, over, refused):
    rc = rotate(lib, **over)
    assert (rc == OVERLAP) == refused and (refused or passes(rc)), rc


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("over,refused", [
    (dict(q=dict(out=Q)), False), (dict(q=dict(out=K)), True), (dict(q=dict(out=V)), True), (dict(q=dict(out=SEQ)), True),
    (dict(q=dict(out=POS)), True), (dict(q=dict(out=TABLE)), True), (dict(q=dict(x=K + 512, out=K + 512)), False),
])
def test_overlapping_queries_of_an_append_are_refused(lib, fp4, over, refused):
    rc = append(lib, fp4=fp4, **over)
    assert (rc == OVERLAP) == refused and (refused or passes(rc)), rc


# --- the binding -------------------------------------------------------------------------------------


def tensors(T=5, H=4, Hkv=2, D=64, kind=torch.bfloat16):
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)  # noqa: E731
    x = lambda h: torch.zeros(T, h, D, dtype=kind)  # noqa: E731
    return dict(q=x(H), q_out=x(H), k=x(Hkv), v=x(Hkv), k_out=x(Hkv), pages=torch.zeros(3, 64, Hkv, D, dtype=kind), codes=u8(3, 64, Hkv, D // 2),
                scales=u8(3, 64, Hkv, D // 32), table=i32(2, 4), seq=i32(T), pos=i32(T), freq=torch.zeros(D // 2), w=torch.zeros(D, dtype=kind),
                ws=u8(1 << 22), slots=i32(T, 8), start=i32(T))


def refused(call, *args, **kw):
    with pytest.raises((TypeError, ValueError)) as e:
        call(*args, **kw)
    return str(e.value)


def test_binding_refuses_rows_of_the_wrong_kind():
    t = tensors()
    good = dict(position=t["pos"], inv_freq=t["freq"])
    call = mqa.mqa_kv_norm_rotate
    assert "q must be bfloat16" in refused(call, t["q"].float(), t["q_out"].float(), **good)
    assert "[T, H, D]" in refused(call, t["q"][0], t["q_out"][0], **good)
    assert "q_out" in refused(call, t["q"], t["q_out"][:4], **good) and "q_out" in refused(call, t["q"], None, **good)
    assert "contiguous" in refused(call, t["q"].transpose(0, 1).contiguous().transpose(0, 1), t["q_out"], **good)
    assert "k must be" in refused(call, t["q"], t["q_out"], k=t["k"][:3], k_out=t["k_out"][:3], **good)
    assert "k_out" in refused(call, t["q"], t["q_out"], k=t["k"], **good)
    assert "go with k" in refused(call, t["q"], t["q_out"], k_weight=t["w"], **good)
    assert "q_weight" in refused(call, t["q"], t["q_out"], q_weight=t["w"][:32], **good)
    assert "q_weight" in refused(call, t["q"], t["q_out"], q_weight=t["w"].float(), **good)
    assert "position" in refused(call, t["q"], t["q_out"], position=t["pos"].long(), inv_freq=t["freq"])
    assert "inv_freq" in refused(call, t["q"], t["q_out"], position=t["pos"], inv_freq=t["freq"].double())


def test_binding_refuses_caches_of_the_wrong_kind():
    t = tensors()
    rest = (t["table"], t["seq"], t["pos"])
    call = mqa.mqa_kv_append
    assert "k_pages must be" in refused(call, t["k"], t["v"], t["pages"].half(), t["pages"].half(), *rest)
    assert "v_pages must be" in refused(call, t["k"], t["v"], t["pages"], t["pages"].to(torch.float8_e4m3fn), *rest)
    assert "k_pages must be" in refused(call, t["k"], t["v"], t["pages"][:, :32], t["pages"], *rest)
    assert "go together" in refused(call, t["k"], None, t["pages"], t["pages"], *rest)
    assert "position" in refused(call, t["k"], t["v"], t["pages"], t["pages"], t["table"], t["seq"], t["pos"][:3])
    assert "block_table" in refused(call, t["k"], t["v"], t["pages"], t["pages"], t["table"][0], t["seq"], t["pos"])
    assert "v must be" in refused(call, t["k"], t["v"][:, :, :32], t["pages"], t["pages"], *rest)
    assert "go with q" in refused(call, t["k"], t["v"], t["pages"], t["pages"], *rest, q_out=t["q_out"])
    assert "v must be" in refused(call, t["k"], t["v"].half(), t["pages"], t["pages"], *rest)
    call, c, s = mqa.mqa_kv_append_fp4, t["codes"], t["scales"]
    assert "k_pages must be" in refused(call, t["k"], t["v"], c[..., :16], s, c, s, *rest)
    assert "k_scale must be" in refused(call, t["k"], t["v"], c, s[..., :1], c, s, *rest)
    assert "v_scale must be" in refused(call, t["k"], t["v"], c, s, c, None, *rest)
    assert "v_pages must be" in refused(call, t["k"], t["v"], c, s, c.short(), s, *rest)
    assert "key heads" in refused(call, t["k"][:, :1], t["v"][:, :1], c, s, c, s, *rest)
    for call, lists in ((mqa.mqa_kv_attention_decode_fp4, (t["table"], t["seq"], t["start"], t["start"])),
                        (mqa.mqa_kv_attention_selected_fp4, (t["slots"], t["start"]))):
        assert "k_scale must be" in refused(call, t["q"], c, s[:2], c, s, *lists, t["q_out"], t["ws"])
        assert "query heads" in refused(call, t["q"][:, :3].contiguous(), c, s, c, s, *lists, t["q_out"][:, :3].contiguous(), t["ws"])
        assert "v_pages" in refused(call, t["q"], c, s, None, None, *lists, t["q_out"], t["ws"])
        assert "out must be" in refused(call, t["q"], c, s, c, s, *lists, t["q_out"][:2], t["ws"])


def test_good_binding_calls_reach_the_library():
    """On host tensors they end at the device checks."""
    t = tensors()
    rest, c, s = (t["table"], t["seq"], t["pos"]), t["codes"], t["scales"]
    for call in (lambda: mqa.mqa_kv_norm_rotate(t["q"], t["q_out"], t["pos"], k=t["k"], k_out=t["k_out"], inv_freq=t["freq"], q_weight=t["w"], stream=0),
                 lambda: mqa.mqa_kv_append(t["k"], t["v"], t["pages"], t["pages"].clone(), *rest, inv_freq=t["freq"], q=t["q"], q_out=t["q_out"], stream=0),
                 lambda: mqa.mqa_kv_append(t["k"], None, t["pages"].to(torch.float8_e4m3fn), None, *rest, k_scale=0.5, stream=0),
                 lambda: mqa.mqa_kv_append_fp4(t["k"], t["v"], c, s, c.clone(), s.clone(), *rest, stream=0),
                 lambda: mqa.mqa_kv_append_fp4(t["k"], None, c, s, None, None, *rest, stream=0)):
        with pytest.raises(mqa.MQAError) as e:
            call()
        assert e.value.code in (DEVICE, HIP)
