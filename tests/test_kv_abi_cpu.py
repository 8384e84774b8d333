"""CPU checks of the key-value cache operators' C ABI and binding: what the host
refuses before any device call."""
import ctypes
import os
import re

import pytest
import torch

import fp4_mqa_scoring_amd as mqa

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "mqa_kv_cache.h")
P = ctypes.c_void_p
p = P(0x1000)
NULL, MISALIGNED, SIZE, UNSUPPORTED = -2, -3, -4, -9


class Cache(ctypes.Structure):
    _fields_ = [("k", P), ("v", P), ("k_stride", ctypes.c_int64 * 3), ("v_stride", ctypes.c_int64 * 3),
                ("num_phys_pages", ctypes.c_int64), ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("type", ctypes.c_int32), ("k_scale", ctypes.c_float), ("v_scale", ctypes.c_float)]


class Query(ctypes.Structure):
    _fields_ = [("q", P), ("row_stride", ctypes.c_int64), ("num_rows", ctypes.c_int64), ("num_heads", ctypes.c_int32),
                ("type", ctypes.c_int32), ("scale", ctypes.c_float)]


class Array(ctypes.Structure):
    _fields_ = [("src", P), ("dst", P), ("src_stride", ctypes.c_int64 * 3), ("dst_stride", ctypes.c_int64 * 3),
                ("row_bytes", ctypes.c_int64), ("rows_per_position", ctypes.c_int64)]


def test_packed_structures_have_the_header_s_layout():
    for packed, plain in ((mqa._KV_CACHE, Cache), (mqa._KV_QUERY, Query), (mqa._KV_ARRAY, Array)):
        assert packed.size == ctypes.sizeof(plain)
    c = Cache.from_buffer_copy(mqa._KV_CACHE.pack(1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11, 12, 0.5, 0.25))
    assert (c.k, c.v, list(c.k_stride), list(c.v_stride), c.num_phys_pages, c.num_kv_heads, c.head_dim, c.type, c.k_scale,
            c.v_scale) == (1, 2, [3, 4, 5], [6, 7, 8], 9, 10, 11, 12, 0.5, 0.25)
    q = Query.from_buffer_copy(mqa._KV_QUERY.pack(1, 2, 3, 4, 5, 0.5))
    assert (q.q, q.row_stride, q.num_rows, q.num_heads, q.type, q.scale) == (1, 2, 3, 4, 5, 0.5)
    a = Array.from_buffer_copy(mqa._KV_ARRAY.pack(*range(1, 11)))
    assert (a.src, a.dst, list(a.src_stride), list(a.dst_stride), a.row_bytes, a.rows_per_position) == (
        1, 2, [3, 4, 5], [6, 7, 8], 9, 10)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(mqa.LIB_PATH):
        from fp4_mqa_scoring_amd import build
        build.build()
    return mqa.lib()


def test_library_exports_every_declared_symbol(lib):
    names = set(re.findall(r"^\s*(?:int32_t|int64_t)\s+(mqa_kv_\w+)\s*\(", open(HEADER).read(), re.M))
    assert names == {"mqa_kv_attention_decode", "mqa_kv_attention_decode_workspace_bytes", "mqa_kv_attention_selected",
                     "mqa_kv_attention_selected_workspace_bytes", "mqa_kv_weights_accumulate", "mqa_kv_evict_select",
                     "mqa_kv_evict_workspace_bytes", "mqa_kv_compact"}
    for n in names:
        assert hasattr(lib, n) and hasattr(mqa, n), n
    assert b"unsupported type" in lib.mqa_fp4_error_string(UNSUPPORTED)
    assert mqa.ERRORS[UNSUPPORTED] == "MQA_ERR_UNSUPPORTED"


def query(**over):
    a = dict(q=0x1000, row_stride=8 * 128, num_rows=4, num_heads=8, type=0, scale=0.1)
    a.update(over)
    return Query(**a)


def cache(**over):
    k_stride, v_stride = over.pop("k_stride", (64 * 256, 256, 128)), over.pop("v_stride", (64 * 256, 256, 128))
    a = dict(k=0x1000, v=0x1000, num_phys_pages=10, num_kv_heads=2, head_dim=128, type=0, k_scale=1.0, v_scale=1.0)
    a.update(over)
    c = Cache(**a)
    c.k_stride[:] = k_stride
    c.v_stride[:] = v_stride
    return c


def decode(lib, q=None, c=None, n_seq=2, pages=5, ws=p, ws_bytes=1 << 40, out=p, lse=None, seq=p, table=p):
    return lib.mqa_kv_attention_decode(ctypes.byref(q or query()), ctypes.byref(c or cache()), table, n_seq, pages, seq, p,
                                       p, out, lse, ws, ws_bytes, None)


def selected(lib, q=None, c=None, K=512, ws=p, ws_bytes=1 << 40, out=p, slots=p, count=p):
    return lib.mqa_kv_attention_selected(ctypes.byref(q or query()), ctypes.byref(c or cache()), slots, count, K, out, None,
                                         ws, ws_bytes, None)


def weights(lib, q=None, c=None, n_seq=2, pages=5, lse=p, acc=p, stride=320):
    return lib.mqa_kv_weights_accumulate(ctypes.byref(q or query()), lse, ctypes.byref(c or cache()), p, n_seq, pages, p, p,
                                         p, acc, stride, None)


@pytest.mark.parametrize("call", [decode, selected, weights])
@pytest.mark.parametrize("code,q,c", [
    (UNSUPPORTED, dict(type=2), {}), (UNSUPPORTED, dict(type=7), {}), (UNSUPPORTED, dict(type=-1), {}),
    (UNSUPPORTED, {}, dict(type=1)), (UNSUPPORTED, {}, dict(type=3)), (UNSUPPORTED, {}, dict(head_dim=96)),
    (UNSUPPORTED, {}, dict(head_dim=0)),
    (SIZE, dict(num_heads=0), {}), (SIZE, dict(num_heads=7), {}), (SIZE, {}, dict(num_kv_heads=0)), (SIZE, dict(num_heads=65538), {}),
    (SIZE, dict(num_rows=-1), {}), (SIZE, dict(num_rows=1 << 24), {}), (SIZE, dict(row_stride=8 * 128 - 8), {}),
    (SIZE, dict(scale=float("inf")), {}), (SIZE, dict(scale=float("nan")), {}), (SIZE, {}, dict(k_scale=float("nan"))),
    (SIZE, {}, dict(v_scale=float("inf"))), (SIZE, dict(scale=3e38), dict(k_scale=10.0)),
    (SIZE, {}, dict(num_phys_pages=-1)), (SIZE, {}, dict(num_phys_pages=(1 << 31) // 64 + 1)),
    (SIZE, {}, dict(k_stride=(-64, 256, 128))), (SIZE, {}, dict(k_stride=(1 << 30, 1 << 25, 128))),
    (SIZE, {}, dict(k_stride=(1 << 30, 256, 1 << 30))), (SIZE, {}, dict(k_stride=(1 << 41, 256, 128))),
    (MISALIGNED, {}, dict(k_stride=(64 * 256, 256, 132))), (MISALIGNED, dict(row_stride=8 * 128 + 4), {}),
    (MISALIGNED, dict(q=0x1008), {}), (MISALIGNED, {}, dict(k=0x1008)),
    (NULL, dict(q=None), {}), (NULL, {}, dict(k=None)),
])
def test_queries_and_caches_are_checked_on_the_host(lib, call, code, q, c):
    assert call(lib, q=query(**q), c=cache(**c)) == code


def test_values_are_checked_where_a_call_reads_them(lib):
    for call in (decode, selected):
        assert call(lib, c=cache(v=None)) == NULL
        assert call(lib, c=cache(v=0x1004)) == MISALIGNED
        assert call(lib, c=cache(v_stride=(64, 256, 4))) == MISALIGNED
    assert weights(lib, c=cache(v=None, v_stride=(0, 0, 0))) not in (NULL, MISALIGNED, SIZE)


def test_windows_outputs_and_workspaces_are_checked_on_the_host(lib):
    assert decode(lib, n_seq=-1) == SIZE and decode(lib, pages=-1) == SIZE
    assert decode(lib, pages=(1 << 31) // 64) == SIZE
    assert decode(lib, n_seq=1 << 20, pages=1 << 20) == SIZE
    assert decode(lib, seq=None) == NULL and decode(lib, table=None) == NULL and decode(lib, out=None) == NULL
    assert decode(lib, out=P(0x1008)) == MISALIGNED and decode(lib, lse=P(0x1002)) == MISALIGNED
    need = mqa.mqa_kv_attention_decode_workspace_bytes(4, 8, 2, 128)
    assert need > 0 and decode(lib, ws_bytes=need - 1) == SIZE
    assert decode(lib, ws=None) == NULL and decode(lib, ws=P(0x1010)) == MISALIGNED
    assert selected(lib, K=-1) == SIZE and selected(lib, K=1 << 31) == SIZE
    assert selected(lib, slots=None) == NULL and selected(lib, count=None) == NULL
    need = mqa.mqa_kv_attention_selected_workspace_bytes(4, 512, 8, 2, 128)
    assert need > 0 and selected(lib, ws_bytes=need - 1) == SIZE and selected(lib, ws=None) == NULL
    assert mqa.mqa_kv_attention_selected_workspace_bytes(4096, 512, 8, 2, 128) == 0
    assert selected(lib, q=query(num_rows=4096), ws=None, ws_bytes=0) not in (NULL, SIZE)
    assert weights(lib, stride=319) == SIZE and weights(lib, lse=None) == NULL and weights(lib, acc=None) == NULL
    assert lib.mqa_kv_attention_decode(None, ctypes.byref(cache()), p, 1, 1, p, p, p, p, None, p, 1 << 40, None) == NULL


def test_workspace_sizes_refuse_bad_sizes(lib):
    for args in ((-1, 8, 2, 128), (4, 8, 3, 128), (4, 0, 1, 128), (1 << 24, 8, 2, 128)):
        with pytest.raises(mqa.MQAError):
            mqa.mqa_kv_attention_decode_workspace_bytes(*args)
    with pytest.raises(mqa.MQAError):
        mqa.mqa_kv_attention_selected_workspace_bytes(4, -1, 8, 2, 128)
    with pytest.raises(mqa.MQAError):
        mqa.mqa_kv_attention_decode_workspace_bytes(4, 8, 2, 80)
    with pytest.raises(mqa.MQAError):
        mqa.mqa_kv_evict_workspace_bytes(-1, 5)
    for args in ((1, (1 << 31) - 512), (1 << 22, 5), (1 << 14, 1 << 30)):
        with pytest.raises(mqa.MQAError):
            mqa.mqa_kv_evict_workspace_bytes(*args)


def test_workspaces_do_not_grow_with_the_capacity_for_ever():
    assert mqa.mqa_kv_evict_workspace_bytes(1000, 16384) == 0
    size = mqa.mqa_kv_evict_workspace_bytes(3, 1 << 21)
    assert size == mqa.mqa_kv_evict_workspace_bytes(3, (1 << 31) - 513) == 256 + 3 * 256 * 3 * 2048 * 4
    for K in range(6, 32):      # at most 512 parts of each head's sums, maximum and sum
        for rows in (1, 3, 100, 511, 512, 5000):
            size = mqa.mqa_kv_attention_selected_workspace_bytes(rows, (1 << K) - 1, 8, 2, 128)
            assert 0 <= size <= 512 * 4 * (128 + 2) * 4 + 512


def test_eviction_is_checked_on_the_host(lib):
    def select(acc=p, stride=1000, lens=p, n=3, max_len=1000, budget=100, recent=10, keep=p, kept=p, ws=p, ws_bytes=1 << 40):
        return lib.mqa_kv_evict_select(acc, stride, lens, n, max_len, budget, recent, keep, kept, None, ws, ws_bytes, None)
    for over in (dict(n=-1), dict(max_len=-1), dict(max_len=1001), dict(budget=-1), dict(recent=-1), dict(recent=101),
                 dict(budget=1 << 31), dict(max_len=1 << 31, stride=1 << 31)):
        assert select(**over) == SIZE, over
    assert select(acc=None) == NULL and select(lens=None) == NULL and select(keep=None) == NULL and select(kept=None) == NULL
    assert select(acc=P(0x1002)) == MISALIGNED

    def compact(n=2, budget=10, sp=3, P_src=5, dp=1, P_dst=5, arrays=None, count=1, keep=p, dst_table=p, **over):
        a = dict(src=0x1000, dst=0x1000, row_bytes=64, rows_per_position=2)
        strides = over.pop("stride", (64 * 128, 128, 64))
        a.update(over)
        x = Array(**a)
        x.src_stride[:] = strides
        x.dst_stride[:] = (64 * 128, 128, 64)
        return lib.mqa_kv_compact(keep, p, n, budget, p, sp, P_src, dst_table, dp, P_dst, ctypes.byref(x) if count else None,
                                  count, None)
    for over in (dict(n=-1), dict(budget=-1), dict(sp=-1), dict(dp=-1), dict(P_src=-1), dict(P_dst=1 << 26), dict(count=-1),
                 dict(count=9), dict(row_bytes=0), dict(rows_per_position=0), dict(row_bytes=1 << 25), dict(stride=(-4, 128, 64)),
                 dict(row_bytes=1 << 20, rows_per_position=17)):
        assert compact(**over) == SIZE, over
    for over in (dict(row_bytes=66), dict(stride=(8192, 130, 64)), dict(src=0x1002), dict(dst=0x1001)):
        assert compact(**over) == MISALIGNED, over
    assert compact(src=None) == NULL and compact(dst=None) == NULL and compact(keep=None) == NULL and compact(dst_table=None) == NULL


def good():
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)
    return dict(q=torch.zeros(4, 8, 128, dtype=torch.bfloat16), k_pages=torch.zeros(3, 64, 2, 128, dtype=torch.bfloat16),
                v_pages=torch.zeros(3, 64, 2, 128, dtype=torch.bfloat16), block_table=i(2, 3), seq_of_row=i(4), row_start=i(4),
                row_end=i(4), out=torch.zeros(4, 8, 128, dtype=torch.bfloat16), workspace=torch.zeros(8, dtype=torch.uint8),
                lse=torch.zeros(4, 8))


@pytest.mark.parametrize("exc,over", [
    (TypeError, dict(q=None)), (TypeError, dict(q=torch.zeros(4, 8, 128))), (ValueError, dict(q=torch.zeros(4, 1024, dtype=torch.bfloat16))),
    (ValueError, dict(q=torch.zeros(4, 128, 8, dtype=torch.bfloat16).transpose(1, 2))),
    (TypeError, dict(k_pages=torch.zeros(3, 64, 2, 128, dtype=torch.float16))),
    (ValueError, dict(k_pages=torch.zeros(3, 32, 2, 128, dtype=torch.bfloat16))),
    (ValueError, dict(k_pages=torch.zeros(3, 64, 3, 128, dtype=torch.bfloat16))),
    (ValueError, dict(v_pages=torch.zeros(4, 64, 2, 128, dtype=torch.bfloat16))),
    (ValueError, dict(v_pages=torch.zeros(3, 64, 2, 128, dtype=torch.float8_e4m3fn))),
    (ValueError, dict(k_pages=torch.zeros(3, 64, 128, 2, dtype=torch.bfloat16).transpose(2, 3))),
    (TypeError, dict(block_table=torch.zeros(2, 3))), (ValueError, dict(row_end=torch.zeros(3, dtype=torch.int32))),
    (TypeError, dict(out=torch.zeros(4, 8, 128, dtype=torch.float16))), (ValueError, dict(out=torch.zeros(4, 8, 64, dtype=torch.bfloat16))),
    (TypeError, dict(out=None)), (ValueError, dict(lse=torch.zeros(8, 4))), (TypeError, dict(lse=torch.zeros(4, 8).double())),
    (TypeError, dict(workspace=torch.zeros(8))),
])
def test_binding_rejects_malformed_attention_tensors(exc, over):
    a = good()
    a.update(over)
    with pytest.raises(exc):
        mqa.mqa_kv_attention_decode(**a)


def test_binding_rejects_malformed_lists_sums_and_arrays():
    a = good()
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)
    with pytest.raises(ValueError):
        mqa.mqa_kv_attention_selected(a["q"], a["k_pages"], a["v_pages"], i(3, 5), i(4), a["out"])
    with pytest.raises(TypeError):
        mqa.mqa_kv_attention_selected(a["q"], a["k_pages"], a["v_pages"], torch.zeros(4, 5), i(4), a["out"])
    w = lambda acc, lse=a["lse"]: mqa.mqa_kv_weights_accumulate(a["q"], lse, a["k_pages"], a["block_table"], a["seq_of_row"],
                                                                a["row_start"], a["row_end"], acc)
    for exc, acc in ((ValueError, torch.zeros(2, 191)), (ValueError, torch.zeros(3, 192)), (TypeError, torch.zeros(2, 192).double()),
                     (ValueError, torch.zeros(192, 2).t()), (ValueError, torch.zeros(192).expand(2, 192))):
        with pytest.raises(exc):
            w(acc)
    with pytest.raises(TypeError):
        w(torch.zeros(2, 192), lse=None)
    with pytest.raises(ValueError):
        mqa.mqa_kv_evict_select(torch.zeros(2, 9), i(2), 5, 1, i(2, 4), i(2))
    with pytest.raises(ValueError):
        mqa.mqa_kv_evict_select(torch.zeros(2, 9), i(2), 5, 1, i(2, 5), i(2), kept_acc=torch.zeros(2, 4))
    page = lambda *s, t=torch.float32: torch.zeros(*s, dtype=t)
    move = lambda *arrays: mqa.mqa_kv_compact(i(2, 5), i(2), i(2, 3), i(2, 1), arrays)
    for exc, pair in ((ValueError, (page(3, 32), page(3, 32))), (ValueError, (page(3, 64, 2), page(3, 64, 3))),
                      (ValueError, (page(3, 64), page(3, 64, t=torch.int32))), (TypeError, (page(3, 64), None)),
                      (ValueError, (page(3, 64, 5, 4).transpose(2, 3), page(3, 64, 4, 5))), (ValueError, (page(64), page(64)))):
        with pytest.raises(exc):
            move(pair)
    with pytest.raises(ValueError):
        move(*[(page(3, 64), page(3, 64))] * 9)
    with pytest.raises(ValueError):
        mqa.mqa_kv_compact(i(2, 5), i(3), i(2, 3), i(2, 1), [])
