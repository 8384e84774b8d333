"""The key-value cache operators' launches at the largest sizes that their hosts accept: all rows are in them, and no
launch has as many threads as 32 bits count (CPU; tests/kv_launches.py stands in for the runtime)."""
import pytest

import fp4_mqa_scoring_amd as mqa
from kv_launches import recorded

MOST = (1 << 24) - 256      # rows times heads
A = [(i + 1) << 44 for i in range(16)]     # addresses far apart


@pytest.fixture(scope="module")
def where(tmp_path_factory):
    from fp4_mqa_scoring_amd import build
    try:
        build.hipcc()
    except RuntimeError:
        pytest.skip("hipcc not found")
    return tmp_path_factory.mktemp("runtime")


def query(rows, H, D, kind=0):
    return mqa._KV_QUERY.pack(A[0], H * D, rows, H, kind, 0.1)


def fp4_cache(Hkv, D):
    codes, scales = (32 * D * Hkv, D // 2 * Hkv, D // 2), (2 * D * Hkv, D // 32 * Hkv, D // 32)
    return mqa._KV_CACHE_FP4.pack(*A[1:5], *codes, *codes, *scales, *scales, 10, Hkv, D)


def cache(Hkv, D, kind=0):
    strides = (64 * D * Hkv, D * Hkv, D)
    return mqa._KV_CACHE.pack(A[1], A[2], *strides, *strides, 10, Hkv, D, kind, 1.0, 1.0)


def selected(rows, H, Hkv, D, K, fp4):
    size = 1 << 43
    return ("mqa_kv_attention_selected_fp4" if fp4 else "mqa_kv_attention_selected",
            [query(rows, H, D), fp4_cache(Hkv, D) if fp4 else cache(Hkv, D), A[5], A[6], K, A[7], A[8], A[9], size, None])


def decode(rows, H, Hkv, D, fp4):
    return ("mqa_kv_attention_decode_fp4" if fp4 else "mqa_kv_attention_decode",
            [query(rows, H, D), fp4_cache(Hkv, D) if fp4 else cache(Hkv, D), A[5], 3, 7, A[6], A[7], A[8], A[9], A[10], A[11], 1 << 43, None])


SHAPES = [(1, 1, 64), (1, 1, 128), (1, 1, 256), (3, 3, 64), (3, 3, 128), (2, 2, 64), (2, 2, 128), (8, 2, 128), (5, 1, 128), (17, 1, 128), (64, 1, 128),
          (70, 1, 256)]


@pytest.mark.parametrize("fp4", [True, False])
@pytest.mark.parametrize("H,Hkv,D", SHAPES)
def test_lists_of_as_many_rows_as_the_host_accepts(where, H, Hkv, D, fp4):
    rows = MOST // H
    some = [1, 1000, 8388480 // H, 8388608 // H, (8388608 + 513) // H, rows]
    for n, (rc, launches) in zip(some, recorded([selected(n, H, Hkv, D, 1, fp4) for n in some], where)):
        assert rc == 0, (n, rc)
        at = 0
        for x in launches:      # each takes the rows behind the ones before it
            assert "kv_selected" in x["kernel"] and x["grid"] * x["block"] < 1 << 32
            address, stride, count = x["q"]
            assert address == A[0] + at * 2 * H * D and count > 0
            at += count
        assert at == n


@pytest.mark.parametrize("fp4", [True, False])
@pytest.mark.parametrize("H,Hkv,D", SHAPES)
def test_windows_of_as_many_rows_as_the_host_accepts(where, H, Hkv, D, fp4):
    (rc, launches), = recorded([decode(MOST // H, H, Hkv, D, fp4)], where)
    assert rc == 0 and launches and all(x["grid"] * x["block"] < 1 << 32 for x in launches)


@pytest.mark.parametrize("fp4", [True, False])
def test_split_lists_go_in_one_launch_and_a_joining(where, fp4):
    (rc, launches), = recorded([selected(3, 8, 2, 128, 4096, fp4)], where)
    assert rc == 0 and [("join" in x["kernel"]) for x in launches] == [False, True]
