"""Rows that one workgroup of norm, rotation and appending takes together lie within what its 32-bit offsets reach, whatever
row stride the host accepts (CPU; tests/kv_launches.py stands in for the runtime)."""
import pytest

import fp4_mqa_scoring_amd as mqa
from kv_launches import recorded

A = [(i + 1) << 58 for i in range(16)]     # addresses farther apart than any span


@pytest.fixture(scope="module")
def where(tmp_path_factory):
    from fp4_mqa_scoring_amd import build
    try:
        build.hipcc()
    except RuntimeError:
        pytest.skip("hipcc not found")
    return tmp_path_factory.mktemp("runtime")


TURN = (A[0] + (1 << 50), A[0] + (1 << 51), 64, 0, 0, 1e-6)


def rows(at, stride, out, out_stride, heads):
    return mqa._KV_ROWS.pack(at, stride, out, out_stride, 0, 0.0, heads)


def rotate(T, H, Hk, D, strides):
    q, q_out, k, k_out, _ = strides
    return ("mqa_kv_norm_rotate", [rows(A[1], q, A[2], q_out, H), rows(A[3], k, A[4], k_out, Hk) if Hk else None, mqa._KV_TURN.pack(*TURN), T, D, 0, None])


def append(T, H, Hkv, D, strides, fp4):
    q, q_out, k, _, v = strides
    new = (rows(A[3], k, 0, 0, Hkv) + rows(A[5], v, 0, 0, Hkv) + mqa._KV_NEW.pack(T, 0, A[6], 3, 7, A[7], A[8]) + mqa._KV_TURN.pack(*TURN))
    at = (64 * D * Hkv, D * Hkv, D)
    if fp4:
        codes, scales = [x // 2 for x in at], [x // 32 for x in at]
        cache = mqa._KV_CACHE_FP4.pack(*A[9:13], *codes, *codes, *scales, *scales, 10, Hkv, D)
    else:
        cache = mqa._KV_CACHE.pack(A[9], A[10], *at, *at, 10, Hkv, D, 0, 1.0, 1.0)
    return ("mqa_kv_append_fp4" if fp4 else "mqa_kv_append", [new, rows(A[1], q, A[2], q_out, H) if H else None, cache, None])


def test_rows_of_a_group_lie_within_32_bits(where):
    far = [1 << 32, (1 << 31) + 8, 1 << 30, 1 << 27, (1 << 26) + 8, 1 << 26]
    made = []
    for T in (512, 4096, 10_000, 1 << 20):
        for H, Hk, D in ((1, 1, 64), (4, 2, 128), (2, 1, 256)):
            for wide in far:
                for which in range(5):      # one of the tensors far apart, the others dense
                    strides = [H * D, H * D, Hk * D, Hk * D, Hk * D]
                    strides[which] = wide
                    if which < 4:
                        made.append((rotate(T, H, Hk, D, strides), wide, T))
                    if which != 3:
                        made += [(append(T, H, Hk, D, strides, fp4), wide, T) for fp4 in (False, True)]
    got = recorded([m[0] for m in made], where)
    for ((name, _), wide, T), (rc, launches) in zip(made, got):
        assert rc == 0 and len(launches) == 1, (name, rc)
        group, splits = launches[0]["more"]
        assert group * wide * 2 <= 1 << 31 or group == 1, (name, wide, group)
        assert launches[0]["grid"] == (T + group - 1) // group * splits


def test_dense_rows_keep_their_groups(where):
    made = [(rotate(8192, 40, 8, 128, [48 * 128, 40 * 128, 48 * 128, 8 * 128, 0]), 2), (rotate(8192, 1, 0, 64, [64] * 5), 16),
            (append(4096, 0, 8, 128, [0, 0, 24 * 128, 0, 24 * 128], True), 2), (append(4096, 0, 1, 128, [0, 0, 128, 0, 128], False), 16),
            (rotate(511, 1, 0, 64, [64] * 5), 1)]
    for (_, want), (rc, launches) in zip(made, recorded([m[0] for m in made], where)):
        assert rc == 0 and launches[0]["more"][0] == want
