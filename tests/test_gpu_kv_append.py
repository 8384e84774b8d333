"""Norm, rotation and appending to a paged cache, on the GPU, against the plain forms in 64 bits
(tests/kv_new_ref.py derives the bounds)."""
import numpy as np
import pytest
import torch

import fp4_mqa_scoring_amd as mqa
from kv_new_ref import (assert_e4m3, assert_fp4, assert_rounded, e4m3_of, fp4_numbers, fp4_of, fp4_values, turned)

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": torch.float8_e4m3fn}


def freqs(R, base=1e4):
    return (base ** (-torch.arange(0, R, 2, dtype=torch.float64) / R)).float()


def raw(t):
    return t.view(torch.uint8 if t.element_size() == 1 else torch.int16)


def fused(T, parts, D, kind, seed, pitch=1):
    """Slices of one projection's output on the device (a row of `pitch` heads more), and their host copies."""
    g = torch.Generator().manual_seed(seed)
    whole = torch.randn(T, sum(parts) + pitch, D, generator=g).to(kind)
    d = whole.to(DEV)
    at, host, dev = 0, [], []
    for n in parts:
        host.append(whole[:, at:at + n])
        dev.append(d[:, at:at + n])
        at += n
    return host, dev


def weights(D, kind, seed):
    g = torch.Generator().manual_seed(seed)
    return [(1 + 0.3 * torch.randn(D, generator=g)).to(kind) for _ in range(2)]


# T, H, Hk, D, type, norm, rotary dims, first of them, interleaved
TURNS = [
    (1, 32, 8, 128, "bf16", True, 128, 0, False), (3, 64, 1, 128, "bf16", False, 64, 64, True), (17, 4, 4, 64, "fp16", True, 64, 0, True),
    (65, 1, 1, 64, "bf16", True, 32, 0, False), (129, 2, 0, 256, "fp16", True, 256, 0, False), (700, 5, 1, 128, "bf16", True, 48, 80, False),
    (33, 7, 7, 256, "bf16", False, 16, 8, True), (2, 3, 2, 64, "bf16", True, 0, 0, False), (1025, 1, 0, 128, "fp16", False, 96, 0, False),
    (2100, 33, 3, 64, "bf16", True, 48, 16, True), (4, 200, 1, 256, "bf16", True, 128, 128, False), (600, 1, 0, 64, "fp16", True, 16, 48, False),
    (5000, 2, 1, 128, "bf16", True, 112, 16, False),
]


@pytest.mark.parametrize("T,H,Hk,D,kind,norm,R,at,pairs", TURNS)
@pytest.mark.parametrize("in_place", [False, True])
def test_norm_and_rotation_match_the_plain_form(T, H, Hk, D, kind, norm, R, at, pairs, in_place):
    kt = TYPES[kind]
    (hq, hk), (q, k) = fused(T, [H, Hk], D, kt, 7 * T + D)
    wq, wk = weights(D, kt, T)
    position = torch.from_numpy(np.random.RandomState(T).randint(0, 2_000_000, T).astype(np.int32))
    freq = freqs(R) if R else None
    q_out = q if in_place else torch.full((T, H, D), 7.0, dtype=kt, device=DEV)
    k_out = k if in_place else torch.full((T, Hk + 2, D), 7.0, dtype=kt, device=DEV)[:, 1:1 + Hk]
    more = dict(k=k, k_out=k_out) if Hk else {}
    if norm:
        more["q_weight"] = wq.to(DEV)
        if Hk:
            more["k_weight"] = wk.to(DEV)
    mqa.mqa_kv_norm_rotate(q, q_out, position.to(DEV), inv_freq=None if freq is None else freq.to(DEV), eps=1e-5,
                           weight_offset=0.25, rotary_offset=at, interleaved=pairs, **more)
    torch.cuda.synchronize()
    for x, got, w in ((hq, q_out, wq), (hk, k_out, wk)):
        y, tol = turned(x, w if norm else None, 0.25, 1e-5, position, freq, at, pairs)
        if got.numel():
            assert_rounded(got.cpu(), y, tol)
    if not in_place:
        whole = k_out._base if k_out._base is not None else k_out
        assert (whole[:, 0] == 7).all() and (whole[:, -1] == 7).all()        # beside the rows


def test_positions_of_any_size():
    """Angles of hundreds of millions of turns, and negative ones."""
    position = torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 16_777_217, 1_000_003], dtype=torch.int32)
    (x,), (q,) = fused(7, [3], 128, torch.float16, 3)
    out = torch.empty(7, 3, 128, dtype=torch.float16, device=DEV)
    mqa.mqa_kv_norm_rotate(q, out, position.to(DEV), inv_freq=freqs(128).to(DEV))
    assert_rounded(out.cpu(), *turned(x, position=position, freq=freqs(128)))


def test_no_rows_and_rows_of_zeros_and_extremes():
    empty = torch.empty(0, 4, 64, dtype=torch.bfloat16, device=DEV)
    mqa.mqa_kv_norm_rotate(empty, empty.clone(), torch.empty(0, dtype=torch.int32, device=DEV), inv_freq=freqs(64).to(DEV))
    x = torch.zeros(1, 6, 64, dtype=torch.bfloat16)
    x[0, 1] = 1e-30
    x[0, 2] = 3e17
    x[0, 3, 5] = float("nan")
    x[0, 4, 7] = float("inf")
    x[0, 5] = torch.linspace(-1, 1, 64).to(torch.bfloat16)
    w = torch.ones(64, dtype=torch.bfloat16)
    out = torch.empty_like(x, device=DEV)
    mqa.mqa_kv_norm_rotate(x.to(DEV), out, q_weight=w.to(DEV))
    y, tol = turned(x, w)
    assert torch.isnan(out[0, 3]).all()
    assert torch.isnan(out[0, 4, 7]) and (out[0, 4, :7] == 0).all()
    for h in (0, 1, 2, 5):      # what is in one head stays in it
        assert_rounded(out[0, h].cpu(), y[0, h], tol[0, h], h)
    # without a norm, numbers outside the rotated dims pass bit by bit, and a pair's infinity stays in the pair
    position = torch.tensor([5], dtype=torch.int32, device=DEV)
    mqa.mqa_kv_norm_rotate(x.to(DEV), out, position, inv_freq=freqs(32).to(DEV), rotary_offset=32)
    assert torch.equal(raw(out[0, 1:, :32]).cpu(), raw(x[0, 1:, :32]))
    mqa.mqa_kv_norm_rotate(x.to(DEV), out, position, inv_freq=freqs(32).to(DEV))
    odd = [i for i in range(64) if i not in (7, 23)]
    assert torch.isinf(out[0, 4, [7, 23]]).all() and (out[0, 4, odd] == 0).all()


# --- appending ------------------------------------------------------------------------------------


class Pool:
    """A pool of pages of every kind, its bytes set, with the tables of some sequences."""

    def __init__(self, lengths, Hkv, D, cache, seed=0, layout="nhd", spare=2, values=True):
        g = torch.Generator().manual_seed(seed)
        pages = [(n + 63) // 64 for n in lengths]
        self.P = sum(pages) + spare
        perm = torch.randperm(self.P, generator=g).int()
        self.table = torch.full((max(1, len(pages)), max(pages + [1]) + 1), -1, dtype=torch.int32)
        at = 0
        for i, n in enumerate(pages):
            self.table[i, :n] = perm[at:at + n]
            at += n
        self.cache, self.Hkv, self.D = cache, Hkv, D
        self.names = ["k", "v"] if values else ["k"]
        self.before, self.dev = {}, {}
        for name in self.names:
            parts = {"": D // 2, "_blocks": D // 32} if cache == "fp4" else {"": D * torch.empty(0, dtype=TYPES[cache]).element_size()}
            for part, width in parts.items():
                t = torch.randint(0, 120, (self.P, 64, Hkv, width), generator=g).to(torch.uint8)
                self.before[name + part] = t
                self.dev[name + part] = self._place(t.to(DEV), layout)

    def _place(self, t, layout):
        if layout == "nhd":
            return t
        if layout == "hnd":
            return t.transpose(1, 2).contiguous().transpose(1, 2)
        whole = torch.zeros((t.shape[0], 2, 64, t.shape[2] + 1, t.shape[3]), dtype=torch.uint8, device=DEV)
        view = whole[:, 1, :, 1:, :]
        view.copy_(t)
        return view

    def tensors(self):
        if self.cache == "fp4":
            return [self.dev.get(n) for n in ("k", "k_blocks", "v", "v_blocks")]
        return [None if n not in self.dev else self.dev[n].view(TYPES[self.cache]) for n in ("k", "v")]

    def append(self, k, v, seq, at, **more):
        call = mqa.mqa_kv_append_fp4 if self.cache == "fp4" else mqa.mqa_kv_append
        call(k, v, *self.tensors(), self.table.to(DEV), i32(seq), i32(at), **more)

    def check(self, rows, k, v, k_scale=1.0, v_scale=1.0, copied=False):
        """rows: (row of k and v, sequence, position) written; k: (y, tol) and v: the 16-bit rows. Everything else has its bytes."""
        torch.cuda.synchronize()
        r, seq, at = (torch.tensor(x, dtype=torch.long) for x in zip(*rows)) if rows else (torch.zeros(0, dtype=torch.long),) * 3
        where = (self.table[seq, at // 64].long(), at % 64)
        kind = None if self.cache == "fp4" else TYPES[self.cache]
        for name in self.names:
            got = {p: self.dev[name + p].cpu() for p in ("", "_blocks") if name + p in self.dev}
            for p, t in got.items():
                rest = t.clone()
                rest[where] = self.before[name + p][where]
                assert torch.equal(rest, self.before[name + p]), name + p
            if not rows:
                continue
            scale = k_scale if name == "k" else v_scale
            mine = got[""][where]
            if self.cache == "fp4":
                if name == "k":
                    assert_fp4(mine, got["_blocks"][where], k[0][r], k[1][r])
                else:
                    value, byte = fp4_of(v[r])
                    assert torch.equal(fp4_values(mine), value) and torch.equal(got["_blocks"][where], byte)
            elif self.cache == "e4m3":
                if name == "k":
                    assert_e4m3(mine.view(kind), k[0][r], k[1][r], scale)
                else:
                    assert torch.equal(mine, raw(e4m3_of(v[r], scale)))
            elif name == "k" and not copied:
                assert_rounded(mine.view(kind), k[0][r], k[1][r])
            else:
                assert torch.equal(mine, (k if name == "k" else v)[r].contiguous().view(torch.uint8))


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).to(DEV)


APPENDS = [
    # T, Hq, Hkv, D, type, cache, norm, rotary dims, first, interleaved, layout
    (1, 32, 8, 128, "bf16", "bf16", True, 128, 0, False, "nhd"), (40, 0, 2, 64, "fp16", "fp16", False, 64, 0, True, "pool"),
    (300, 5, 1, 256, "bf16", "bf16", True, 64, 192, False, "hnd"), (7, 0, 3, 128, "bf16", "bf16", False, 0, 0, False, "nhd"),
    (200, 0, 8, 128, "bf16", "e4m3", False, 128, 0, False, "nhd"), (65, 6, 3, 64, "fp16", "e4m3", True, 48, 16, False, "pool"),
    (33, 2, 1, 256, "fp16", "e4m3", True, 256, 0, True, "hnd"), (1, 0, 1, 64, "bf16", "e4m3", False, 0, 0, False, "nhd"),
    (200, 0, 8, 128, "bf16", "fp4", True, 128, 0, False, "nhd"), (77, 4, 1, 64, "fp16", "fp4", False, 32, 0, False, "pool"),
    (150, 16, 2, 256, "bf16", "fp4", True, 128, 128, True, "hnd"), (1, 64, 1, 128, "bf16", "fp4", False, 64, 64, True, "nhd"),
    (700, 0, 1, 128, "fp16", "fp4", False, 0, 0, False, "nhd"), (1500, 0, 1, 64, "bf16", "bf16", True, 64, 0, False, "nhd"),
]


@pytest.mark.parametrize("T,Hq,Hkv,D,kind,cache,norm,R,first,pairs,layout", APPENDS)
def test_append_matches_the_plain_form_and_leaves_the_rest_alone(T, Hq, Hkv, D, kind, cache, norm, R, first, pairs, layout):
    kt = TYPES[kind]
    lengths = [T // 2 + 1, T + 3, 700, 64]
    p = Pool(lengths, Hkv, D, cache, seed=T + D, layout=layout)
    rng = np.random.RandomState(T)
    slots = [(s, i) for s, n in enumerate(lengths) for i in range(n)]
    chosen = [slots[i] for i in rng.permutation(len(slots))[:T]]
    (hq, hk, hv), (q, k, v) = fused(T, [Hq, Hkv, Hkv], D, kt, T)
    wq, wk = weights(D, kt, T)
    far = torch.from_numpy(rng.randint(0, 500_000, T).astype(np.int32))
    freq = freqs(R, 1e6) if R else None
    scales = dict(k_scale=0.03, v_scale=0.0625) if cache == "e4m3" else {}
    more = dict(scales, inv_freq=None if freq is None else freq.to(DEV), rotary_offset=first, interleaved=pairs,
                rotary_position=far.to(DEV) if R else None)
    if norm:
        more["k_weight"] = wk.to(DEV)
    q_out = torch.empty(T, Hq, D, dtype=kt, device=DEV)
    if Hq:
        more.update(q=q, q_out=q_out, q_weight=wq.to(DEV) if norm else None)
    seq, at = zip(*chosen)
    p.append(k, v, seq, at, **more)
    turn = dict(position=far, freq=freq, at=first, interleaved=pairs)
    copied = not norm and not R
    p.check([(r, s, i) for r, (s, i) in enumerate(chosen)], hk if copied and cache not in ("e4m3", "fp4") else turned(hk, wk if norm else None, **turn),
            hv, copied=copied, **scales)
    if Hq:
        assert_rounded(q_out.cpu(), *turned(hq, wq if norm else None, **turn))


@pytest.mark.parametrize("cache", ["bf16", "e4m3", "fp4"])
def test_rows_that_are_padding_or_fail_write_nothing(cache):
    p = Pool([100, 70], 2, 64, cache, seed=1)
    p.table[1, 1] = p.P                                   # outside the pool
    rows = [(0, 0), (0, -1), (5, -1), (0, 99), (2, 3), (-1, 3), (0, -2), (0, 64 * p.table.shape[1]), (1, 64), (1, 63),
            (0, 2 ** 31 - 1), (0, 64 * p.table.shape[1] - 1)]
    (hq, hk, hv), (q, k, v) = fused(len(rows), [3, 2, 2], 64, torch.bfloat16, 5)
    seq, at = zip(*rows)
    q_out = torch.empty(len(rows), 3, 64, dtype=torch.bfloat16, device=DEV)
    freq = freqs(64)
    mqa.mqa_fp4_status()
    p.append(k, v, seq, at, inv_freq=freq.to(DEV), q=q, q_out=q_out)
    position = torch.tensor(at, dtype=torch.int32)
    p.check([(r, *rows[r]) for r in (0, 3, 9)], turned(hk, position=position, freq=freq), hv)
    assert mqa.mqa_fp4_status() == mqa.STATUS_BAD_WINDOW | mqa.STATUS_BAD_PAGE
    assert_rounded(q_out.cpu(), *turned(hq, position=position, freq=freq))      # queries of every row
    p.append(k[1:3], v[1:3], seq[1:3], at[1:3])
    torch.cuda.synchronize()
    assert mqa.mqa_fp4_status() == 0
    p.append(k[:0], v[:0], [], [])


@pytest.mark.parametrize("cache", ["fp16", "fp4"])
def test_keys_only_and_no_pages(cache):
    p = Pool([90], 1, 128, cache, seed=2, values=False)
    (hk,), (k,) = fused(90, [1], 128, torch.float16, 6)
    args = [x for x in p.tensors()]
    call = mqa.mqa_kv_append_fp4 if cache == "fp4" else mqa.mqa_kv_append
    at = np.arange(90)[::-1].copy()
    if cache == "fp4":
        call(k, None, args[0], args[1], None, None, p.table.to(DEV), i32(np.zeros(90)), i32(at))
    else:
        call(k, None, args[0], None, p.table.to(DEV), i32(np.zeros(90)), i32(at))
    copied = cache != "fp4"
    p.check([(r, 0, int(at[r])) for r in range(90)], hk if copied else (hk.double(), torch.zeros(90, 1, 128, dtype=torch.float64)), None,
            copied=copied)
    mqa.mqa_fp4_status()
    none = [None if t is None else t[:0] for t in args]
    if cache == "fp4":
        call(k, None, none[0], none[1], None, None, p.table.to(DEV), i32(np.zeros(90)), i32(at))
    else:
        call(k, None, none[0], None, p.table.to(DEV), i32(np.zeros(90)), i32(at))
    assert mqa.mqa_fp4_status() == mqa.STATUS_BAD_PAGE


def test_bits_of_values_and_unturned_keys_are_kept():
    """Infinities, every NaN and -0 included."""
    bits = torch.arange(65536).to(torch.int32).sub(32768).to(torch.int16).reshape(512, 1, 128)
    x = bits.view(torch.bfloat16)
    p = Pool([512], 1, 128, "bf16", seed=3)
    p.append(x.to(DEV), x.to(DEV), np.zeros(512), np.arange(512))
    torch.cuda.synchronize()
    at = torch.arange(512)
    for name in ("k", "v"):
        got = p.dev[name].view(torch.bfloat16).cpu().view(torch.int16)[p.table[0].long()[at // 64], at % 64]
        assert torch.equal(got, bits)


def test_8_bits_saturate_and_round_to_even():
    every = torch.arange(65536).to(torch.int32).sub(32768).to(torch.int16).reshape(512, 1, 128).view(torch.float16)
    p = Pool([512], 1, 128, "e4m3", seed=4)
    p.append(every.to(DEV), every.to(DEV), np.zeros(512), np.arange(512), k_scale=0.37, v_scale=1.0)
    torch.cuda.synchronize()
    at = torch.arange(512)
    for name, scale in (("k", 0.37), ("v", 1.0)):
        got = p.dev[name].cpu()[p.table[0].long()[at // 64], at % 64].view(torch.float8_e4m3fn)
        want = e4m3_of(every, scale)
        nan = torch.isnan(want.float())
        assert torch.equal(torch.isnan(got.float()), nan)
        assert torch.equal(raw(got)[~nan], raw(want)[~nan])


def test_4_bits_are_the_indexer_s_own():
    """Keys of one head of 128 dims, as mqa_fp4_cache_write writes them from 32 bits: every magnitude that bf16 has,
    ties, zeros, infinities and NaN among them."""
    g = torch.Generator().manual_seed(9)
    n = 640
    x = (torch.randn(n, 128, generator=g) * torch.exp2(torch.randint(-126, 126, (n, 1), generator=g).float())).to(torch.bfloat16)
    x[0] = 0.0
    x[1, :32] = -0.0
    x[2, 5] = float("nan")
    x[3, 40] = float("inf")
    x[4] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 4.0] * 16)
    x[5] = 1e-39
    x[6] = 3.3e38
    p = Pool([n], 1, 128, "fp4", seed=5, values=False)
    mqa.mqa_kv_append_fp4(x.to(DEV)[:, None], None, p.dev["k"], p.dev["k_blocks"], None, None, p.table.to(DEV), i32(np.zeros(n)),
                          i32(np.arange(n)))
    codes, scales = torch.zeros(p.P, 64, 64, dtype=torch.uint8, device=DEV), torch.zeros(p.P, 64, 4, dtype=torch.uint8, device=DEV)
    mqa.mqa_fp4_cache_write(x.float().to(DEV), i32(np.arange(n)), p.table[0].contiguous().to(DEV), codes, scales)
    torch.cuda.synchronize()
    at = torch.arange(n)
    where = (p.table[0].long()[at // 64], at % 64)
    assert torch.equal(p.dev["k_blocks"].cpu()[where][:, 0], scales.cpu()[where])
    assert torch.equal(p.dev["k"].cpu()[where][:, 0], codes.cpu()[where])
    value, byte = fp4_of(x)
    assert torch.equal(scales.cpu()[where], byte) and torch.equal(fp4_values(codes.cpu()[where]), value)


def test_offsets_beyond_32_bits():
    """A pool of 6 GiB whose used pages lie at both ends."""
    P = 6 * 2 ** 30 // (64 * 8 * 128 * 2)
    k = torch.zeros(P, 64, 8, 128, dtype=torch.bfloat16, device=DEV)
    v = torch.zeros_like(k)
    table = i32([[0, P - 1, P // 2 + 1]])
    (hk, hv), (dk, dv) = fused(130, [8, 8], 128, torch.bfloat16, 8)
    mqa.mqa_kv_append(dk, dv, k, v, table, i32(np.zeros(130)), i32(np.arange(130)))
    for t, want in ((k, hk), (v, hv)):
        got = t[[0, P - 1, P // 2 + 1]].reshape(192, 8, 128).cpu()
        assert torch.equal(raw(got[:130]), raw(want.contiguous())) and (got[130:] == 0).all()
        assert int((t.view(torch.int16) != 0).sum()) == int((raw(want.contiguous()) != 0).sum())


def test_streams_and_graphs():
    T, H, Hkv, D = 64, 16, 4, 128
    p = Pool([600] * T, Hkv, D, "bf16", seed=10)
    (hq, hk, hv), (q, k, v) = fused(T, [H, Hkv, Hkv], D, torch.bfloat16, 11)
    wq, wk = (w.to(DEV) for w in weights(D, torch.bfloat16, 12))
    freq = freqs(D)
    at, seq, table = i32(np.arange(T) * 9), i32(np.arange(T)), p.table.to(DEV)
    q_out, alone = torch.empty(T, H, D, dtype=torch.bfloat16, device=DEV), torch.empty(T, H, D, dtype=torch.bfloat16, device=DEV)

    def step(out, stream=None):
        mqa.mqa_kv_append(k, v, *p.tensors(), table, seq, at, inv_freq=freq.to(DEV) if stream else d_freq, k_weight=wk, q=q, q_out=out,
                          q_weight=wq, stream=stream)

    d_freq = freq.to(DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    mqa.mqa_kv_norm_rotate(q, alone, at, inv_freq=d_freq, q_weight=wq, stream=side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(q_out)
    for i in range(3):
        at.copy_(i32(np.arange(T) * 9 - i))                 # row 0 becomes padding, then fails
        q_out.fill_(3.0)
        mqa.mqa_fp4_status()
        graph.replay()
        torch.cuda.synchronize()
        assert mqa.mqa_fp4_status() == (mqa.STATUS_BAD_WINDOW if i == 2 else 0)
        position = at.cpu()
        want = turned(hq, wq.cpu(), position=position, freq=freq)
        assert_rounded(q_out.cpu(), *want)
        if i == 0:
            assert torch.equal(raw(q_out), raw(alone))
        y, tol = turned(hk, wk.cpu(), position=position, freq=freq)
        got = p.dev["k"].view(torch.bfloat16).cpu()
        live = torch.arange(T)[position >= 0]
        where = (p.table[live, position[live].long() // 64].long(), position[live].long() % 64)
        assert_rounded(got[where], y[live], tol[live])
        assert torch.equal(raw(p.dev["v"].view(torch.bfloat16).cpu()[where]), raw(hv[live].contiguous()))


def test_fp4_reference_agrees_with_itself():
    g = torch.Generator().manual_seed(1)
    x = torch.randn(50, 64, generator=g)
    value, byte = fp4_of(x)
    code = (torch.searchsorted(torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64), value.abs())
            + 8 * torch.signbit(value)).to(torch.uint8)
    packed = code[:, 0::2] | (code[:, 1::2] << 4)
    assert torch.equal(fp4_values(packed), value)
    assert ((fp4_numbers(packed, byte) - x.double()).abs() <= x.abs().double() / 2 + 2.0 ** (byte.double() - 129).repeat_interleave(32, 1)).all()
