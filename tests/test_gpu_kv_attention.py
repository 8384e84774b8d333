"""Attention over the paged key-value cache and over selected slots, on the GPU,
against the plain form in 64 bits (tests/kv_ref.py derives the bounds)."""
import numpy as np
import pytest
import torch

import fp4_mqa_scoring_amd as mqa
from kv_ref import Row, assert_row

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": torch.float8_e4m3fn}
DEV = "cuda:0"


def numbers(t, scale):
    """What a cache tensor's elements stand for, in 64 bits on the host."""
    return t.cpu().float().double() * scale


class Case:
    """Sequences of the given lengths over a shuffled pool whose unused positions,
    and pages, hold NaN."""

    def __init__(self, lengths, H, Hkv, D, qtype="bf16", cache=None, seed=0, spread=2.0, layout="nhd",
                 k_scale=None, spare=2, capacity=0):
        g = torch.Generator().manual_seed(seed)
        self.H, self.Hkv, self.D = H, Hkv, D
        self.qt, self.ct = TYPES[qtype], TYPES[cache or qtype]
        self.e4m3 = self.ct == torch.float8_e4m3fn
        self.k_scale, self.v_scale = (0.25, 0.5) if self.e4m3 else (1.0, 1.0)
        if k_scale is not None:
            self.k_scale = k_scale
        self.lengths = list(lengths)
        pages = [(n + 63) // 64 for n in lengths]
        self.P = sum(pages) + spare
        perm = torch.randperm(self.P, generator=g).int()
        width = max(max(pages, default=0), capacity, 1)
        self.table = torch.full((max(1, len(pages)), width), -1, dtype=torch.int32)
        at = 0
        for i, n in enumerate(pages):
            self.table[i, :n] = perm[at:at + n]
            at += n
        shape = (self.P, 64, Hkv, D)
        k = (torch.randn(shape, generator=g) / (0.25 if self.e4m3 else 1.0)).to(self.ct)
        v = (torch.randn(shape, generator=g) / (0.5 if self.e4m3 else 1.0)).to(self.ct)
        used = torch.zeros(self.P, 64, dtype=torch.bool)
        for i, n in enumerate(self.lengths):
            for p in range(pages[i]):
                used[self.table[i, p], : min(64, n - 64 * p)] = True
        junk = 0x7F if self.e4m3 else 0x7FFF
        raw = torch.uint8 if self.e4m3 else torch.int16
        k.view(raw)[~used] = junk
        v.view(raw)[~used] = junk
        self.k, self.v = k, v
        self.spread = spread
        self.g = g
        self.dk, self.dv = (self._place(t, layout) for t in (k, v))

    def _place(self, t, layout):
        d = t.to(DEV)
        if layout == "nhd":
            return d
        if layout == "hnd":      # [P, Hkv, 64, D] memory
            return d.view(torch.uint8).view(*t.shape[:3], -1).transpose(1, 2).contiguous().transpose(1, 2).view(t.dtype)
        raw = torch.zeros((t.shape[0], 2, 64, t.shape[2] + 1, t.shape[3] * t.element_size()), dtype=torch.uint8, device=DEV)
        view = raw[:, 1, :, 1:, :]   # one half of a pool, one head short of its pitch
        view.copy_(d.view(torch.uint8))
        return view.view(t.dtype)

    def queries(self, n):
        return (torch.randn(n, self.H, self.D, generator=self.g) * self.spread).to(self.qt)

    def at(self, seq, lo, hi):
        pos = torch.arange(lo, hi)
        page = self.table[seq].long()[pos // 64]
        raw = torch.uint8 if self.e4m3 else torch.int16
        take = lambda t, s: numbers(t.view(raw)[page, pos % 64].view(t.dtype), s)
        return take(self.k, self.k_scale), take(self.v, self.v_scale)

    def by_slot(self, slots):
        raw = torch.uint8 if self.e4m3 else torch.int16
        s = torch.as_tensor(slots).long()
        take = lambda t, c: numbers(t.view(raw)[s // 64, s % 64].view(t.dtype), c)
        return take(self.k, self.k_scale), take(self.v, self.v_scale)


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).to(DEV)


def run_decode(c, q, seq, start, end, lse=True, scale=None, stream=None, workspace=None, dq=None):
    dq = q.to(DEV) if dq is None else dq
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device=DEV)
    got_lse = torch.full(q.shape[:2], 7.0, device=DEV) if lse else None
    if workspace is None:
        workspace = torch.full((mqa.mqa_kv_attention_decode_workspace_bytes(q.shape[0], c.H, c.Hkv, c.D),), 0xFF,
                               dtype=torch.uint8, device=DEV)   # NaN, if any of it counted
    mqa.mqa_kv_attention_decode(dq, c.dk, c.dv, c.table.to(DEV), i32(seq), i32(start), i32(end), out, workspace,
                                lse=got_lse, scale=scale, k_scale=c.k_scale, v_scale=c.v_scale, stream=stream)
    torch.cuda.synchronize()
    return out.cpu(), got_lse.cpu() if lse else None


def check_decode(c, q, seq, start, end, out, lse, scale=None):
    scale = c.D ** -0.5 if scale is None else scale
    for r in range(q.shape[0]):
        k, v = c.at(int(seq[r]), int(start[r]), int(end[r]))
        assert_row(out[r], None if lse is None else lse[r], Row(q[r], k, v, scale, c.qt), f"row {r}")


SHAPES = [
    # H, Hkv, D, q type, cache
    (8, 2, 128, "bf16", "bf16"), (16, 1, 128, "fp16", "fp16"), (64, 1, 128, "bf16", "bf16"), (5, 5, 64, "fp16", "fp16"),
    (40, 2, 64, "bf16", "bf16"), (128, 1, 64, "fp16", "fp16"), (3, 1, 256, "bf16", "bf16"), (48, 2, 256, "fp16", "fp16"),
    (14, 2, 128, "bf16", "e4m3"), (65, 1, 128, "fp16", "e4m3"), (8, 8, 64, "bf16", "e4m3"), (33, 1, 64, "fp16", "e4m3"),
    (4, 2, 256, "fp16", "e4m3"), (70, 2, 256, "bf16", "e4m3"), (17, 1, 128, "fp16", "fp16"), (70, 1, 128, "bf16", "bf16"),
]


@pytest.mark.parametrize("H,Hkv,D,qtype,cache", SHAPES)
def test_decode_matches_the_plain_form(H, Hkv, D, qtype, cache):
    lengths = [1, 0, 31, 32, 33, 63, 64, 65, 127, 129, 200, 1000, 2777]
    c = Case(lengths, H, Hkv, D, qtype, cache, seed=H * 1000 + D)
    q = c.queries(len(lengths))
    seq = list(range(len(lengths)))
    out, lse = run_decode(c, q, seq, [0] * len(lengths), lengths)
    check_decode(c, q, seq, [0] * len(lengths), lengths, out, lse)


@pytest.mark.parametrize("layout", ["hnd", "pool"])
@pytest.mark.parametrize("cache,D,H,Hkv", [("bf16", 128, 12, 3), ("e4m3", 64, 12, 3), ("bf16", 256, 34, 1)])
def test_decode_windows_rows_and_strides(layout, cache, D, H, Hkv):
    """Windows that start and end anywhere, several rows per sequence in no order,
    a query tensor with a row pitch, other cache layouts, no lse."""
    c = Case([700, 1400, 64, 333], H, Hkv, D, "bf16", cache, seed=5, layout=layout, capacity=100)
    wins = [(0, 0, 700), (1, 1337, 1400), (3, 100, 101), (1, 31, 33), (0, 699, 700), (2, 0, 64), (2, 64, 64),
            (1, 0, 0), (3, 33, 290), (0, 63, 65), (1, 640, 1281), (2, 5, 5)]
    seq, start, end = zip(*wins)
    q = c.queries(len(wins))
    wide = torch.zeros(len(wins), H + 4, D, dtype=c.qt, device=DEV)
    wide[:, 2:2 + H] = q.to(DEV)
    out, lse = run_decode(c, q, seq, start, end, lse=False, dq=wide[:, 2:2 + H])
    assert lse is None
    check_decode(c, q, seq, start, end, out, None)


@pytest.mark.parametrize("scale", [-0.3, 0.0, 3.0])
def test_decode_scales(scale):
    """A negative scale, a scale of 0 (plain mean), and a steep one."""
    c = Case([500, 70], 6, 2, 128, "bf16", seed=8, spread=1.0)
    q = c.queries(2)
    out, lse = run_decode(c, q, [0, 1], [0, 3], [500, 70], scale=scale)
    check_decode(c, q, [0, 1], [0, 3], [500, 70], out, lse, scale=scale)


@pytest.mark.parametrize("H,Hkv", [(8, 2), (64, 1)])
def test_decode_scores_that_rise_and_fall_over_the_window(H, Hkv):
    """The running maximum changes in every tile, or never after the first."""
    c = Case([1500, 1500], H, Hkv, 64, "fp16", seed=11, spread=1.0)
    ramp = torch.linspace(-6, 6, 1500)
    for s, sign in ((0, 1.0), (1, -1.0)):
        for p in range(1500):
            c.k[c.table[s, p // 64], p % 64] = (sign * ramp[p]).to(c.ct)
    c.dk = c.k.to(DEV)
    q = (torch.rand(2, H, 64, generator=c.g) * 0.6 + 0.2).to(c.qt)
    out, lse = run_decode(c, q, [0, 1], [0, 0], [1500, 1500])
    check_decode(c, q, [0, 1], [0, 0], [1500, 1500], out, lse)


def test_decode_more_rows_than_one_workgroup_plans():
    lengths = [int(x) for x in np.random.RandomState(3).randint(0, 150, 40)]
    c = Case(lengths, 4, 2, 64, "bf16", seed=13)
    rows = 1500
    rng = np.random.RandomState(4)
    seq = rng.randint(0, 40, rows)
    end = np.array([rng.randint(0, lengths[s] + 1) for s in seq])
    start = np.array([rng.randint(0, e + 1) for e in end])
    q = c.queries(rows)
    out, lse = run_decode(c, q, seq, start, end)
    check_decode(c, q, seq, start, end, out, lse)


@pytest.mark.parametrize("rows", [1, 1023, 1024, 1025])
def test_decode_row_counts_around_the_plan(rows):
    c = Case([40, 90], 2, 1, 64, "bf16", seed=17)
    seq = np.arange(rows) % 2
    end = np.where(seq == 0, 40, 90)
    start = np.minimum(np.arange(rows) % 50, end)
    q = c.queries(rows)
    out, lse = run_decode(c, q, seq, start, end)
    check_decode(c, q, seq, start, end, out, lse)


@pytest.mark.parametrize("H,Hkv,D", [(8, 2, 128), (64, 1, 128), (4, 1, 256)])
def test_decode_one_long_sequence_is_split_and_joined(H, Hkv, D):
    c = Case([40000], H, Hkv, D, "bf16", seed=19)
    q = c.queries(1)
    out, lse = run_decode(c, q, [0], [0], [40000])
    check_decode(c, q, [0], [0], [40000], out, lse)


def test_decode_rows_that_fail_closed_leave_the_others_alone():
    c = Case([300, 200, 100], 8, 2, 128, "bf16", seed=23)
    c.table[1, 2] = c.P            # outside the pool
    c.table[2, 0] = -1
    rows = [(0, 0, 300), (3, 0, 10), (-1, 0, 10), (0, -1, 10), (0, 20, 10), (0, 0, 64 * c.table.shape[1] + 1),
            (1, 0, 200), (1, 0, 128), (2, 0, 100), (2, 64, 100), (2, 64, 64), (0, 0, 0)]
    seq, start, end = zip(*rows)
    q = c.queries(len(rows))
    mqa.mqa_fp4_status()
    out, lse = run_decode(c, q, seq, start, end)
    assert mqa.mqa_fp4_status() == mqa.STATUS_BAD_WINDOW | mqa.STATUS_BAD_PAGE
    good = [0, 7, 9, 10, 11]
    for r in range(len(rows)):
        if r in good:
            k, v = c.at(*rows[r])
            assert_row(out[r], lse[r], Row(q[r], k, v, c.D ** -0.5, c.qt), f"row {r}")
        else:
            assert torch.isnan(out[r]).all() and torch.isnan(lse[r]).all(), r
    run_decode(c, q[:1], [0], [0], [300])
    assert mqa.mqa_fp4_status() == 0


def test_decode_nan_and_infinities_inside_the_window():
    """IEEE rules inside the window: a NaN key makes the row NaN, an infinite value an
    infinite dim; a key that scores -infinity drops out."""
    c = Case([100, 100, 100], 2, 1, 64, "bf16", seed=29)
    c.k[c.table[0, 1], 3] = float("nan")
    c.v[c.table[1, 0], 5, 0, 7] = float("inf")
    q = c.queries(3)
    q[2] = q[2].abs() + 0.1
    c.k[c.table[2, 0], 9] = float("-inf")
    c.dk, c.dv = c.k.to(DEV), c.v.to(DEV)
    out, lse = run_decode(c, q, [0, 1, 2], [0, 0, 0], [100, 100, 100])
    assert torch.isnan(out[0]).all() and torch.isnan(lse[0]).all()
    assert torch.isinf(out[1, :, 7]).all() and (out[1, :, 7] > 0).all()
    assert torch.isfinite(out[1, :, :7]).all() and torch.isfinite(out[1, :, 8:]).all()
    k, v = c.at(2, 0, 100)
    keep = torch.arange(100) != 9
    assert_row(out[2], lse[2], Row(q[2], k[keep], v[keep], 64 ** -0.5, c.qt), "row 2")
    out, lse = run_decode(c, q[2:], [2], [9], [10])     # nothing but -infinity
    assert torch.isnan(out).all() and (lse == float("-inf")).all()


@pytest.mark.parametrize("H,Hkv", [(8, 2), (64, 1)])
def test_parts_whose_scores_are_all_minus_infinity_drop_out(H, Hkv):
    """Of a sequence that many workgroups share, the first and the last of them meet nothing but -infinity."""
    n, lo, hi = 20000, 9001, 10002
    c = Case([n], H, Hkv, 64, "bf16", seed=30)
    q = c.queries(1).abs() + 0.1
    pos = torch.arange(n)
    out_of = pos[(pos < lo) | (pos >= hi)]
    c.k[c.table[0].long()[out_of // 64], out_of % 64] = float("-inf")
    c.dk = c.k.to(DEV)
    want = Row(q[0], *c.at(0, lo, hi), 64 ** -0.5, c.qt)
    out, lse = run_decode(c, q, [0], [0], [n])
    assert_row(out[0], lse[0], want)
    slots = (c.table[0].long()[pos // 64] * 64 + pos % 64)[None].numpy()
    out, lse = run_selected(c, q, slots, [n])
    assert_row(out[0], lse[0], want)


def test_batches_without_rows_sequences_or_pages():
    c = Case([70], 4, 2, 64, "bf16", seed=33)
    q = c.queries(0)
    assert run_decode(c, q, [], [], [])[0].shape == (0, 4, 64)
    assert run_selected(c, q, np.zeros((0, 5), np.int64), [])[0].shape == (0, 4, 64)
    mqa.mqa_fp4_status()
    q = c.queries(3)
    c.dk, c.dv = c.dk[:0], c.dv[:0]                 # no pages: empty windows and lists only
    out, lse = run_decode(c, q, [0, 0, 0], [0, 5, 0], [0, 5, 1])
    assert mqa.mqa_fp4_status() == mqa.STATUS_BAD_PAGE
    assert (out[:2] == 0).all() and (lse[:2] == float("-inf")).all() and torch.isnan(out[2]).all()
    out, lse = run_selected(c, q, np.zeros((3, 2), np.int64), [0, 0, 1])
    assert mqa.mqa_fp4_status() == mqa.STATUS_BAD_PAGE
    assert (out[:2] == 0).all() and (lse[:2] == float("-inf")).all() and torch.isnan(out[2]).all()
    c.table = c.table[:0]                           # no sequences
    out, lse = run_decode(c, q, [0, 0, -1], [0, 0, 0], [0, 0, 0])
    assert mqa.mqa_fp4_status() == mqa.STATUS_BAD_WINDOW
    assert torch.isnan(out).all() and torch.isnan(lse).all()


def test_decode_offsets_beyond_32_bits():
    """A pool of 6 GiB whose used pages lie at both ends."""
    P = 6 * 2 ** 30 // (64 * 128 * 2)
    k = torch.empty(P, 64, 1, 128, dtype=torch.bfloat16, device=DEV)
    v = torch.empty_like(k)
    c = Case([200], 16, 1, 128, "bf16", seed=31, spare=0)
    places = [0, P - 1, P // 2 + 1, P - 2]
    for i in range(4):
        page = int(c.table[0, i])
        k[places[i]] = c.k[page].to(DEV)
        v[places[i]] = c.v[page].to(DEV)
    q = c.queries(1)
    want_k, want_v = c.at(0, 0, 200)
    table = i32([places])
    out = torch.empty(1, 16, 128, dtype=torch.bfloat16, device=DEV)
    lse = torch.empty(1, 16, device=DEV)
    ws = torch.empty(mqa.mqa_kv_attention_decode_workspace_bytes(1, 16, 1, 128), dtype=torch.uint8, device=DEV)
    mqa.mqa_kv_attention_decode(q.to(DEV), k, v, table, i32([0]), i32([0]), i32([200]), out, ws, lse=lse)
    row = Row(q[0], want_k, want_v, 128 ** -0.5, c.qt)
    assert_row(out[0].cpu(), lse[0].cpu(), row)
    slots = i32([[places[p // 64] * 64 + p % 64 for p in range(200)]])
    ws = torch.empty(mqa.mqa_kv_attention_selected_workspace_bytes(1, 200, 16, 1, 128), dtype=torch.uint8, device=DEV)
    mqa.mqa_kv_attention_selected(q.to(DEV), k, v, slots, i32([200]), out, ws, lse=lse)
    assert_row(out[0].cpu(), lse[0].cpu(), row)


def test_decode_repeats_bit_for_bit_on_streams_and_in_graphs():
    c = Case([3000, 50, 900, 0, 5000], 16, 4, 128, "bf16", seed=37)
    q = c.queries(5)
    args = ([0, 1, 2, 3, 4], [0] * 5, c.lengths)
    out, lse = run_decode(c, q, *args)
    again = run_decode(c, q, *args)
    assert torch.equal(out.view(torch.int16), again[0].view(torch.int16)) and torch.equal(lse, again[1])

    d = dict(q=q.to(DEV), seq=i32(args[0]), start=i32(args[1]), end=i32(args[2]), table=c.table.to(DEV))
    size = mqa.mqa_kv_attention_decode_workspace_bytes(5, 16, 4, 128)
    sides = []
    for _ in range(2):      # two calls at once, each with its own workspace and stream
        sides.append((torch.cuda.Stream(), torch.empty_like(d["q"]), torch.empty(size, dtype=torch.uint8, device=DEV)))
    torch.cuda.synchronize()
    for st, o, w in sides:
        mqa.mqa_kv_attention_decode(d["q"], c.dk, c.dv, d["table"], d["seq"], d["start"], d["end"], o, w, stream=st)
    torch.cuda.synchronize()
    for _, o, _ in sides:
        assert torch.equal(o.cpu().view(torch.int16), out.view(torch.int16))

    o, w, l = torch.empty_like(d["q"]), sides[0][2], torch.empty(5, 16, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mqa.mqa_kv_attention_decode(d["q"], c.dk, c.dv, d["table"], d["seq"], d["start"], d["end"], o, w, lse=l)
    for step in range(3):       # lengths and queries change between replays
        lens = [max(0, n - 17 * step) for n in c.lengths]
        qs = c.queries(5)
        d["end"].copy_(i32(lens))
        d["q"].copy_(qs)
        o.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        want = run_decode(c, qs, args[0], args[1], lens)
        assert torch.equal(o.cpu().view(torch.int16), want[0].view(torch.int16)) and torch.equal(l.cpu(), want[1])


# --- selected slots -------------------------------------------------------------


def run_selected(c, q, slots, count, lse=True, scale=None):
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device=DEV)
    got_lse = torch.full(q.shape[:2], 7.0, device=DEV) if lse else None
    size = mqa.mqa_kv_attention_selected_workspace_bytes(q.shape[0], slots.shape[1], c.H, c.Hkv, c.D)
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device=DEV) if size else None
    mqa.mqa_kv_attention_selected(q.to(DEV), c.dk, c.dv, i32(slots), i32(count), out, ws, lse=got_lse, scale=scale,
                                  k_scale=c.k_scale, v_scale=c.v_scale)
    torch.cuda.synchronize()
    return out.cpu(), got_lse.cpu() if lse else None


def check_selected(c, q, slots, count, out, lse):
    for r in range(q.shape[0]):
        k, v = c.by_slot(slots[r, : count[r]])
        assert_row(out[r], None if lse is None else lse[r], Row(q[r], k, v, c.D ** -0.5, c.qt), f"row {r}")


def lists(c, rows, K, seed, counts=None):
    rng = np.random.RandomState(seed)
    good = np.concatenate([np.asarray(c.table[s].numpy(), np.int64)[np.arange(n) // 64] * 64 + np.arange(n) % 64
                           for s, n in enumerate(c.lengths)])
    count = rng.randint(0, K + 1, rows) if counts is None else np.resize(counts, rows)
    slots = np.full((rows, K), -1, np.int64)
    for r in range(rows):
        slots[r, : count[r]] = rng.choice(good, count[r], replace=count[r] > len(good))
    return slots, count


@pytest.mark.parametrize("H,Hkv,D,qtype,cache", SHAPES)
def test_selected_matches_the_plain_form(H, Hkv, D, qtype, cache):
    c = Case([900, 300], H, Hkv, D, qtype, cache, seed=H * 77 + D)
    slots, count = lists(c, 9, 515, 1, [515, 0, 1, 31, 32, 33, 64, 130, 514])
    q = c.queries(9)
    out, lse = run_selected(c, q, slots, count)
    check_selected(c, q, slots, count, out, lse)


@pytest.mark.parametrize("rows,K", [(1, 1), (1, 2500), (3, 1024), (700, 40), (1100, 64), (2, 1025), (5, 0)])
@pytest.mark.parametrize("H,Hkv,layout", [(8, 2, "pool"), (64, 1, "hnd")])
def test_selected_row_counts_and_list_lengths(rows, K, H, Hkv, layout):
    """One workgroup per row, several, and several blocks of one list; the same slot more than once."""
    c = Case([900, 333], H, Hkv, 64, "bf16", seed=rows + K, layout=layout)
    slots, count = lists(c, rows, K, 2)
    if rows < 10 and K:
        count[:] = K
        slots, _ = lists(c, rows, K, 3, [K])
    q = c.queries(rows)
    out, lse = run_selected(c, q, slots, count, lse=rows % 2 == 1)
    check_selected(c, q, slots, count, out, lse)


@pytest.mark.parametrize("rows", [4, 600])
def test_selected_rows_that_fail_closed_leave_the_others_alone(rows):
    c = Case([500], 16, 2, 64, "fp16", seed=41)
    slots, count = lists(c, rows, 512, 5, [512])
    slots[1, 300] = 64 * c.P
    slots[2, 511] = -1
    q = c.queries(rows)
    mqa.mqa_fp4_status()
    out, lse = run_selected(c, q, slots, count)
    assert mqa.mqa_fp4_status() == mqa.STATUS_BAD_PAGE
    good = [r for r in range(rows) if r not in (1, 2)]
    assert torch.isnan(out[1:3]).all() and torch.isnan(lse[1:3]).all()
    check_selected(c, q[good], slots[good], count[good], out[good], lse[good])
    count[0], count[3] = 513, -2
    out, lse = run_selected(c, q, slots, count)
    assert mqa.mqa_fp4_status() == mqa.STATUS_BAD_PAGE | mqa.STATUS_BAD_WINDOW
    assert torch.isnan(out[:4]).all() and torch.isnan(lse[:4]).all()
    check_selected(c, q[4:], slots[4:], count[4:], out[4:], lse[4:])
    assert mqa.mqa_fp4_status() == 0


def test_selected_replays_in_a_graph():
    c = Case([2000], 64, 1, 128, "bf16", seed=43)
    slots, count = lists(c, 4, 512, 6, [512])
    q = c.queries(4)
    d = dict(q=q.to(DEV), slots=i32(slots), count=i32(count), out=torch.empty(4, 64, 128, dtype=c.qt, device=DEV),
             ws=torch.empty(mqa.mqa_kv_attention_selected_workspace_bytes(4, 512, 64, 1, 128), dtype=torch.uint8, device=DEV))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mqa.mqa_kv_attention_selected(d["q"], c.dk, c.dv, d["slots"], d["count"], d["out"], d["ws"])
    for step in range(3):
        slots, count = lists(c, 4, 512, 60 + step)
        d["slots"].copy_(i32(slots))
        d["count"].copy_(i32(count))
        graph.replay()
        torch.cuda.synchronize()
        want, _ = run_selected(c, q, slots, count)
        assert torch.equal(d["out"].cpu().view(torch.int16), want.view(torch.int16))
        check_selected(c, q, slots, count, d["out"].cpu(), None)
