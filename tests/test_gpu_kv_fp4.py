"""Attention over a paged cache in 4 bits, on the GPU, against the plain form in 64 bits: the numbers that the codes
stand for are exact in the queries' type, so the bounds are those of tests/kv_ref.py."""
import numpy as np
import pytest
import torch

import fp4_mqa_scoring_amd as mqa
from kv_new_ref import fp4_numbers
from kv_ref import Row, assert_row

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
DEV = "cuda:0"


class Case:
    """Sequences of the given lengths over a shuffled pool whose unused positions hold scales of NaN."""

    def __init__(self, lengths, H, Hkv, D, kind="bf16", seed=0, layout="nhd", spare=2, capacity=0, exponents=(124, 128)):
        g = self.g = torch.Generator().manual_seed(seed)
        self.H, self.Hkv, self.D, self.qt, self.lengths = H, Hkv, D, TYPES[kind], list(lengths)
        pages = [(n + 63) // 64 for n in lengths]
        self.P = sum(pages) + spare
        perm = torch.randperm(self.P, generator=g).int()
        self.table = torch.full((max(1, len(pages)), max(max(pages, default=0), capacity, 1)), -1, dtype=torch.int32)
        at = 0
        for i, n in enumerate(pages):
            self.table[i, :n] = perm[at:at + n]
            at += n
        used = torch.zeros(self.P, 64, dtype=torch.bool)
        for i, n in enumerate(self.lengths):
            for p in range(pages[i]):
                used[self.table[i, p], : min(64, n - 64 * p)] = True
        self.host = {}
        for name in "kv":
            self.host[name] = torch.randint(0, 256, (self.P, 64, Hkv, D // 2), generator=g).to(torch.uint8)
            s = torch.randint(exponents[0], exponents[1] + 1, (self.P, 64, Hkv, D // 32), generator=g).to(torch.uint8)
            s[~used] = 255
            self.host[name + "s"] = s
        self.layout = layout
        self.upload()

    def upload(self):
        self.dev = {n: self._place(t.to(DEV)) for n, t in self.host.items()}

    def _place(self, t):
        if self.layout == "nhd":
            return t
        if self.layout == "hnd":
            return t.transpose(1, 2).contiguous().transpose(1, 2)
        whole = torch.full((t.shape[0], 2, 64, t.shape[2] + 1, t.shape[3]), 255, dtype=torch.uint8, device=DEV)
        view = whole[:, 1, :, 1:, :]
        view.copy_(t)
        return view

    def cache(self):
        return [self.dev[n] for n in ("k", "ks", "v", "vs")]

    def queries(self, n, spread=1.5):
        return (torch.randn(n, self.H, self.D, generator=self.g) * spread).to(self.qt)

    def slots(self, seq, lo, hi):
        pos = torch.arange(lo, hi)
        return self.table[seq].long()[pos // 64] * 64 + pos % 64

    def numbers(self, slots):
        s = torch.as_tensor(np.asarray(slots, dtype=np.int64))
        return [fp4_numbers(self.host[n][s // 64, s % 64], self.host[n + "s"][s // 64, s % 64]) for n in "kv"]

    def row(self, q, slots, scale=None):
        return Row(q, *self.numbers(slots), self.D ** -0.5 if scale is None else scale, self.qt)


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).to(DEV)


def run_decode(c, q, seq, start, end, lse=True, scale=None, dq=None, out=None):
    dq = q.to(DEV) if dq is None else dq
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device=DEV) if out is None else out
    got_lse = torch.full(q.shape[:2], 7.0, device=DEV) if lse else None
    ws = torch.full((mqa.mqa_kv_attention_decode_workspace_bytes(q.shape[0], c.H, c.Hkv, c.D),), 0xFF, dtype=torch.uint8, device=DEV)
    mqa.mqa_kv_attention_decode_fp4(dq, *c.cache(), c.table.to(DEV), i32(seq), i32(start), i32(end), out, ws, lse=got_lse, scale=scale)
    torch.cuda.synchronize()
    return out.cpu(), got_lse.cpu() if lse else None


def check_decode(c, q, seq, start, end, out, lse, scale=None):
    for r in range(q.shape[0]):
        assert_row(out[r], None if lse is None else lse[r], c.row(q[r], c.slots(int(seq[r]), int(start[r]), int(end[r])), scale), f"row {r}")


SHAPES = [(8, 2, 128, "bf16"), (16, 1, 128, "fp16"), (64, 1, 128, "bf16"), (5, 5, 64, "fp16"), (40, 2, 64, "bf16"), (128, 1, 64, "fp16"),
          (3, 1, 256, "bf16"), (48, 2, 256, "fp16"), (65, 1, 128, "fp16"), (8, 8, 64, "bf16"), (33, 1, 64, "fp16"), (70, 2, 256, "bf16"),
          (17, 1, 128, "fp16"), (70, 1, 128, "bf16"), (34, 1, 256, "bf16"), (100, 2, 128, "fp16")]


@pytest.mark.parametrize("H,Hkv,D,kind", SHAPES)
def test_decode_matches_the_plain_form(H, Hkv, D, kind):
    lengths = [1, 0, 31, 32, 33, 63, 64, 65, 127, 129, 200, 1000, 2777]
    c = Case(lengths, H, Hkv, D, kind, seed=H * 1000 + D)
    q = c.queries(len(lengths))
    args = (list(range(len(lengths))), [0] * len(lengths), lengths)
    out, lse = run_decode(c, q, *args)
    check_decode(c, q, *args, out, lse)


@pytest.mark.parametrize("layout", ["hnd", "pool"])
@pytest.mark.parametrize("D,H,Hkv", [(128, 12, 3), (64, 12, 3), (256, 34, 1), (64, 34, 1), (128, 66, 2)])
def test_decode_windows_rows_and_strides(layout, D, H, Hkv):
    """Windows that start and end anywhere, several rows per sequence in no order, queries with a row pitch, no lse."""
    c = Case([700, 1400, 64, 333], H, Hkv, D, "bf16", seed=5, layout=layout, capacity=100)
    wins = [(0, 0, 700), (1, 1337, 1400), (3, 100, 101), (1, 31, 33), (0, 699, 700), (2, 0, 64), (2, 64, 64), (1, 0, 0), (3, 33, 290),
            (0, 63, 65), (1, 640, 1281), (2, 5, 5)]
    seq, start, end = zip(*wins)
    q = c.queries(len(wins))
    wide = torch.zeros(len(wins), H + 4, D, dtype=c.qt, device=DEV)
    wide[:, 2:2 + H] = q.to(DEV)
    out, _ = run_decode(c, q, seq, start, end, lse=False, dq=wide[:, 2:2 + H])
    check_decode(c, q, seq, start, end, out, None)


@pytest.mark.parametrize("H,Hkv", [(6, 2), (40, 1)])
@pytest.mark.parametrize("scale", [-0.3, 0.0, 3.0])
def test_decode_scales(scale, H, Hkv):
    c = Case([500, 70], H, Hkv, 128, "bf16", seed=8)
    q = c.queries(2, 0.7)
    args = ([0, 1], [0, 3], [500, 70])
    out, lse = run_decode(c, q, *args, scale=scale)
    check_decode(c, q, *args, out, lse, scale=scale)


@pytest.mark.parametrize("kind,exponents", [("bf16", (0, 40)), ("bf16", (180, 190)), ("fp16", (104, 110)), ("fp16", (136, 140))])
@pytest.mark.parametrize("H", [4, 40])
def test_decode_block_scales_far_from_one(kind, exponents, H):
    """Numbers at both ends of the queries' type; the score's factor keeps the scores near one."""
    c = Case([300], H, 1, 64, kind, seed=12, exponents=exponents)
    q = c.queries(1)
    scale = 0.05 * 2.0 ** (127 - exponents[1])
    if not 1e-38 < scale < 1e38:
        scale = 1e37
    out, lse = run_decode(c, q, [0], [0], [300], scale=scale)
    check_decode(c, q, [0], [0], [300], out, lse, scale=scale)


def test_decode_more_rows_than_one_workgroup_plans():
    lengths = [int(x) for x in np.random.RandomState(3).randint(0, 150, 40)]
    c = Case(lengths, 4, 2, 64, "bf16", seed=13)
    rng = np.random.RandomState(4)
    seq = rng.randint(0, 40, 1500)
    end = np.array([rng.randint(0, lengths[s] + 1) for s in seq])
    start = np.array([rng.randint(0, e + 1) for e in end])
    q = c.queries(1500)
    out, lse = run_decode(c, q, seq, start, end)
    check_decode(c, q, seq, start, end, out, lse)


@pytest.mark.parametrize("H,Hkv,D", [(8, 2, 128), (64, 1, 128), (4, 1, 256), (40, 1, 64), (32, 1, 256)])
def test_decode_one_long_sequence_is_split_and_joined(H, Hkv, D):
    c = Case([40000], H, Hkv, D, "bf16", seed=19)
    q = c.queries(1)
    out, lse = run_decode(c, q, [0], [0], [40000])
    check_decode(c, q, [0], [0], [40000], out, lse)


@pytest.mark.parametrize("H,Hkv", [(8, 2), (40, 1)])
def test_decode_rows_that_fail_closed_leave_the_others_alone(H, Hkv):
    c = Case([300, 200, 100], H, Hkv, 128, "bf16", seed=23)
    c.table[1, 2] = c.P
    c.table[2, 0] = -1
    rows = [(0, 0, 300), (3, 0, 10), (-1, 0, 10), (0, -1, 10), (0, 20, 10), (0, 0, 64 * c.table.shape[1] + 1), (1, 0, 200), (1, 0, 128),
            (2, 0, 100), (2, 64, 100), (2, 64, 64), (0, 0, 0)]
    seq, start, end = zip(*rows)
    q = c.queries(len(rows))
    mqa.mqa_fp4_status()
    out, lse = run_decode(c, q, seq, start, end)
    assert mqa.mqa_fp4_status() == mqa.STATUS_BAD_WINDOW | mqa.STATUS_BAD_PAGE
    for r in range(len(rows)):
        if r in (0, 7, 9, 10, 11):
            assert_row(out[r], lse[r], c.row(q[r], c.slots(*rows[r])), f"row {r}")
        else:
            assert torch.isnan(out[r]).all() and torch.isnan(lse[r]).all(), r


@pytest.mark.parametrize("H", [4, 40])
def test_a_scale_of_nan_counts_inside_the_window_only(H):
    c = Case([100, 100], H, 1, 64, "bf16", seed=29)
    c.host["ks"][c.table[0, 1], 3, 0, 1] = 255
    c.host["vs"][c.table[1, 0], 5, 0, 1] = 255
    c.upload()
    q = c.queries(4)
    out, lse = run_decode(c, q, [0, 1, 0, 1], [0, 0, 0, 6], [100, 100, 67, 100])
    assert torch.isnan(out[0]).all() and torch.isnan(lse[0]).all()
    assert torch.isnan(out[1, :, 32:]).all() and torch.isfinite(out[1, :, :32]).all()
    for r, (s, lo, hi) in ((2, (0, 0, 67)), (3, (1, 6, 100))):
        assert_row(out[r], lse[r], c.row(q[r], c.slots(s, lo, hi)), r)


def test_batches_without_rows_sequences_or_pages():
    c = Case([70], 4, 2, 64, "bf16", seed=33)
    assert run_decode(c, c.queries(0), [], [], [])[0].shape == (0, 4, 64)
    mqa.mqa_fp4_status()
    q = c.queries(3)
    c.dev = {n: t[:0] for n, t in c.dev.items()}
    out, lse = run_decode(c, q, [0, 0, 0], [0, 5, 0], [0, 5, 1])
    assert mqa.mqa_fp4_status() == mqa.STATUS_BAD_PAGE
    assert (out[:2] == 0).all() and (lse[:2] == float("-inf")).all() and torch.isnan(out[2]).all()
    out, lse = run_selected(c, q, np.zeros((3, 2), np.int64), [0, 0, 1])
    assert mqa.mqa_fp4_status() == mqa.STATUS_BAD_PAGE
    assert (out[:2] == 0).all() and torch.isnan(out[2]).all()


@pytest.mark.parametrize("H", [16, 40])
def test_offsets_beyond_32_bits(H):
    """A pool of 5 GiB of codes whose used pages lie at both ends."""
    P = 5 * 2 ** 30 // (64 * 64)
    c = Case([200], H, 1, 128, "bf16", seed=31, spare=0)
    places = [0, P - 1, P // 2 + 1, P - 2]
    big = {n: torch.empty(P, 64, 1, t.shape[3], dtype=torch.uint8, device=DEV) for n, t in c.host.items()}
    for i in range(4):
        for n, t in c.host.items():
            big[n][places[i]] = t[int(c.table[0, i])].to(DEV)
    q = c.queries(1)
    row = c.row(q[0], c.slots(0, 0, 200))
    c.dev, c.table = big, torch.tensor([places], dtype=torch.int32)
    out, lse = run_decode(c, q, [0], [0], [200])
    assert_row(out[0], lse[0], row)
    out, lse = run_selected(c, q, [[places[p // 64] * 64 + p % 64 for p in range(200)]], [200])
    assert_row(out[0], lse[0], row)


@pytest.mark.parametrize("H,Hkv", [(16, 4), (64, 1)])
def test_decode_repeats_bit_for_bit_on_streams_in_place_and_in_graphs(H, Hkv):
    c = Case([3000, 50, 900, 0, 5000], H, Hkv, 128, "bf16", seed=37)
    q = c.queries(5)
    args = ([0, 1, 2, 3, 4], [0] * 5, c.lengths)
    out, lse = run_decode(c, q, *args)
    again = run_decode(c, q, *args)
    assert torch.equal(out.view(torch.int16), again[0].view(torch.int16)) and torch.equal(lse, again[1])
    same = q.to(DEV)
    got, _ = run_decode(c, q, *args, dq=same, out=same)
    assert torch.equal(got.view(torch.int16), out.view(torch.int16))
    d = dict(q=q.to(DEV), seq=i32(args[0]), start=i32(args[1]), end=i32(args[2]), table=c.table.to(DEV))
    size = mqa.mqa_kv_attention_decode_workspace_bytes(5, H, Hkv, 128)
    sides = [(torch.cuda.Stream(), torch.empty_like(d["q"]), torch.empty(size, dtype=torch.uint8, device=DEV)) for _ in range(2)]
    torch.cuda.synchronize()
    for st, o, w in sides:
        mqa.mqa_kv_attention_decode_fp4(d["q"], *c.cache(), d["table"], d["seq"], d["start"], d["end"], o, w, stream=st)
    torch.cuda.synchronize()
    for _, o, _ in sides:
        assert torch.equal(o.cpu().view(torch.int16), out.view(torch.int16))
    o, w, l = torch.empty_like(d["q"]), sides[0][2], torch.empty(5, H, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mqa.mqa_kv_attention_decode_fp4(d["q"], *c.cache(), d["table"], d["seq"], d["start"], d["end"], o, w, lse=l)
    for step in range(3):
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
    slots = np.asarray(slots)
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device=DEV)
    got_lse = torch.full(q.shape[:2], 7.0, device=DEV) if lse else None
    size = mqa.mqa_kv_attention_selected_workspace_bytes(q.shape[0], slots.shape[1], c.H, c.Hkv, c.D)
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device=DEV) if size else None
    mqa.mqa_kv_attention_selected_fp4(q.to(DEV), *c.cache(), i32(slots), i32(count), out, ws, lse=got_lse, scale=scale)
    torch.cuda.synchronize()
    return out.cpu(), got_lse.cpu() if lse else None


def check_selected(c, q, slots, count, out, lse):
    for r in range(q.shape[0]):
        assert_row(out[r], None if lse is None else lse[r], c.row(q[r], slots[r, : count[r]]), f"row {r}")


def lists(c, rows, K, seed, counts=None):
    rng = np.random.RandomState(seed)
    good = np.concatenate([c.slots(s, 0, n).numpy() for s, n in enumerate(c.lengths)])
    count = rng.randint(0, K + 1, rows) if counts is None else np.resize(counts, rows)
    slots = np.full((rows, K), -1, np.int64)
    for r in range(rows):
        slots[r, : count[r]] = rng.choice(good, count[r], replace=count[r] > len(good))
    return slots, count


@pytest.mark.parametrize("H,Hkv,D,kind", SHAPES)
def test_selected_matches_the_plain_form(H, Hkv, D, kind):
    c = Case([900, 300], H, Hkv, D, kind, seed=H * 77 + D)
    slots, count = lists(c, 9, 515, 1, [515, 0, 1, 31, 32, 33, 64, 130, 514])
    q = c.queries(9)
    out, lse = run_selected(c, q, slots, count)
    check_selected(c, q, slots, count, out, lse)


@pytest.mark.parametrize("rows,K", [(1, 1), (1, 2500), (3, 1024), (700, 40), (1100, 64), (2, 1025), (5, 0)])
@pytest.mark.parametrize("H,Hkv,layout", [(8, 2, "pool"), (64, 1, "hnd")])
def test_selected_row_counts_and_list_lengths(rows, K, H, Hkv, layout):
    c = Case([900, 333], H, Hkv, 64, "bf16", seed=rows + K, layout=layout)
    slots, count = lists(c, rows, K, 3, [K] if rows < 10 and K else None)
    q = c.queries(rows)
    out, lse = run_selected(c, q, slots, count, lse=rows % 2 == 1)
    check_selected(c, q, slots, count, out, lse)


@pytest.mark.parametrize("rows", [4, 600])
@pytest.mark.parametrize("H,Hkv", [(16, 2), (40, 1)])
def test_selected_rows_that_fail_closed_leave_the_others_alone(rows, H, Hkv):
    c = Case([500], H, Hkv, 64, "fp16", seed=41)
    slots, count = lists(c, rows, 512, 5, [512])
    slots[1, 300] = 64 * c.P
    slots[2, 511] = -1
    q = c.queries(rows)
    mqa.mqa_fp4_status()
    count[0], count[3] = 513, -2
    out, lse = run_selected(c, q, slots, count)
    assert mqa.mqa_fp4_status() == mqa.STATUS_BAD_PAGE | mqa.STATUS_BAD_WINDOW
    assert torch.isnan(out[:4]).all() and torch.isnan(lse[:4]).all()
    check_selected(c, q[4:], slots[4:], count[4:], out[4:], lse[4:])


def test_selected_replays_in_a_graph():
    c = Case([2000], 64, 1, 128, "bf16", seed=43)
    slots, count = lists(c, 4, 512, 6, [512])
    q = c.queries(4)
    d = dict(q=q.to(DEV), slots=i32(slots), count=i32(count), out=torch.empty(4, 64, 128, dtype=c.qt, device=DEV),
             ws=torch.empty(mqa.mqa_kv_attention_selected_workspace_bytes(4, 512, 64, 1, 128), dtype=torch.uint8, device=DEV))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mqa.mqa_kv_attention_selected_fp4(d["q"], *c.cache(), d["slots"], d["count"], d["out"], d["ws"])
    for step in range(3):
        slots, count = lists(c, 4, 512, 60 + step)
        d["slots"].copy_(i32(slots))
        d["count"].copy_(i32(count))
        graph.replay()
        torch.cuda.synchronize()
        want, _ = run_selected(c, q, slots, count)
        assert torch.equal(d["out"].cpu().view(torch.int16), want.view(torch.int16))
        check_selected(c, q, slots, count, d["out"].cpu(), None)
