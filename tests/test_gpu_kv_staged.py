"""Attention over the key-value cache with more than 16 query heads per key head: keys and values go
through LDS stages (two of them, or four where a page's keys take 8 KB and less). The hard cases of the
register kernels on these, on the GPU, against the plain form in 64 bits; and scales for lists and weights."""

import numpy as np
import pytest
import torch

import fp4_mqa_scoring_amd as mqa
from kv_ref import Row, assert_row
from test_gpu_kv_attention import DEV, Case, check_decode, i32, lists, run_decode, run_selected
from test_gpu_kv_evict import run_weights

pytestmark = pytest.mark.gpu

# H, Hkv, D, q type, cache: two stages, four stages; one and two tiles of 16 heads per half; key heads, halves without heads
TWO = [(64, 1, 128, "bf16", "bf16"), (34, 2, 256, "fp16", "fp16")]
FOUR = [(20, 1, 64, "bf16", "e4m3"), (40, 2, 64, "fp16", "fp16"), (50, 1, 64, "bf16", "bf16"), (24, 1, 128, "fp16", "e4m3"),
        (100, 2, 128, "bf16", "e4m3"), (36, 1, 256, "bf16", "e4m3")]
STAGED = TWO + FOUR


def check_rows(c, q, rows, out, lse, good, scale=None):
    """Rows in `good` match, all others failed closed."""
    scale = c.D ** -0.5 if scale is None else scale
    for r, row in enumerate(rows):
        if r in good:
            k, v = c.at(*row)
            assert_row(out[r], lse[r], Row(q[r], k, v, scale, c.qt), f"row {r}")
        else:
            assert torch.isnan(out[r]).all() and torch.isnan(lse[r]).all(), r


@pytest.mark.parametrize("H,Hkv,D,qtype,cache", STAGED + [
    (17, 1, 64, "fp16", "e4m3"), (32, 1, 64, "bf16", "e4m3"), (62, 2, 128, "fp16", "e4m3"), (17, 1, 128, "bf16", "e4m3"),
    (32, 1, 64, "fp16", "fp16"), (64, 2, 128, "fp16", "fp16")])
def test_lengths_and_lists(H, Hkv, D, qtype, cache):
    lengths = [1, 0, 15, 16, 17, 31, 32, 33, 63, 64, 65, 129, 500, 3001]
    c = Case(lengths, H, Hkv, D, qtype, cache, seed=H + D)
    q = c.queries(len(lengths))
    args = (list(range(len(lengths))), [0] * len(lengths), lengths)
    check_decode(c, q, *args, *run_decode(c, q, *args))
    slots, count = lists(c, 9, 515, 1, [515, 0, 1, 15, 16, 17, 64, 130, 514])
    out, lse = run_selected(c, q[:9], slots, count)
    for r in range(9):
        assert_row(out[r], lse[r], Row(q[r], *c.by_slot(slots[r, :count[r]]), D ** -0.5, c.qt), f"row {r}")


@pytest.mark.parametrize("layout", ["nhd", "hnd", "pool"])
@pytest.mark.parametrize("H,Hkv,D,qtype,cache", FOUR + TWO[:1])
def test_windows_anywhere(H, Hkv, D, qtype, cache, layout):
    """Windows that start and end inside pages and stages, several rows per sequence in no order, a query pitch."""
    c = Case([700, 1400, 64, 333], H, Hkv, D, qtype, cache, seed=5, layout=layout, capacity=100)
    wins = [(0, 0, 700), (1, 1337, 1400), (3, 100, 101), (1, 31, 33), (0, 699, 700), (2, 0, 64), (2, 64, 64), (1, 0, 0),
            (3, 33, 290), (0, 63, 65), (1, 640, 1281), (2, 5, 5), (1, 15, 17), (1, 47, 1343), (0, 1, 32), (0, 48, 64)]
    seq, start, end = zip(*wins)
    q = c.queries(len(wins))
    wide = torch.zeros(len(wins), H + 4, D, dtype=c.qt, device=DEV)
    wide[:, 2:2 + H] = q.to(DEV)
    out, lse = run_decode(c, q, seq, start, end, dq=wide[:, 2:2 + H])
    check_decode(c, q, seq, start, end, out, lse)


@pytest.mark.parametrize("scale", [-0.3, 0.0, 3.0])
@pytest.mark.parametrize("H,Hkv,D,qtype,cache", [(6, 2, 128, "bf16", "bf16"), (3, 1, 64, "fp16", "e4m3")] + TWO + FOUR[:3])
def test_scales(H, Hkv, D, qtype, cache, scale):
    """A negative scale, a scale of 0 (plain mean) and a steep one, for windows, lists and weights."""
    c = Case([500, 70], H, Hkv, D, qtype, cache, seed=8, spread=1.0)
    q = c.queries(2)
    out, lse = run_decode(c, q, [0, 1], [0, 3], [500, 70], scale=scale)
    check_decode(c, q, [0, 1], [0, 3], [500, 70], out, lse, scale=scale)
    slots, count = lists(c, 2, 300, 4, [300, 77])
    got, got_lse = run_selected(c, q, slots, count, scale=scale)
    for r in range(2):
        assert_row(got[r], got_lse[r], Row(q[r], *c.by_slot(slots[r, :count[r]]), scale, c.qt), f"row {r}")
    acc = torch.rand(2, 64 * c.table.shape[1], generator=c.g)
    given, want, tol = lse.clone(), acc.double().clone(), torch.zeros(acc.shape, dtype=torch.float64)
    for r, (lo, hi) in enumerate(((0, 500), (3, 70))):
        row = Row(q[r], c.at(r, lo, hi)[0], None, scale, c.qt)
        given[r] = row.lse.float()
        want[r, lo:hi] += (row.w * torch.exp(row.lse - given[r].double())[:, None]).sum(0)
        tol[r, lo:hi] += 1.01 * row.w_tol.sum(0) + (H + 2) * 2.0 ** -24 * want[r, lo:hi]
    got = run_weights(c, q, given, [0, 1], [0, 3], [500, 70], acc, scale=scale)
    assert ((got.double() - want).abs() <= tol).all()


@pytest.mark.parametrize("rows", [1024, 1025, 1500])
@pytest.mark.parametrize("H,Hkv,D,qtype,cache", [TWO[0], FOUR[0], FOUR[1]])
def test_more_rows_than_one_workgroup_plans(H, Hkv, D, qtype, cache, rows):
    lengths = [int(x) for x in np.random.RandomState(3).randint(0, 150, 40)]
    c = Case(lengths, H, Hkv, D, qtype, cache, seed=13)
    rng = np.random.RandomState(4)
    seq = rng.randint(0, 40, rows)
    end = np.array([rng.randint(0, lengths[s] + 1) for s in seq])
    start = np.array([rng.randint(0, e + 1) for e in end])
    q = c.queries(rows)
    out, lse = run_decode(c, q, seq, start, end)
    some = np.unique(np.r_[0:40, rng.randint(0, rows, 200), rows - 5:rows])
    check_decode(c, q[some], seq[some], start[some], end[some], out[some], lse[some])
    empty = torch.from_numpy(end == start)
    assert (out[empty] == 0).all() and (lse[empty] == float("-inf")).all()


@pytest.mark.parametrize("H,Hkv,D,qtype,cache", STAGED)
def test_rows_that_fail_closed_leave_the_others_alone(H, Hkv, D, qtype, cache):
    c = Case([300, 200, 100, 20000, 20000], H, Hkv, D, qtype, cache, seed=23)
    width = c.table.shape[1]
    c.table[1, 2] = c.P            # outside the pool
    c.table[2, 0] = -1
    c.table[4, 150] = c.P + 5      # in one of the many parts of a long sequence
    rows = [(0, 0, 300), (5, 0, 10), (-1, 0, 10), (0, -1, 10), (0, 20, 10), (0, 0, 64 * width + 1), (1, 0, 200), (1, 0, 128),
            (2, 0, 100), (2, 64, 100), (2, 64, 64), (0, 0, 0), (3, 5, 20000), (4, 5, 20000), (4, 5, 9600), (4, 9664, 20000)]
    seq, start, end = zip(*rows)
    q = c.queries(len(rows))
    mqa.mqa_fp4_status()
    out, lse = run_decode(c, q, seq, start, end)
    assert mqa.mqa_fp4_status() == mqa.STATUS_BAD_WINDOW | mqa.STATUS_BAD_PAGE
    check_rows(c, q, rows, out, lse, {0, 7, 9, 10, 11, 12, 14, 15})
    run_decode(c, q[:1], [0], [0], [300])
    assert mqa.mqa_fp4_status() == 0


@pytest.mark.parametrize("rows", [4, 600])
@pytest.mark.parametrize("H,Hkv,D,qtype,cache", [TWO[0], FOUR[0], FOUR[1], FOUR[4]])
def test_lists_that_fail_closed_leave_the_others_alone(H, Hkv, D, qtype, cache, rows):
    """Bad slots in the first block of 1,024 and behind it, with the list in one part and in several."""
    c = Case([500], H, Hkv, D, qtype, cache, seed=41)
    K = 1500
    slots, count = lists(c, rows, K, 5, [K])
    slots[1, 300], slots[2, K - 1], slots[3, 1024] = 64 * c.P, -1, 2 ** 31 - 1
    q = c.queries(rows)
    mqa.mqa_fp4_status()

    def check(good):
        for r in good[:8] + good[-8:]:
            assert_row(out[r], lse[r], Row(q[r], *c.by_slot(slots[r, :count[r]]), D ** -0.5, c.qt), f"row {r}")

    out, lse = run_selected(c, q, slots, count)
    assert mqa.mqa_fp4_status() == mqa.STATUS_BAD_PAGE
    assert torch.isnan(out[1:4]).all() and torch.isnan(lse[1:4]).all()
    check([r for r in range(rows) if r not in (1, 2, 3)])
    count[:4] = K + 1, 300, -2, 0
    out, lse = run_selected(c, q, slots, count)
    assert mqa.mqa_fp4_status() == mqa.STATUS_BAD_WINDOW
    assert torch.isnan(out[[0, 2]]).all() and torch.isnan(lse[[0, 2]]).all()
    assert (out[3] == 0).all() and (lse[3] == float("-inf")).all()
    check([1] + list(range(4, rows)))
    assert mqa.mqa_fp4_status() == 0


@pytest.mark.parametrize("H,Hkv,D,qtype,cache", [(2, 1, 64, "bf16", "bf16"), TWO[0], TWO[1], FOUR[1], FOUR[2]])
def test_nan_and_infinities_inside_the_window(H, Hkv, D, qtype, cache):
    """IEEE rules inside the window and the list: a NaN key and a score of +infinity make the row NaN, an infinite value an
    infinite dim; a key that scores -infinity drops out, and nothing but such ones is NaN."""
    c = Case([100] * 4, H, Hkv, D, qtype, cache, seed=29)
    c.k[c.table[0, 1], 3] = float("nan")
    c.v[c.table[1, 0], 5, :, 7] = float("inf")
    q = c.queries(4)
    q[2:] = q[2:].abs() + 0.1
    c.k[c.table[2, 0], 9] = float("-inf")
    c.k[c.table[3, 1], 20] = float("inf")
    c.dk, c.dv = c.k.to(DEV), c.v.to(DEV)
    slots = np.stack([[int(c.table[s, p // 64]) * 64 + p % 64 for p in range(100)] for s in range(4)])
    k, v = c.at(2, 0, 100)
    keep = torch.arange(100) != 9
    want = Row(q[2], k[keep], v[keep], D ** -0.5, c.qt)
    for out, lse in (run_decode(c, q, [0, 1, 2, 3], [0] * 4, [100] * 4), run_selected(c, q, slots, [100] * 4)):
        assert torch.isnan(out[0]).all() and torch.isnan(lse[0]).all()
        assert torch.isinf(out[1, :, 7]).all() and (out[1, :, 7] > 0).all()
        assert torch.isfinite(out[1, :, :7]).all() and torch.isfinite(out[1, :, 8:]).all()
        assert_row(out[2], lse[2], want, "row 2")
        assert torch.isnan(out[3]).all()
    for out, lse in (run_decode(c, q[2:3], [2], [9], [10]), run_selected(c, q[2:3], slots[2:3, 9:10], [1])):
        assert torch.isnan(out).all() and (lse == float("-inf")).all()


@pytest.mark.parametrize("H,cache", [(64, "bf16"), (20, "e4m3")])
def test_offsets_beyond_32_bits(H, cache):
    """A pool of 6 GiB whose used pages lie at both ends."""
    size = 1 if cache == "e4m3" else 2
    P = 6 * 2 ** 30 // (64 * 128 * size)
    c = Case([200], H, 1, 128, "bf16", cache, seed=31, spare=0)
    raw = torch.uint8 if size == 1 else torch.int16
    k = torch.empty(P, 64, 1, 128, dtype=raw, device=DEV)
    v = torch.empty_like(k)
    places = [0, P - 1, P // 2 + 1, P - 2]
    for i in range(4):
        page = int(c.table[0, i])
        k[places[i]] = c.k[page].view(raw).to(DEV)
        v[places[i]] = c.v[page].view(raw).to(DEV)
    q = c.queries(1)
    row = Row(q[0], *c.at(0, 0, 200), 128 ** -0.5, c.qt)
    c.dk, c.dv = k.view(c.ct), v.view(c.ct)
    c.table = torch.tensor([places], dtype=torch.int32)
    out, lse = run_decode(c, q, [0], [0], [200])
    assert_row(out[0], lse[0], row)
    slots = np.array([[places[p // 64] * 64 + p % 64 for p in range(200)]])
    out, lse = run_selected(c, q, slots, [200])
    assert_row(out[0], lse[0], row)


@pytest.mark.parametrize("H,Hkv,D,qtype,cache", [TWO[0], FOUR[1], FOUR[3]])
def test_graph_replays_give_the_eager_bits(H, Hkv, D, qtype, cache):
    c = Case([3000, 50, 900, 0, 5000], H, Hkv, D, qtype, cache, seed=37)
    q = c.queries(5)
    d = dict(q=q.to(DEV), seq=i32(range(5)), start=i32([0] * 5), end=i32(c.lengths), table=c.table.to(DEV))
    ws = torch.empty(mqa.mqa_kv_attention_decode_workspace_bytes(5, H, Hkv, D), dtype=torch.uint8, device=DEV)
    o, l = torch.empty_like(d["q"]), torch.empty(5, H, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mqa.mqa_kv_attention_decode(d["q"], c.dk, c.dv, d["table"], d["seq"], d["start"], d["end"], o, ws, lse=l,
                                    k_scale=c.k_scale, v_scale=c.v_scale)
    for step in range(4):
        lens = [max(0, n - 17 * step) for n in c.lengths]
        qs = c.queries(5)
        d["end"].copy_(i32(lens))
        d["q"].copy_(qs)
        o.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        out, lse = run_decode(c, qs, range(5), [0] * 5, lens)
        assert torch.equal(o.cpu().view(torch.int16), out.view(torch.int16)) and torch.equal(l.cpu(), lse)
        check_decode(c, qs, range(5), [0] * 5, lens, out, lse)
