"""Accumulated attention weight, the choice of what a budget keeps, and the move of
it, on the GPU, against the plain forms in 64 bits."""
import numpy as np
import pytest
import torch

import fp4_mqa_scoring_amd as mqa
from kv_ref import Row, evict_keep
from test_gpu_kv_attention import DEV, Case, i32

pytestmark = pytest.mark.gpu


def run_weights(c, q, lse, seq, start, end, acc, scale=None):
    d = acc.to(DEV)
    mqa.mqa_kv_weights_accumulate(q.to(DEV), lse.to(DEV), c.dk, c.table.to(DEV), i32(seq), i32(start), i32(end), d,
                                  scale=scale, k_scale=c.k_scale)
    torch.cuda.synchronize()
    return d.cpu()


def expected_weights(c, q, seq, start, end, acc, skip=()):
    """(sums, their bounds, whether a window holds them, lse): a sum of t terms added in 32 bits is off by
    the terms' own bounds and (t + 2) 2^-24 of the total."""
    want, tol = acc.double().clone(), torch.zeros(acc.shape, dtype=torch.float64)
    held = torch.zeros(acc.shape, dtype=torch.bool)
    terms = torch.zeros(acc.shape, dtype=torch.float64)
    lse = torch.full((q.shape[0], c.H), float("-inf"))
    for r in range(q.shape[0]):
        if r in skip or end[r] <= start[r]:
            continue
        k, _ = c.at(int(seq[r]), int(start[r]), int(end[r]))
        row = Row(q[r], k, None, c.D ** -0.5, c.qt)
        lse[r] = row.lse.float()
        # the weights go by the 32-bit lse that the call is given
        w = row.w * torch.exp(row.lse - lse[r].double())[:, None]
        at = slice(int(start[r]), int(end[r]))
        want[seq[r], at] += w.sum(0)
        tol[seq[r], at] += 1.01 * row.w_tol.sum(0)
        terms[seq[r], at] += c.H
        held[seq[r], at] = True
    tol += (terms + 2) * 2.0 ** -24 * want
    return want, tol, held, lse


@pytest.mark.parametrize("H,Hkv,D,qtype,cache", [
    (8, 2, 128, "bf16", "bf16"), (64, 1, 128, "bf16", "bf16"), (5, 5, 64, "fp16", "fp16"), (70, 2, 64, "fp16", "e4m3"),
    (3, 1, 256, "bf16", "e4m3"), (40, 1, 256, "fp16", "fp16"), (130, 1, 128, "bf16", "e4m3"), (24, 24, 64, "bf16", "bf16")])
def test_weights_match_the_plain_form(H, Hkv, D, qtype, cache):
    """Ragged sequences, several rows of one sequence in no order, windows anywhere; what no window
    holds keeps its bits."""
    c = Case([1, 63, 64, 65, 0, 500, 2500], H, Hkv, D, qtype, cache, seed=H + D, capacity=45)
    rows = [(6, 0, 2500), (0, 0, 1), (5, 33, 400), (1, 0, 63), (6, 1000, 2499), (2, 0, 64), (3, 64, 65), (6, 31, 32),
            (4, 0, 0), (5, 399, 500), (3, 3, 3)]
    seq, start, end = (np.array(x) for x in zip(*rows))
    q = c.queries(len(rows))
    acc = torch.rand(7, 64 * 45, generator=c.g)
    acc[:, 2600:] = -0.0
    want, tol, held, lse = expected_weights(c, q, seq, start, end, acc)
    got = run_weights(c, q, lse, seq, start, end, acc)
    assert torch.equal(got[~held].view(torch.int32), acc[~held].view(torch.int32))
    err = (got.double() - want).abs()
    assert (err <= tol)[held].all(), f"{(err / tol)[held].max():.3g} of the bound"
    again = run_weights(c, q, lse, seq, start, end, acc)
    assert torch.equal(got, again)


def test_weights_of_rows_that_do_not_count():
    """Rows with a bad sequence, window or page, and heads whose lse is not finite, add nothing."""
    c = Case([300, 200, 400], 4, 2, 64, "bf16", seed=3)
    rows = [(0, 0, 300), (3, 0, 5), (-1, 0, 5), (0, -1, 5), (0, 9, 5), (0, 0, 64 * 7 + 1), (1, 0, 200), (2, 0, 400)]
    seq, start, end = (np.array(x) for x in zip(*rows))
    q = c.queries(len(rows))
    acc = torch.rand(3, 64 * 7, generator=c.g)
    _, _, _, lse = expected_weights(c, q, seq, start, end, acc, skip=set(range(1, 6)))
    lse[6] = torch.tensor([float("nan"), float("inf"), float("-inf"), float("nan")])
    lse[7, 1] = float("nan")
    k, _ = c.at(2, 0, 400)      # as it was before its page was lost
    c.table[2, 3] = -5
    mqa.mqa_fp4_status()
    got = run_weights(c, q, lse, seq, start, end, acc)
    assert mqa.mqa_fp4_status() == mqa.STATUS_BAD_WINDOW | mqa.STATUS_BAD_PAGE
    want, tol, held, _ = expected_weights(c, q[:1], seq[:1], start[:1], end[:1], acc)
    assert ((got[0].double() - want[0]).abs() <= tol[0] + 1e-300).all()
    assert torch.equal(got[1], acc[1])
    assert torch.equal(got[2, 192:256], acc[2, 192:256])
    row = Row(q[7], k, None, 64 ** -0.5, c.qt)
    w = (row.w * torch.exp(row.lse - torch.where(torch.isnan(lse[7]), row.lse.float(), lse[7]).double())[:, None])
    some = [0, 2, 3]
    at = torch.ones(400, dtype=torch.bool)
    at[192:256] = False
    want2 = acc[2, :400].double() + w[some].sum(0)
    err = (got[2, :400].double() - want2).abs()[at]
    assert (err <= (1.01 * row.w_tol[some].sum(0) + 6 * 2.0 ** -24 * want2)[at]).all()


def test_weights_with_more_sequences_than_one_plan_and_a_wide_pitch():
    n = 1100
    lengths = [int(x) for x in np.random.RandomState(0).randint(0, 130, n)]
    c = Case(lengths, 2, 1, 64, "bf16", seed=7)
    q = c.queries(n)
    order = np.random.RandomState(1).permutation(n)
    end = np.array(lengths)[order]
    pitch = torch.zeros(n, 64 * c.table.shape[1] + 9)
    want, tol, held, lse = expected_weights(c, q, order, np.zeros(n, int), end, pitch)
    d = torch.zeros(n, pitch.shape[1] + 5, device=DEV)[:, 2:-3]
    mqa.mqa_kv_weights_accumulate(q.to(DEV), lse.to(DEV), c.dk, c.table.to(DEV), i32(order), i32(np.zeros(n)), i32(end), d)
    got = d.cpu()
    assert ((got.double() - want).abs() <= tol).all()


def test_weights_of_sequences_far_apart():
    """Few rows among many sequences; the sums of the others keep their bits."""
    n, places = 5000, [4999, 0, 2047, 2048, 1023]
    c = Case([130] * 5, 2, 1, 64, "bf16", seed=9)
    q = c.queries(5)
    small = torch.rand(5, 64 * c.table.shape[1], generator=c.g)
    order, zero, end = np.arange(5), np.zeros(5, int), np.array([130, 64, 1, 129, 100])
    want, tol, _, lse = expected_weights(c, q, order, zero, end, small)
    table = torch.full((n, c.table.shape[1]), -1, dtype=torch.int32)
    table[places] = c.table
    acc = torch.full((n, small.shape[1]), 0.25)
    acc[places] = small
    c.table = table
    mqa.mqa_fp4_status()
    got = run_weights(c, q, lse, places, zero, end, acc)
    assert mqa.mqa_fp4_status() == 0
    assert ((got[places].double() - want).abs() <= tol + 1e-300).all()
    others = torch.ones(n, dtype=torch.bool)
    others[places] = False
    assert (got[others] == 0.25).all()


def test_weights_without_rows_sequences_or_pages():
    c = Case([70], 4, 2, 64, "bf16", seed=10)
    acc = torch.rand(1, 128)
    mqa.mqa_fp4_status()
    assert torch.equal(run_weights(c, c.queries(0), torch.zeros(0, 4), [], [], [], acc), acc)
    q = c.queries(2)
    c.dk = c.dk[:0]
    assert torch.equal(run_weights(c, q, torch.zeros(2, 4), [0, 0], [0, 3], [0, 3], acc), acc)
    assert mqa.mqa_fp4_status() == 0
    assert torch.equal(run_weights(c, q, torch.zeros(2, 4), [0, 0], [0, 0], [0, 1], acc), acc)
    assert mqa.mqa_fp4_status() == mqa.STATUS_BAD_PAGE
    c.table = c.table[:0]
    run_weights(c, q, torch.zeros(2, 4), [0, -1], [0, 0], [0, 0], acc[:0])
    assert mqa.mqa_fp4_status() == mqa.STATUS_BAD_WINDOW


# --- the choice -------------------------------------------------------------------


def run_select(acc, lens, budget, recent, kept_acc=True):
    n = len(lens)
    keep = torch.full((n, budget), 77, dtype=torch.int32, device=DEV)
    kept = torch.full((n,), 77, dtype=torch.int32, device=DEV)
    ka = torch.full((n, budget), 7.0, device=DEV) if kept_acc else None
    d = acc if acc.is_cuda else acc.to(DEV)
    size = mqa.mqa_kv_evict_workspace_bytes(n, acc.shape[1])
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device=DEV)
    mqa.mqa_kv_evict_select(d, i32(lens), budget, recent, keep, kept, ws, kept_acc=ka)
    torch.cuda.synchronize()
    return keep.cpu().numpy(), kept.cpu().numpy(), ka.cpu().numpy() if kept_acc else None


def check_select(acc, lens, budget, recent, keep, kept, kept_acc):
    a = acc.cpu().numpy()
    for s, n in enumerate(lens):
        want = evict_keep(a[s], n, budget, recent)
        m = len(want)
        assert kept[s] == m, s
        assert np.array_equal(keep[s, :m], want), s
        assert (keep[s, m:] == -1).all(), s
        if kept_acc is not None:
            assert np.array_equal(kept_acc[s, :m].view(np.int32), a[s, want].view(np.int32)), s
            assert (kept_acc[s, m:] == 0).all(), s


@pytest.mark.parametrize("budget,recent", [(1, 0), (1, 1), (64, 0), (64, 64), (100, 33), (1000, 10), (5000, 1), (0, 0)])
@pytest.mark.parametrize("values", ["spread", "ties", "special"])
def test_select_matches_the_plain_form(budget, recent, values):
    lens = [0, 1, 2, 63, 64, 65, 99, 100, 101, 1000, 1001, 1024, 1025, 4097, 6000]
    g = torch.Generator().manual_seed(budget + recent)
    acc = torch.exp(3 * torch.randn(len(lens), 6000, generator=g))
    if values == "ties":
        acc = torch.randint(0, 4, acc.shape, generator=g).float() / 4
    if values == "special":
        pick = torch.tensor([float("nan"), float("inf"), float("-inf"), 0.0, -0.0, 1.0, -1.0, 1e-42, -1e-42, 1 + 2 ** -23,
                             float("-nan"), 3.4e38])
        acc = pick[torch.randint(0, len(pick), acc.shape, generator=g)]
    check_select(acc, lens, budget, recent, *run_select(acc, lens, budget, recent))


def test_select_neighbouring_values_and_equal_rows():
    """Sums one step apart, and rows whose sums are all equal."""
    acc = torch.empty(3, 5000)
    acc[0] = torch.from_numpy((np.arange(5000)[np.random.RandomState(0).permutation(5000)] + 0x3F800000).astype(np.int32)
                              .view(np.float32))
    acc[1] = 2.5
    acc[2] = 0.0
    check_select(acc, [5000] * 3, 1234, 77, *run_select(acc, [5000] * 3, 1234, 77))
    keep, kept, _ = run_select(acc, [5000] * 3, 1234, 77, kept_acc=False)
    check_select(acc, [5000] * 3, 1234, 77, keep, kept, None)


@pytest.mark.parametrize("n,length", [(1, 131072), (1, 70001), (3, 200000), (40, 20011), (700, 1500)])
def test_select_long_and_many(n, length):
    g = torch.Generator(device=DEV).manual_seed(n)
    acc = torch.exp(2 * torch.randn(n, length + 3, generator=g, device=DEV))[:, 1:-1]    # a pitch, an odd base
    lens = [length - 7 * (s % 5) for s in range(n)]
    for budget, recent in ((length // 3, length // 20), (length - 100, 0), (5, 2)):
        check_select(acc, lens, budget, recent, *run_select(acc, lens, budget, recent))


def test_select_more_positions_than_chunks_of_one_piece():
    """Above 2,097,152 positions a chunk has several pieces; shorter sequences beside them have not."""
    g = torch.Generator(device=DEV).manual_seed(4)
    lens = [5000001, 2097153, 2097152, 16385, 1, 0]
    acc = torch.exp(2 * torch.randn(len(lens), 5000001, generator=g, device=DEV))
    acc[1] = torch.randint(0, 4, (5000001,), generator=g, device=DEV).float() / 4
    for budget, recent in ((1000003, 77), (2097152, 0), (5, 2)):
        check_select(acc, lens, budget, recent, *run_select(acc, lens, budget, recent))


def test_select_and_compact_without_sequences_positions_or_budget():
    e = torch.empty(0, dtype=torch.int32, device=DEV)
    mqa.mqa_kv_evict_select(torch.empty(0, 5, device=DEV), e, 3, 1, e.view(0, 3), e)
    keep, kept, _ = run_select(torch.empty(2, 0), [0, 0], 3, 1)
    assert (keep == -1).all() and (kept == 0).all()
    table = i32([[0], [1]])
    pool, new = torch.rand(2, 64, device=DEV), torch.zeros(2, 64, device=DEV)
    mqa.mqa_kv_compact(i32(keep), i32(kept), table, table, [(pool, new)])
    mqa.mqa_kv_compact(e.view(0, 3), e, e.view(0, 1), e.view(0, 1), [(pool, new)])
    mqa.mqa_kv_compact(i32(keep)[:, :0].contiguous(), i32(kept), table, table, [(pool, new)])
    mqa.mqa_kv_compact(i32(keep), i32(kept), table, table, [])
    assert (new == 0).all()


def test_select_lengths_that_fail_closed():
    acc = torch.rand(4, 500)
    mqa.mqa_fp4_status()
    keep, kept, ka = run_select(acc, [500, 501, -1, 400], 50, 10)
    assert mqa.mqa_fp4_status() == mqa.STATUS_BAD_WINDOW
    assert kept.tolist() == [50, -1, -1, 50]
    assert (keep[1:3] == -1).all() and (ka[1:3] == 0).all()
    check_select(acc[[0, 3]], [500, 400], 50, 10, keep[[0, 3]], kept[[0, 3]], ka[[0, 3]])


# --- the move ---------------------------------------------------------------------


def test_compact_moves_every_kind_of_array():
    """Keys in three layouts, 8-bit values, codes, scales and one float per position, out of and into one
    shuffled pool; what is behind the last kept position keeps its bits."""
    rng = np.random.RandomState(0)
    n, budget, P = 4, 150, 60
    lens = [700, 150, 40, 0]
    pages = rng.permutation(P)
    src = np.full((n, 11), -1)
    at = 0
    for s, m in enumerate(lens):
        k = (m + 63) // 64
        src[s, :k] = pages[at:at + k]
        at += k
    dst = pages[at:at + 3 * n].reshape(n, 3)
    keep = np.full((n, budget), -1)
    kept = np.array([150, 150, 40, 0])
    for s in range(n):
        keep[s, : kept[s]] = np.sort(rng.choice(lens[s], kept[s], replace=False)) if lens[s] else []
    raw = lambda *shape: torch.from_numpy(rng.randint(0, 256, shape).astype(np.uint8)).to(DEV)
    arrays = [
        raw(P, 64, 2, 256).view(torch.bfloat16),                                    # [P, 64, Hkv, D]
        raw(P, 2, 64, 256).view(torch.bfloat16).transpose(1, 2),                    # heads outside positions
        raw(P, 2, 64, 3, 128).view(torch.float16)[:, 1],                            # half of a pool
        raw(P, 64, 1, 64).view(torch.float8_e4m3fn),
        raw(P, 64, 64), raw(P, 64, 4),                                              # the indexer's codes and scales
        raw(P, 64, 4).view(torch.float32)[:, :, 0],
        raw(P, 64, 36)[:, :, 4:16],                                                 # words, not 16-byte aligned
    ]
    before = [a.clone().cpu() for a in arrays]
    mqa.mqa_fp4_status()
    mqa.mqa_kv_compact(i32(keep), i32(kept), i32(src), i32(dst), [(a, a) for a in arrays])
    assert mqa.mqa_fp4_status() == 0
    as_bytes = lambda t: t.contiguous().view(torch.uint8).reshape(t.shape[0] * 64, -1)
    for b, a in zip(before, arrays):
        want = as_bytes(b).clone()
        old = as_bytes(b)
        for s in range(n):
            for j in range(kept[s]):
                p = keep[s, j]
                want[dst[s, j // 64] * 64 + j % 64] = old[src[s, p // 64] * 64 + p % 64]
        assert torch.equal(as_bytes(a.cpu()), want)


def test_compact_leaves_out_what_it_cannot_place():
    P, n = 12, 4
    a = torch.arange(P * 64, dtype=torch.int32, device=DEV).reshape(P, 64)
    b = torch.full((P, 64), -1, dtype=torch.int32, device=DEV)
    src = np.array([[0, 1], [2, P], [4, 5], [6, -1]])
    dst = np.array([[0], [1], [2], [P]])
    keep = np.array([[0, 64, 128, 5], [1, 70, 3, 4], [0, 1, 2, 3], [0, 1, 2, 3]])
    mqa.mqa_fp4_status()
    mqa.mqa_kv_compact(i32(keep), i32([4, 4, -1, 4]), i32(src), i32(dst), [(a, b)])
    assert mqa.mqa_fp4_status() == mqa.STATUS_BAD_WINDOW | mqa.STATUS_BAD_PAGE
    want = torch.full((P, 64), -1, dtype=torch.int32)
    want[0, :4] = torch.tensor([0, 64, -1, 5])
    want[1, :4] = torch.tensor([129, -1, 131, 132])
    assert torch.equal(b.cpu(), want)
    mqa.mqa_kv_compact(i32(np.zeros((1, 100))), i32([65]), i32([[0]]), i32([[3]]), [(a, b)])     # more than one page holds
    assert mqa.mqa_fp4_status() == mqa.STATUS_BAD_WINDOW
    mqa.mqa_kv_compact(i32(np.zeros((1, 10))), i32([11]), i32([[0]]), i32([[3]]), [(a, b)])      # more than the budget
    assert mqa.mqa_fp4_status() == mqa.STATUS_BAD_WINDOW
    assert torch.equal(b.cpu(), want)


# --- a run of them together --------------------------------------------------------


def test_decode_step_with_selection_and_eviction():
    """Index, select, attend, accumulate, evict, and go on in the smaller cache: key-value pages and the
    indexer's own pages share one block table throughout."""
    from fp4_mqa_scoring_amd import synth
    K, n_seq, H, D = 512, 3, 64, 128
    inp = synth.make_decode_inputs(n_seq, 1, 1500, 2600, K, seed=5, spare_pages=80)
    t = {k: torch.from_numpy(np.ascontiguousarray(getattr(inp, k))).to(DEV)
         for k in ("q", "q_scale", "k_pages", "k_scale", "weights", "block_table", "seq_of_row", "row_start", "row_end")}
    P = t["k_pages"].shape[0]
    g = torch.Generator(device=DEV).manual_seed(1)
    keys = torch.randn(P, 64, 1, D, generator=g, device=DEV).bfloat16()
    values = torch.randn(P, 64, 1, D, generator=g, device=DEV).bfloat16()
    q = (2 * torch.randn(n_seq, H, D, generator=g, device=DEV)).bfloat16()
    acc = torch.zeros(n_seq, 64 * t["block_table"].shape[1], device=DEV)
    lens = inp.row_end.astype(int)
    mqa.mqa_fp4_status()

    def index(table, end):
        raw, slot, count = mqa.alloc_outputs(n_seq, K, DEV)
        ws = torch.empty(mqa.mqa_fp4_decode_workspace_bytes(n_seq, K), dtype=torch.uint8, device=DEV)
        mqa.mqa_fp4_topk_decode(t["q"], t["q_scale"], t["k_pages"], t["k_scale"], t["weights"], table, t["seq_of_row"],
                                t["row_start"], end, K, raw, slot, count, ws)
        return raw, slot, count

    def attend_selected(slot, count):
        out, lse = torch.empty_like(q), torch.empty(n_seq, H, device=DEV)
        ws = torch.empty(mqa.mqa_kv_attention_selected_workspace_bytes(n_seq, K, H, 1, D), dtype=torch.uint8, device=DEV)
        mqa.mqa_kv_attention_selected(q, keys, values, slot, count, out, ws, lse=lse)
        return out, lse

    raw, slot, count = index(t["block_table"], t["row_end"])
    out, lse = attend_selected(slot, count)
    for r in range(n_seq):
        s = slot[r].cpu().long()
        kk, vv = (x.view(P * 64, 1, D)[s.to(DEV)].cpu().float().double() for x in (keys, values))
        row = Row(q[r].cpu(), kk, vv, D ** -0.5, torch.bfloat16)
        assert ((out[r].cpu().double() - row.out).abs() <= row.out_tol).all()

    full, full_lse = torch.empty_like(q), torch.empty(n_seq, H, device=DEV)
    ws = torch.empty(mqa.mqa_kv_attention_decode_workspace_bytes(n_seq, H, 1, D), dtype=torch.uint8, device=DEV)
    mqa.mqa_kv_attention_decode(q, keys, values, t["block_table"], t["seq_of_row"], t["row_start"], t["row_end"], full, ws,
                                lse=full_lse)
    mqa.mqa_kv_weights_accumulate(q, full_lse, keys, t["block_table"], t["seq_of_row"], t["row_start"], t["row_end"], acc)
    total = acc.double().sum(1).cpu()     # every head's weights sum to one
    assert (total - H).abs().max() < 1e-3 * H

    budget, recent = 1000, 64
    keep = torch.empty(n_seq, budget, dtype=torch.int32, device=DEV)
    kept = torch.empty(n_seq, dtype=torch.int32, device=DEV)
    kept_acc = torch.empty(n_seq, budget, device=DEV)
    wsz = mqa.mqa_kv_evict_workspace_bytes(n_seq, acc.shape[1])
    mqa.mqa_kv_evict_select(acc, t["row_end"], budget, recent, keep, kept, torch.empty(wsz, dtype=torch.uint8, device=DEV),
                            kept_acc=kept_acc)
    a = acc.cpu().numpy()
    for s in range(n_seq):
        assert np.array_equal(keep[s].cpu().numpy(), evict_keep(a[s], lens[s], budget, recent))
    used = set(inp.block_table[inp.block_table >= 0].tolist())
    free = [p for p in range(P) if p not in used]
    new_table = i32(np.array(free[: 16 * n_seq]).reshape(n_seq, 16))
    arrays = [keys, values, t["k_pages"], t["k_scale"]]
    mqa.mqa_kv_compact(keep, kept, t["block_table"], new_table, [(x, x) for x in arrays])

    raw2, slot2, count2 = index(new_table, kept)
    full2, ws2 = torch.empty_like(q), ws
    mqa.mqa_kv_attention_decode(q, keys, values, new_table, t["seq_of_row"], t["row_start"], kept, full2, ws2)
    assert mqa.mqa_fp4_status() == 0
    for r in range(n_seq):
        # the same keys in the old pages
        old = inp.block_table[r][keep[r].cpu().numpy() // 64].astype(np.int64) * 64 + keep[r].cpu().numpy() % 64
        o = torch.from_numpy(old).to(DEV)
        kk, vv = (x.view(P * 64, 1, D)[o].cpu().float().double() for x in (keys, values))
        row = Row(q[r].cpu(), kk, vv, D ** -0.5, torch.bfloat16)
        assert ((full2[r].cpu().double() - row.out).abs() <= row.out_tol).all()
        # what the indexer selects among the kept positions, it finds at their new places
        new = raw2[r].cpu().numpy()
        assert np.array_equal(slot2[r].cpu().numpy(), new_table[r].cpu().numpy()[new // 64] * 64 + new % 64)
        before = set(raw[r].cpu().numpy().tolist()) & set(keep[r].cpu().numpy().tolist())
        assert before <= set(keep[r].cpu().numpy()[new].tolist())


@pytest.mark.parametrize("capacity", [64 * 40, 64 * 400])
def test_accumulate_choose_and_move_in_graphs_and_on_streams(capacity):
    """The three calls in one graph, replayed as the lengths and sums change, and at once on two streams."""
    lengths, budget, recent, H = [2500, 700, 64], 333, 20, 8
    c = Case(lengths, H, 2, 64, "bf16", seed=12, capacity=capacity // 64, spare=20)
    q = c.queries(3).to(DEV)
    used = set(c.table[c.table >= 0].tolist())
    free = [p for p in range(c.P) if p not in used]
    new_table = i32(np.array(free[:18]).reshape(3, 6))
    table, seq, zero, end = c.table.to(DEV), i32([0, 1, 2]), i32([0, 0, 0]), i32(lengths)
    size = mqa.mqa_kv_evict_workspace_bytes(3, capacity)
    assert (size > 0) == (capacity > 16384)
    lse = torch.full((3, H), 5.0, device=DEV)

    def outputs():
        return dict(acc=torch.rand(3, capacity, generator=torch.Generator().manual_seed(1)).to(DEV),
                    keep=torch.zeros(3, budget, dtype=torch.int32, device=DEV),
                    kept=torch.zeros(3, dtype=torch.int32, device=DEV), kept_acc=torch.zeros(3, budget, device=DEV),
                    ws=torch.full((size,), 0xFF, dtype=torch.uint8, device=DEV), pool=torch.zeros_like(c.dk))

    def step(o, stream=None):
        mqa.mqa_kv_weights_accumulate(q, lse, c.dk, table, seq, zero, end, o["acc"], stream=stream)
        mqa.mqa_kv_evict_select(o["acc"], end, budget, recent, o["keep"], o["kept"], o["ws"], kept_acc=o["kept_acc"],
                                stream=stream)
        mqa.mqa_kv_compact(o["keep"], o["kept"], table, new_table, [(c.dk, o["pool"])], stream=stream)

    def same(a, b):
        return all(torch.equal(a[k].view(torch.uint8), b[k].view(torch.uint8)) for k in ("acc", "keep", "kept", "kept_acc", "pool"))

    eager = outputs()
    step(eager)
    torch.cuda.synchronize()
    a = eager["acc"].cpu().numpy()
    for s in range(3):
        assert np.array_equal(eager["keep"][s, : eager["kept"][s]].cpu().numpy(), evict_keep(a[s], lengths[s], budget, recent))
    sides = [(torch.cuda.Stream(), outputs()) for _ in range(2)]
    torch.cuda.synchronize()
    for st, o in sides:
        step(o, st)
    torch.cuda.synchronize()
    assert all(same(o, eager) for _, o in sides)

    o = outputs()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(o)
    o["acc"].copy_(outputs()["acc"])
    eager = outputs()
    for i in range(3):
        end.copy_(i32([max(0, n - 200 * i) for n in lengths]))
        q.copy_(c.queries(3))
        graph.replay()
        torch.cuda.synchronize()
        step(eager)
        torch.cuda.synchronize()
        assert same(o, eager), i
