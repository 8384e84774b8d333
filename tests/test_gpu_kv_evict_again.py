"""Going on after an eviction: kept sums, new lengths and pages take the next token, its weights and the next
eviction, with a budget that ends inside a page. On the GPU, against the plain forms in 64 bits."""
import numpy as np
import pytest
import torch

import fp4_mqa_scoring_amd as mqa
from kv_ref import Row, assert_row, evict_keep
from test_gpu_kv_attention import DEV, Case, i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H,Hkv,D,qtype", [(8, 2, 64, "bf16"), (40, 1, 128, "fp16")])
@pytest.mark.parametrize("budget,recent", [(333, 20), (200, 0), (65, 64)])
def test_evict_append_accumulate_evict(H, Hkv, D, qtype, budget, recent):
    c = Case([700, 333, 1200, 64, 0], H, Hkv, D, qtype, seed=budget, spare=100)
    n, steps = len(c.lengths), 3
    pages = (budget + 1 + 63) // 64             # the kept positions and one more
    free = [p for p in range(c.P) if p not in set(c.table[c.table >= 0].tolist())]
    tables = [c.table.to(DEV)] + [i32(np.array(free[i * n * pages:(i + 1) * n * pages]).reshape(n, pages)) for i in range(steps)]
    k, v = c.dk, c.dv
    lens, seq, zero = i32(c.lengths), i32(range(n)), i32([0] * n)
    acc = torch.zeros(n, 64 * max(c.table.shape[1], pages), device=DEV)
    keep = torch.empty(n, budget, dtype=torch.int32, device=DEV)
    kept_acc = torch.empty(n, budget, device=DEV)
    ws = torch.empty(mqa.mqa_kv_attention_decode_workspace_bytes(n, H, Hkv, D), dtype=torch.uint8, device=DEV)
    out, lse = torch.empty(n, H, D, dtype=c.qt, device=DEV), torch.empty(n, H, device=DEV)
    mqa.mqa_fp4_status()
    for step in range(steps):
        table = tables[step]
        before, host_lens = acc.cpu().double(), lens.tolist()
        q = c.queries(n)
        dq = q.to(DEV)
        mqa.mqa_kv_attention_decode(dq, k, v, table, seq, zero, lens, out, ws, lse=lse)
        mqa.mqa_kv_weights_accumulate(dq, lse, k, table, seq, zero, lens, acc)
        sums = acc.cpu()
        pool = [x.cpu() for x in (k, v)]
        for s in range(n):
            pos = torch.arange(host_lens[s])
            at = table[s].cpu().long()[pos // 64]
            kk, vv = (x[at, pos % 64].double() for x in pool)
            row = Row(q[s], kk, vv, D ** -0.5, c.qt)
            assert_row(out[s].cpu(), lse[s].cpu(), row, f"step {step}, sequence {s}")
            m = len(pos)
            # the lse of 32 bits that the call was given, off by lse_tol from the exact one
            given = lse[s].cpu().double()
            w = (row.w * torch.exp(row.lse - given)[:, None]).sum(0) if m else torch.zeros(0, dtype=torch.float64)
            want = before[s, :m] + w
            tol = 1.01 * row.w_tol.sum(0) + (H + 2) * 2.0 ** -24 * want
            assert ((sums[s, :m].double() - want).abs() <= tol).all(), (step, s)
            assert (sums[s, m:] == before[s, m:]).all() and (sums[s, m:] == 0).all()
        mqa.mqa_kv_evict_select(acc, lens, budget, recent, keep, lens, kept_acc=kept_acc)      # the new lengths in the old ones' place
        mqa.mqa_kv_compact(keep, lens, table, tables[step + 1], [(k, k), (v, v)])
        new_lens = lens.tolist()
        for s in range(n):
            want = evict_keep(sums[s].numpy(), host_lens[s], budget, recent)
            assert new_lens[s] == len(want) and np.array_equal(keep[s, :new_lens[s]].cpu().numpy(), want)
        # the kept positions' sums are the first ones of the next
        acc.zero_()
        acc[:, :budget] = kept_acc
        for s in range(n):
            assert torch.equal(acc[s, :new_lens[s]].cpu(), sums[s, keep[s, :new_lens[s]].cpu().long()])
        # the next token
        page, at = tables[step + 1].long().gather(1, (lens.long() // 64)[:, None])[:, 0], lens.long() % 64
        for x in (k, v):
            x[page, at] = torch.randn(n, Hkv, D, generator=c.g).to(c.qt).to(DEV)
        lens += 1
    assert mqa.mqa_fp4_status() == 0
