"""Outputs that may take an input's place, on the GPU."""
import numpy as np
import pytest
import torch

import fp4_mqa_scoring_amd as mqa
from kv_ref import evict_keep

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("n,length,capacity", [(300, 3000, 3000), (300, 9000, 16384), (40, 20011, 20011), (6, 131072, 140000),
                                               (1, 2200000, 2200000)])
@pytest.mark.parametrize("captured", [False, True])
def test_kept_in_the_lengths_place(n, length, capacity, captured):
    """One workgroup per sequence, several, and chunks of several pieces; twice over, as the lengths shrink."""
    g = torch.Generator(device=DEV).manual_seed(n + length)
    acc = torch.exp(2 * torch.randn(n, capacity, generator=g, device=DEV))
    host = acc.cpu().numpy()
    lens = torch.tensor([max(0, length - 7 * (s % 5)) for s in range(n)], dtype=torch.int32, device=DEV)
    if n > 5:
        lens[3], lens[4] = -1, capacity + 1
    budget, recent = length // 3, length // 20
    keep = torch.empty(n, budget, dtype=torch.int32, device=DEV)
    ws = torch.full((mqa.mqa_kv_evict_workspace_bytes(n, capacity),), 0xFF, dtype=torch.uint8, device=DEV)
    call = lambda: mqa.mqa_kv_evict_select(acc, lens, budget, recent, keep, lens, ws)
    if captured:
        before = lens.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        lens.copy_(before)
        call = graph.replay
    for _ in range(2):
        old = lens.cpu().numpy().copy()
        call()
        torch.cuda.synchronize()
        new, got = lens.cpu().numpy(), keep.cpu().numpy()
        for s in range(n):
            if not 0 <= old[s] <= capacity:
                assert new[s] == -1 and (got[s] == -1).all(), s
                continue
            want = evict_keep(host[s], old[s], budget, recent)
            assert new[s] == len(want) and np.array_equal(got[s, :new[s]], want) and (got[s, new[s]:] == -1).all(), s
    mqa.mqa_fp4_status()


@pytest.mark.parametrize("H,Hkv,D,qtype", [(8, 2, 128, "bf16"), (64, 1, 128, "bf16"), (40, 1, 256, "fp16"), (130, 1, 64, "fp16")])
@pytest.mark.parametrize("length,rows", [(200, 3), (9000, 2), (300, 700)])
def test_attention_in_its_queries_place(H, Hkv, D, qtype, length, rows):
    """Whole rows, rows that are cut and joined, lists with and without parts: the bits of a call with an output of its own."""
    t = dict(bf16=torch.bfloat16, fp16=torch.float16)[qtype]
    g = torch.Generator(device=DEV).manual_seed(length)
    pages = (length + 63) // 64
    k, v = (torch.randn(pages, 64, Hkv, D, generator=g, device=DEV).to(t) for _ in range(2))
    q = torch.randn(rows, H, D, generator=g, device=DEV).to(t)
    i32 = lambda x: torch.as_tensor(x, dtype=torch.int32).to(DEV)
    table = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)[None]
    seq, start = i32([0] * rows), i32([0] * rows)
    end = i32([0 if r == 1 else length - r % 60 for r in range(rows)])
    slots = torch.randint(0, 64 * pages, (rows, 515), generator=g, device=DEV).to(torch.int32)
    count = i32([0 if r == 1 else 515 - r % 500 for r in range(rows)])
    ws = torch.empty(max(mqa.mqa_kv_attention_decode_workspace_bytes(rows, H, Hkv, D),
                         mqa.mqa_kv_attention_selected_workspace_bytes(rows, 515, H, Hkv, D)), dtype=torch.uint8, device=DEV)
    for call in (lambda x, o: mqa.mqa_kv_attention_decode(x, k, v, table, seq, start, end, o, ws),
                 lambda x, o: mqa.mqa_kv_attention_selected(x, k, v, slots, count, o, ws)):
        want, own = torch.full_like(q, 7.0), q.clone()
        call(q, want)
        call(own, own)
        torch.cuda.synchronize()
        assert torch.isfinite(want.float()).all()
        assert torch.equal(own.view(torch.int16), want.view(torch.int16))
