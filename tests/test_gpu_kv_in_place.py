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
