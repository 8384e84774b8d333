"""Lists over a cache in 4 bits for more rows than one launch's threads can be counted for, on the GPU."""
import pytest
import torch

import fp4_mqa_scoring_amd as mqa
from kv_new_ref import fp4_numbers

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def test_more_rows_than_one_launch_takes():
    """One slot to a row: its output is that slot's values, bit for bit, and the sum's logarithm its score."""
    D, P, rows = 64, 40, (1 << 23) + 4099
    g = torch.Generator().manual_seed(3)
    codes = [torch.randint(0, 256, (P, 64, 1, D // 2), generator=g).to(torch.uint8) for _ in range(2)]
    scales = [torch.randint(124, 129, (P, 64, 1, D // 32), generator=g).to(torch.uint8) for _ in range(2)]
    keys, values = (fp4_numbers(c, s).reshape(P * 64, D) for c, s in zip(codes, scales))
    d = torch.Generator(device=DEV).manual_seed(4)
    q = torch.randn(rows, 1, D, generator=d, device=DEV).to(torch.bfloat16)
    slots = torch.randint(0, 64 * P, (rows, 1), generator=d, device=DEV, dtype=torch.int32)
    count = (torch.rand(rows, generator=d, device=DEV) < 0.9).int()
    out, lse = torch.full_like(q, 7.0), torch.full((rows, 1), 7.0, device=DEV)
    assert mqa.mqa_kv_attention_selected_workspace_bytes(rows, 1, 1, 1, D) == 0
    mqa.mqa_fp4_status()
    mqa.mqa_kv_attention_selected_fp4(q, codes[0].to(DEV), scales[0].to(DEV), codes[1].to(DEV), scales[1].to(DEV), slots, count, out, lse=lse,
                                      scale=0.125)
    torch.cuda.synchronize()
    assert mqa.mqa_fp4_status() == 0
    held = values.to(torch.bfloat16).to(DEV)
    for at in range(0, rows, 1 << 21):
        cut = slice(at, at + (1 << 21))
        want = torch.where(count[cut, None] > 0, held[slots[cut, 0].long()], 0)
        assert torch.equal(out[cut, 0], want), at
        s = q[cut, 0].double() * keys.to(DEV)[slots[cut, 0].long()]
        score = s.sum(-1) * 0.125
        # products are exact, 64 terms are added in 32 bits; then the factor log2(e) / 8, its inverse and the sum's logarithm
        bound = 66 * 2.0 ** -24 * s.abs().sum(-1) * 0.125 + 4 * 2.0 ** -24 * (score.abs() + 1)
        off = (lse[cut, 0].double() - score).abs()
        empty = count[cut] == 0
        assert (off[~empty] <= bound[~empty]).all() and (lse[cut, 0][empty] == float("-inf")).all(), at
