"""Caches and paged arrays whose strides of one head, page or piece are arbitrary, on the GPU: the bits of
contiguous ones."""
import pytest
import torch

import fp4_mqa_scoring_amd as mqa

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def i32(x):
    return torch.as_tensor(x, dtype=torch.int32).to(DEV)


@pytest.mark.parametrize("H", [4, 40])
@pytest.mark.parametrize("kind", ["one head", "one page"])
def test_attention_and_weights(H, kind):
    g = torch.Generator(device=DEV).manual_seed(H)
    P, Hkv, D = (3, 1, 128) if kind == "one head" else (1, 2, 64)
    k, v = (torch.randn(P, 64, Hkv, D, generator=g, device=DEV).bfloat16() for _ in range(2))

    def odd(t):
        if kind == "one head":
            x = torch.empty(P, 64, D, 1, dtype=t.dtype, device=DEV).transpose(2, 3)
        else:
            x = torch.empty(2, 64 * Hkv * D + 4, dtype=t.dtype, device=DEV)[:1, :64 * Hkv * D].unflatten(1, (64, Hkv, D))
        return x.copy_(t)

    n = 64 * P - 7
    q = torch.randn(2, H, D, generator=g, device=DEV).bfloat16()
    table, seq, start, end = i32([list(range(P))]), i32([0, 0]), i32([0, 5]), i32([n, n - 3])
    slots, count = i32([list(range(n))] * 2), i32([n, 40])
    ws = torch.empty(mqa.mqa_kv_attention_decode_workspace_bytes(2, H, Hkv, D), dtype=torch.uint8, device=DEV)
    ws2 = torch.empty(mqa.mqa_kv_attention_selected_workspace_bytes(2, n, H, Hkv, D), dtype=torch.uint8, device=DEV)
    got = []
    for kk, vv in ((k, v), (odd(k), odd(v)), (k, odd(v))):
        out, sel, lse = torch.empty_like(q), torch.empty_like(q), torch.empty(2, H, device=DEV)
        acc = torch.zeros(1, 64 * P, device=DEV)
        mqa.mqa_kv_attention_decode(q, kk, vv, table, seq, start, end, out, ws, lse=lse)
        mqa.mqa_kv_attention_selected(q, kk, vv, slots, count, sel, ws2)
        mqa.mqa_kv_weights_accumulate(q, lse, kk, table, seq, start, end, acc)
        torch.cuda.synchronize()
        assert torch.isfinite(out.float()).all() and torch.isfinite(sel.float()).all() and acc.sum() > H
        got.append((out.view(torch.int16), sel.view(torch.int16), lse.view(torch.int32), acc.view(torch.int32)))
    for x in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(x, got[0]))


def test_moves():
    src = torch.arange(64 * 8, dtype=torch.int32, device=DEV).to(torch.uint8).reshape(1, 64, 8)
    keep, kept, page = i32([[1, 3, 63, -1]]), i32([3]), i32([[0]])
    for odd in (lambda t: torch.empty(2, 513, dtype=torch.uint8, device=DEV)[:1, :512].unflatten(1, (64, 8)).copy_(t),
                lambda t: torch.empty(1, 64, 8, 1, dtype=torch.uint8, device=DEV).transpose(2, 3).copy_(t.unsqueeze(2))):
        a, b = odd(src), odd(torch.zeros_like(src))
        mqa.mqa_kv_compact(keep, kept, page, page, [(a, b)])
        got = b.reshape(64, 8)
        assert torch.equal(got[:3], src[0, [1, 3, 63]]) and (got[3:] == 0).all()


def test_moves_of_pools_of_different_sizes():
    """A page that the smallest pool lacks is in none: what maps there is left out of every array."""
    small, large = torch.rand(3, 64, device=DEV), torch.rand(5, 64, 2, device=DEV)
    to = torch.zeros(4, 64, device=DEV), torch.zeros(6, 64, 2, device=DEV)
    keep, kept = i32([[0, 64], [0, 1]]), i32([2, 2])
    mqa.mqa_fp4_status()
    mqa.mqa_kv_compact(keep, kept, i32([[1, 4], [2, 0]]), i32([[3], [4]]), [(small, to[0]), (large, to[1])])
    assert mqa.mqa_fp4_status() == mqa.STATUS_BAD_PAGE
    want = torch.zeros_like(to[0]), torch.zeros_like(to[1])
    want[0][3, 0], want[1][3, 0] = small[1, 0], large[1, 0]
    assert torch.equal(to[0], want[0]) and torch.equal(to[1], want[1])
