"""Attention whose weight lies on one position while many others share the rest: each of their weights is
below fp16's normal range, their sum is not. Many rows, so that one wave meets the large weight and many of the
small ones under one running maximum. On the GPU, against the plain form in 64 bits."""
import numpy as np
import pytest
import torch

from kv_ref import Row, half_step
from test_gpu_kv_attention import DEV, Case, run_decode, run_selected

pytestmark = pytest.mark.gpu


def bound(row, k, v, D, t):
    """kv_ref's bound without its allowance for weights below the type's normal range: half a step of
    fp16's smallest number per value, a weight of 1 being the largest. The kernels keep the largest at 2^7 at
    least, so that this step is 2^-32 of it; the sum of the weights is at least the largest."""
    vv = v.double().repeat_interleave(row.out.shape[0] // v.shape[1], 1)
    tiny = torch.finfo(t).smallest_normal * torch.finfo(t).eps / 2
    return row.out_tol - vv.abs().sum(0) * tiny * (1 - 2.0 ** -7)


def check(out, lse, row, tol):
    err = (out.double() - row.out).abs()
    assert (err <= tol).all(), f"{(err / tol).max():.3g} of the bound, {(err / row.out.abs()).max():.3g} of the value"
    assert ((lse.double() - row.lse).abs() <= row.lse_tol).all()


# the first position's score above the others', in steps of log 2
@pytest.mark.parametrize("above", [12.0, 17.5, 23.4, 24.7, 26.0])
@pytest.mark.parametrize("H,Hkv,D,qtype,cache", [
    (4, 1, 64, "fp16", "fp16"), (64, 1, 64, "fp16", "fp16"), (2, 1, 128, "fp16", "e4m3"), (40, 2, 128, "fp16", "e4m3"),
    (3, 1, 256, "fp16", "fp16"), (24, 1, 256, "fp16", "fp16"), (4, 1, 64, "bf16", "bf16"), (64, 1, 64, "bf16", "bf16")])
def test_many_small_weights_beside_one_large(H, Hkv, D, qtype, cache, above):
    n, sink, rows = 4096, 7, 600
    c = Case([n], H, Hkv, D, qtype, cache, seed=int(10 * above) + H)
    g = torch.Generator().manual_seed(H + D)
    pos = torch.arange(n)
    page, at = c.table[0].long()[pos // 64], pos % 64
    raw = torch.uint8 if c.e4m3 else torch.int16
    # keys: the first dim alone carries the score; values: nothing at the large one, near one elsewhere
    keys = torch.zeros(n, Hkv, D)
    keys[:, :, 0] = (torch.rand(n, Hkv, generator=g) < 0.5).float() * 0.5
    keys[sink, :, 0] = 8.0
    values = 0.5 + torch.rand(n, Hkv, D, generator=g)
    values[sink] = 0.0
    for t, x, s in ((c.k, keys, c.k_scale), (c.v, values, c.v_scale)):
        t.view(raw)[page, at] = (x / s).to(c.ct).view(raw)
    c.dk, c.dv = c.k.to(DEV), c.v.to(DEV)
    q = torch.zeros(rows, H, D, dtype=c.qt)
    q[:, :, 0] = above * np.log(2.0) / 8.0 * D ** 0.5 * torch.linspace(0.9, 1.0, H)
    k, v = c.at(0, 0, n)
    row = Row(q[0], k, v, D ** -0.5, c.qt)
    tol = bound(row, k, v, D, c.qt)
    out, lse = run_decode(c, q, [0] * rows, [0] * rows, [n] * rows)
    for r in (0, 301, 599):
        check(out[r], lse[r], row, tol)
    slots = (page * 64 + at).expand(rows, n).numpy()
    out, lse = run_selected(c, q, slots, [n] * rows)
    for r in (0, 301, 599):
        check(out[r], lse[r], row, tol)
