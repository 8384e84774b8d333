"""Plain 64-bit forms of the key-value cache operators, with the error bounds that
the GPU tests compare against (host tensors; no code shared with the library)."""
import math

import numpy as np
import torch


def half_step(dtype):
    """Largest relative error of one rounding to dtype."""
    return torch.finfo(dtype).eps / 2


class Row:
    """Attention of one row: q [H, D], keys and values [n, Hkv, D] (already the
    numbers that the cache stands for, in 64 bits), score factor c.

    Bounds. Unit roundoff of 32 bits u32 = 2^-24, of the query's type u.
    - score: a sum of D products, each exact in 32 bits (two 11-bit significands),
      added in 32 bits, with at most 2 u32 per addition (the matrix unit may
      truncate): 2 D u32 sum|q k|. The factor c log2(e) carries two roundings and
      the multiplication one more: 3 u32 |s|, and the maximum's product and
      the difference to it two of |m|: es = c 2 D u32 max sum|q k| + 8 u32 (max |s| + 1).
    - weight relative to its exact value: es, plus the exponential's 2 u32 and 2^-126
      below which it is flushed to zero.
    - its rounding to the query's type: u relative, or half of the type's
      smallest subnormal, absolute, where the weight is below the type's
      normal range; the weights are relative to a maximum of 1 whose sum is at least 1.
    - sums over n positions in 32 bits: n terms in any order, (n + 8) u32 of the
      sum of the magnitudes (twice: numerator and denominator).
    - the output's rounding: u |out|, or half a subnormal step.
    """

    def __init__(self, q, k, v, c, out_dtype):
        q, k = q.double(), k.double()
        H, n, hkv = q.shape[0], k.shape[0], k.shape[1]
        g = H // hkv
        u32, u = 2.0 ** -24, half_step(out_dtype)
        tiny = torch.finfo(out_dtype).smallest_normal * torch.finfo(out_dtype).eps / 2
        D = q.shape[1]
        if n == 0:
            self.out = torch.zeros(H, D, dtype=torch.float64)
            self.lse = torch.full((H,), -math.inf, dtype=torch.float64)
            self.out_tol = torch.zeros_like(self.out)
            self.lse_tol = torch.zeros_like(self.lse)
            self.w = torch.zeros(H, 0, dtype=torch.float64)
            self.w_tol = torch.zeros(H, 0, dtype=torch.float64)
            return
        kk = k.repeat_interleave(g, 1)
        s = torch.einsum("hd,nhd->hn", q, kk) * c
        mag = torch.einsum("hd,nhd->hn", q.abs(), kk.abs()).amax(1) * abs(c)
        es = 2 * D * u32 * mag + 8 * u32 * (s.abs().amax(1) + 1)
        self.lse = torch.logsumexp(s, 1)
        p = torch.exp(s - self.lse[:, None])
        sum_err = (n + 8) * u32
        self.lse_tol = es + sum_err + 4 * u32 * (self.lse.abs() + 1)
        self.w = p
        # weights against a given (exact) lse: the score's error and the difference's and exponential's
        self.w_tol = p * (es[:, None] + 8 * u32 * ((s - self.lse[:, None]).abs() + 2)) + 2.0 ** -120
        if v is None:
            return
        vv = v.double().repeat_interleave(g, 1)
        self.out = torch.einsum("hn,nhd->hd", p, vv)
        a = torch.einsum("hn,nhd->hd", p, vv.abs())
        self.out_tol = (a * (u + 2 * es[:, None] + 2 * sum_err + 8 * u32) + u * self.out.abs()
                        + vv.abs().sum(0) * (tiny + 2.0 ** -126) + tiny)


def assert_row(got_out, got_lse, row, where=""):
    out = got_out.double()
    err = (out - row.out).abs()
    assert torch.isfinite(out).all(), f"{where}: out is not finite"
    bad = err > row.out_tol
    assert not bad.any(), f"{where}: out off by {err[bad].max():.3g}, {(err / row.out_tol.clamp(min=1e-300)).max():.3g} of its bound"
    if got_lse is not None:
        lse = got_lse.double()
        both_inf = torch.isinf(row.lse) & (lse == row.lse)
        ok = both_inf | ((lse - row.lse).abs() <= row.lse_tol)
        assert ok.all(), f"{where}: lse {lse[~ok]} instead of {row.lse[~ok]}"


def total_order(values):
    """Positions of a float32 array in the total order: value descending, position
    ascending; NaN below every number, +0 above -0."""
    v = np.asarray(values, np.float32)
    nan = np.isnan(v)
    key = np.where(nan, -np.inf, v).astype(np.float64)
    zero = np.where((v == 0) & ~np.signbit(v), 1, 0)
    return np.lexsort((np.arange(len(v)), -zero, -key, nan))


def evict_keep(acc, length, budget, recent):
    """Rising positions that a budget keeps."""
    if length <= budget:
        return np.arange(length)
    old = length - recent
    best = total_order(acc[:old])[: budget - recent]
    return np.sort(np.concatenate([best, np.arange(old, length)])).astype(np.int64)
