"""Plain 64-bit forms of norm, rotation and what a cache holds in 8 and 4 bits, with the error bounds that the GPU
tests compare against (host tensors; no code shared with the library)."""
import math

import torch

U32 = 2.0 ** -24
E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def turned(x, weight=None, offset=0.0, eps=1e-6, position=None, freq=None, at=0, interleaved=False):
    """(y, tol): rows x [T, H, D] normed and rotated in 64 bits, and how far 32-bit arithmetic may be off before the
    result is rounded.

    Bounds, in units of u = 2^-24.
    - norm: D squares added in 32 bits, in any order, D u relative (each term positive), half of it after the root; the
      mean's factor, eps, root and quotient one rounding each, w + offset one, two products: (D / 2 + 8) u relative.
    - cosine and sine: the angle in turns is rounded to 32 bits once, its fraction is at most 1/2: pi u in radians
      (2 pi * u / 2), and the function itself is good to 4 u; the product in 64 bits loses 2^-51 of the angle.
    - a cos - b sin: two products and a sum, 3 u of (|a| + |b|).
    """
    x = x.double()
    D = x.shape[-1]
    tol = torch.zeros_like(x)
    if weight is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * (weight.double() + offset)
        tol = x.abs() * (D / 2 + 8) * U32
    if freq is None:
        return x, tol
    R = 2 * len(freq)
    angle = position.double()[:, None] * freq.double()[None, :]
    lost = ((math.pi + 4) * U32 + angle.abs() * 2.0 ** -51)[:, None, :]
    c, s = torch.cos(angle)[:, None, :], torch.sin(angle)[:, None, :]
    dims = torch.arange(at, at + R)
    first, second = (dims[0::2], dims[1::2]) if interleaved else (dims[: R // 2], dims[R // 2:])
    a, b, ta, tb = x[..., first], x[..., second], tol[..., first], tol[..., second]
    y, t = x.clone(), tol.clone()
    y[..., first], y[..., second] = a * c - b * s, b * c + a * s
    t[..., first] = t[..., second] = (a.abs() + b.abs()) * (lost + 3 * U32) + ta + tb
    return y, t


def assert_rounded(got, y, tol, where=""):
    """got is y, within tol, rounded once to got's type."""
    info = torch.finfo(got.dtype)
    g = got.double()
    allowed = tol + (y.abs() + tol) * info.eps / 2 + info.smallest_normal * info.eps / 2
    over = y.abs() > info.max
    ok = ((g - y).abs() <= allowed) | (over & torch.isinf(g)) | (torch.isnan(y) & torch.isnan(g)) | (torch.isinf(y) & (g == y))
    assert ok.all(), f"{where}: off by {((g - y).abs() / allowed.clamp(min=1e-300))[~ok].max():.3g} of the bound, {(~ok).sum()} numbers"


def e4m3_of(x, scale):
    """What 8 bits hold of x / scale, the quotient rounded to 32 bits first: saturating, NaN kept."""
    return (x.float() / torch.tensor(scale, dtype=torch.float32)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)


def assert_e4m3(got, y, tol, scale, where=""):
    """got holds y / scale, within tol / scale, rounded once and saturating."""
    want, t = (y / scale).clamp(-448.0, 448.0), tol / scale + (y / scale).abs() * U32
    allowed = t + ((want.abs() + t) * 2.0 ** -4).clamp(min=2.0 ** -10)
    assert ((got.float().double() - want).abs() <= allowed).all(), where


def fp4_of(x):
    """(codes as values, scale bytes) of x [..., D] by the OCP rule, in 64 bits."""
    b = x.double().unflatten(-1, (-1, 32))
    top = b.abs().amax(-1)
    bad = ~torch.isfinite(b).all(-1)
    e = torch.frexp(torch.where(bad, torch.ones_like(top), top)).exponent.long() - 1
    byte = torch.where(top > 0, (e - 2 + 127).clamp(0, 254), torch.zeros_like(e))
    t = torch.where(bad[..., None], torch.zeros_like(b), b) * torch.exp2(127.0 - byte.double())[..., None]
    gap = (t.abs()[..., None] - E2M1).abs() + torch.arange(8) % 2 * 1e-13    # ties to the even code
    value = torch.copysign(E2M1[gap.argmin(-1)], t)
    return value.flatten(-2), torch.where(bad, torch.full_like(byte, 255), byte).to(torch.uint8)


def fp4_values(codes):
    """Values [..., D] that codes [..., D / 2] stand for, unscaled."""
    both = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()
    return torch.cat([E2M1, -E2M1])[both]


def fp4_numbers(codes, scales):
    s = torch.exp2(scales.double() - 127)
    s = torch.where(scales == 255, torch.full_like(s, math.nan), s)
    return (fp4_values(codes).unflatten(-1, (-1, 32)) * s[..., None]).flatten(-2)


def assert_fp4(codes, scales, y, tol, where=""):
    """codes and scales hold y, within tol: a scale of a maximum in the bounds, and the nearest number under it."""
    b, t = y.unflatten(-1, (-1, 32)), tol.unflatten(-1, (-1, 32))
    byte = lambda top: torch.where(top > 0, (torch.frexp(top).exponent.long() + 124).clamp(0, 254), torch.zeros_like(top).long())  # noqa: E731
    lo, hi = byte((b.abs() - t).clamp(min=0).amax(-1)), byte((b.abs() + t).amax(-1))
    got = scales.long()
    assert ((got >= lo) & (got <= hi)).all(), where
    s = torch.exp2(got.double() - 127)[..., None]
    v = fp4_values(codes).unflatten(-1, (-1, 32)) * s
    top = (b.abs() + t) / s
    half = torch.where(top <= 2, 0.25, torch.where(top <= 4, 0.5, 1.0)) * s
    want = torch.minimum(b.abs(), 6 * s) * torch.sign(b)
    assert ((v - want).abs() <= half + t).all(), where
