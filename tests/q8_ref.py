"""Inputs and plain fp64 implementations for the tests of the 8-bit cache, with
error bounds derived from the number formats.

Norm and rotation, per element, u24 = 2^-24 the half step of fp32: the sum of D
squares is 16 products in a thread and up to 4 additions across threads, each
addition off by u24 of a sum below the whole: 20 u24; its root's reciprocal is off
by half of that, by 2 u24 from the mean and eps, and by 2 steps (4 u24) of its own;
two products: 2 u24.  18 u24 of the normed value in all, and the rotation adds 3.1
u24 of its two terms.

Numbers in an e4m3 cache: rounding is monotone, so a value known to within e must
be stored as a number between the rounded ends of [value - e, value + e], which is
one number nearly always.
"""
from __future__ import annotations

import torch

from grouped_ref import TINY, U, make_case, rotate

E4M3 = torch.float8_e4m3fn
U24 = 2.0 ** -24


def to_e4m3(x):
    """x (fp64) at the nearest e4m3 number, ties to even, saturated at 448."""
    exponent = torch.frexp(x)[1].clamp(min=-5) - 4
    step = torch.ldexp(torch.ones_like(x), exponent)
    return (torch.round(x / step) * step).clamp(-448.0, 448.0)


def scales_for(seed, heads, lo=0.005, hi=0.03):
    g = torch.Generator().manual_seed(seed)
    return lo + (hi - lo) * torch.rand(heads, generator=g)


def codes(x, scale):
    """The e4m3 tensor of x [.., H, B, D] with a scale per head (dim -3)."""
    return to_e4m3(x.double() / scale.double()[:, None, None]).float().to(E4M3)


def make_q8_case(seed, ctx, new, q_heads, kv_heads, D, B, dtype, **kw):
    """grouped_ref.make_case with its caches as e4m3 numbers (k8, v8 with ks, vs);
    k_cache and v_cache hold the values that these stand for, in 64 bits."""
    c = make_case(seed, ctx, new, q_heads, kv_heads, D, B, dtype, **kw)
    c.ks, c.vs = scales_for(seed, kv_heads), scales_for(seed + 1, kv_heads)
    c.k8, c.v8 = codes(c.k_cache, c.ks), codes(c.v_cache, c.vs)
    refresh(c)
    return c


def refresh(c):
    c.k_cache = c.k8.float().double() * c.ks.double()[:, None, None]
    c.v_cache = c.v8.float().double() * c.vs.double()[:, None, None]


def normed(x, weight, eps):
    """fp64 [T, H, D]."""
    if weight is None:
        return x
    return x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps) * weight.double()


def norm_rotate(x, weight, eps, cos_sin, positions, interleaved):
    """(value, error of the fp32 arithmetic) of x's heads, fp64 [T, H, D]."""
    y = normed(x.double(), weight, eps)
    r = 0.0 if weight is None else 18.0
    if cos_sin is None:
        return y, r * U24 * y.abs()
    h = cos_sin.shape[1] // 2
    cs = cos_sin.double()[positions.clamp(0, cos_sin.shape[0] - 1).long()]
    z, mag = rotate(y, cs[:, :h], cs[:, h:], interleaved)
    return z, (r + 3.1) * U24 * mag


def assert_rows(got, want, err, dtype, what):
    """16-bit rows: one rounding to the type, and err before it."""
    bound = U[dtype] * want.abs() + 1.01 * err + TINY[dtype]
    worst = ((got.double() - want).abs() / bound.clamp(min=1e-300)).max().item() if want.numel() else 0.0
    assert worst <= 1.0, f"{what}: error {worst:.3g} x the bound"


def assert_codes(got, want, err, scale, what):
    """e4m3 rows [T, H, D] of `want` / scale [H]; the division is off by U24."""
    s = scale.double()[:, None]
    e = err + U24 * want.abs()
    lo, hi = to_e4m3((want - e) / s), to_e4m3((want + e) / s)
    g = got.float().double()
    bad = ~((g >= lo) & (g <= hi))
    assert not bad.any(), f"{what}: {int(bad.sum())} numbers outside their bounds"
    # and nearly always there is one number that it can be
    assert (lo != hi).double().mean() <= 1e-3 or want.numel() < 10000
