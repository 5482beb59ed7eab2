"""Inputs and a plain fp64 CPU implementation for the tests of rope_and_cache,
decode_grouped and prefill_grouped, with error bounds derived from the number
formats (u = half a step of the output type, relative: 2^-11 fp16, 2^-8 bf16).

Attention, per output element with weights p_j (summing to 1) and values v_j:
  * a score off by at most d moves every weight by a factor within e^(+-2d), so
    the output by at most 2.1 d sum p|v| for small d.  d collects
      - the fp32 dot product: D additions, each off by at most 2^-23 of the
        running sum's bound: D 2^-23 scale sum_i |q_i k_i| (tensor cores may
        truncate where an fp32 add rounds, which 2^-23 covers);
      - the cap: tanh is taken to a few fp32 steps of 1: cap 2^-20;
      - the bias: slope * distance rounded to fp32 and added: 2^-22 of it;
      - the exponent itself (ex2 to 2^-22) and its argument's rounding, at most
        a few steps of the largest score: 2^-21 max|s|;
  * the products and sums over n keys in fp32: n 2^-23 sum p|v| at most, and
    less in practice; the bound uses (64 + n / 16) 2^-23, since every partial
    sum covers one tile's keys and tiles are joined pairwise or in order;
  * weights in 16 bits (prefill): each off by u relative: u sum p|v|;
    as a 16-bit pair (decode): 2^-16 sum p|v|;
  * the output's rounding: u |o|, and half a subnormal step in fp16.
"""
from __future__ import annotations

import math

import torch

U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 0.0}
BAD_ENTRY = 0x7FFFFFF0


class Case:
    pass


def make_case(seed, ctx, new, q_heads, kv_heads, D, B, dtype, window=0, prefix=None, cap=0.0,
              alibi=False, q_scale=1.0, extra_blocks=3, scale=None):
    """A shuffled pool.  Every key row that no query sees through a used block
    past its context, and every block that is in no table, holds NaN; table
    entries past a context, or of blocks no query sees, are out of range."""
    g = torch.Generator().manual_seed(seed)
    c = Case()
    S = len(ctx)
    need = [-(-n // B) for n in ctx]
    N = sum(need) + extra_blocks
    MB = max(need + [1]) + 1
    c.k_cache = torch.full((N, kv_heads, B, D), float("nan"), dtype=dtype)
    c.v_cache = torch.full((N, kv_heads, B, D), float("nan"), dtype=dtype)
    order = torch.randperm(N, generator=g).tolist()
    c.tables = torch.full((S, MB), BAD_ENTRY, dtype=torch.int32)
    at = 0
    for s in range(S):
        pre = 0 if prefix is None else max(0, min(int(prefix[s]), ctx[s]))
        lo = max(0, ctx[s] - new[s] - window + 1) if window else 0
        for b in range(need[s]):
            blk = order[at]
            at += 1
            first, last = b * B, min((b + 1) * B, ctx[s]) - 1
            if last < lo and first >= pre:      # no query sees a key of it
                c.tables[s, b] = -7
                continue
            c.tables[s, b] = blk
            n = last - first + 1
            c.k_cache[blk, :, :n] = torch.randn(kv_heads, n, D, generator=g).to(dtype)
            c.v_cache[blk, :, :n] = torch.randn(kv_heads, n, D, generator=g).to(dtype)
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    c.q = (torch.randn(starts[-1], q_heads, D, generator=g) * q_scale).to(dtype)
    c.ctx, c.new, c.starts_list = list(ctx), list(new), starts
    c.starts = torch.tensor(starts, dtype=torch.int32)
    c.lens = torch.tensor(ctx, dtype=torch.int32)
    c.scale = D ** -0.5 if scale is None else scale
    c.cap, c.window = cap, window
    c.slopes = (2.0 ** (-8.0 * torch.arange(1, q_heads + 1).float() / q_heads)) if alibi else None
    c.prefix = None if prefix is None else torch.tensor(prefix, dtype=torch.int32)
    c.dtype, c.D, c.B, c.kv_heads, c.q_heads = dtype, D, B, kv_heads, q_heads
    return c


def seen_mask(c, s):
    """[new, ctx] bool: the keys each query of sequence s sees."""
    n, ctx = c.new[s], c.ctx[s]
    p = torch.arange(ctx - n, ctx)[:, None]
    j = torch.arange(ctx)[None]
    seen = j <= p
    if c.window:
        seen &= j > p - c.window
    if c.prefix is not None:
        seen |= j < int(c.prefix[s])
    return seen


def reference(c, weights16):
    """(output, bound), both fp64 [rows, Hq, D]."""
    f = torch.float64
    out = torch.zeros(c.q.shape, dtype=f)
    bound = torch.zeros(c.q.shape, dtype=f)
    G = c.q_heads // c.kv_heads
    u = U[c.dtype]
    for s, ctx in enumerate(c.ctx):
        r0, r1 = c.starts_list[s], c.starts_list[s + 1]
        if ctx == 0 or r0 == r1:
            continue
        seen = seen_mask(c, s)
        used = seen.any(0)
        blk = c.tables[s, torch.arange(ctx) // c.B].long()
        blk = torch.where(used, blk, torch.zeros_like(blk))
        off = torch.arange(ctx) % c.B
        p = torch.arange(ctx - (r1 - r0), ctx)[:, None]
        dist = (p - torch.arange(ctx)[None]).abs().to(f)
        for h in range(c.kv_heads):
            K = c.k_cache[blk, h, off].to(f)
            V = c.v_cache[blk, h, off].to(f)
            K[~used] = 0.0
            V[~used] = 0.0
            for g in range(G):
                hq = h * G + g
                q = c.q[r0:r1, hq].to(f)
                x = q @ K.T * c.scale
                d = c.D * 2.0 ** -23 * abs(c.scale) * (q.abs() @ K.abs().T)
                if c.cap:
                    x = c.cap * torch.tanh(x / c.cap)
                    d = d + c.cap * 2.0 ** -20
                if c.slopes is not None:
                    bias = c.slopes[hq].to(f) * dist
                    x = x - bias
                    d = d + 2.0 ** -22 * bias
                d = d + 2.0 ** -21 * x.abs()
                x = x.masked_fill(~seen, -math.inf)
                w = torch.softmax(x, -1)
                o = w @ V
                mag = w @ V.abs()
                # keys whose weight is below 2^-40 of the largest cannot matter, nor their error
                d = torch.where(x >= x.amax(-1, keepdim=True) - 28.0, d, torch.zeros_like(d))
                n = seen.sum(-1, keepdim=True).to(f)
                rel = 2.1 * d.amax(-1, keepdim=True) + (64 + n / 16) * 2.0 ** -23
                rel = rel + (u if weights16 else 2.0 ** -16)
                out[r0:r1, hq] = o
                bound[r0:r1, hq] = (u * o.abs() + rel * mag) * 1.001 + TINY[c.dtype]
    return out, bound


def rotate(x, cos, sin, interleaved):
    """fp64 rotation of x [T, H, D] by cos, sin [T, r / 2]; also sum |terms|."""
    h = cos.shape[1]
    y, mag = x.clone(), x.abs().clone()
    a = torch.arange(h) * 2 if interleaved else torch.arange(h)
    b = a + 1 if interleaved else a + h
    c, s = cos[:, None], sin[:, None]
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    mag[..., a] = (x[..., a] * c).abs() + (x[..., b] * s).abs()
    mag[..., b] = (x[..., b] * c).abs() + (x[..., a] * s).abs()
    return y, mag


def rope_bound(y, mag, dtype):
    """One rounding to the type, and three fp32 roundings of the two terms."""
    return U[dtype] * y.abs() + 3.1 * 2.0 ** -24 * mag + TINY[dtype]
