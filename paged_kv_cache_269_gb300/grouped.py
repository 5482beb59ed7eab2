"""Rotary cache appends and grouped-query attention over the paged cache.

The binding of pa_rope_and_cache, pa_decode_grouped and pa_prefill_grouped:
query heads that share K/V heads (num_q_heads a multiple of the cache's
heads), rotary positions, and scores that may be capped by a tanh, get a bias
by distance (ALiBi) and be limited to a window and a prefix.  Like the rest of
the package it only marshals arguments.

Workspaces and counters are cached per (device, stream).  Inside a CUDA graph
capture they come from the graph's own memory pool instead (and the counters
are zeroed by the graph), so graphs never share them with each other or with
eager calls.  Buffers that the caller passes are used as they are, and must not
be used by two calls at once.
"""
from __future__ import annotations

import ctypes


class AttnOpts(ctypes.Structure):
    _fields_ = [("softcap", ctypes.c_float), ("window", ctypes.c_int32),
                ("alibi_slopes", ctypes.c_void_p), ("prefix_lens", ctypes.c_void_p)]


def declare(l, dims_p):
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    op = ctypes.POINTER(AttnOpts)
    l.pa_rope_and_cache.argtypes = [vp] * 9 + [i32, i32, i64, i64, i64, i64, i32, i32, i32, dims_p,
                                               vp]
    l.pa_decode_grouped.argtypes = [vp] * 6 + [ctypes.c_float, i32, dims_p, i32, op, vp, sz, vp, sz,
                                               vp]
    l.pa_prefill_grouped.argtypes = [vp] * 7 + [i32, i32, ctypes.c_float, i32, dims_p, i32, op, vp,
                                                sz, vp, sz, vp]
    for name in ("pa_rope_and_cache", "pa_decode_grouped", "pa_prefill_grouped"):
        getattr(l, name).restype = ctypes.c_int
    l.pa_decode_grouped_workspace_bytes.argtypes = [dims_p, i32]
    l.pa_decode_grouped_counters_bytes.argtypes = [dims_p, i32]
    l.pa_prefill_grouped_workspace_bytes.argtypes = [dims_p, i32, i32]
    l.pa_prefill_grouped_counters_bytes.argtypes = [dims_p, i32]
    for name in ("pa_decode_grouped_workspace_bytes", "pa_decode_grouped_counters_bytes",
                 "pa_prefill_grouped_workspace_bytes", "pa_prefill_grouped_counters_bytes"):
        getattr(l, name).restype = sz


def _pa():
    import paged_kv_cache_269_gb300 as pa
    return pa


def rope_table(max_positions, rotary_dim, base=10000.0, inv_freq=None, device=None):
    """The fp32 [max_positions, rotary_dim] table rope_and_cache takes: row p
    holds cos(p f_i), then sin(p f_i), i < rotary_dim / 2, with
    f_i = base^(-2 i / rotary_dim) or the given inv_freq [rotary_dim / 2].
    Angles are taken in 64 bits, so far positions keep their phase.  Made once,
    when a model is loaded."""
    import torch
    if rotary_dim <= 0 or rotary_dim % 2:
        raise ValueError("rotary_dim must be even and positive")
    half = rotary_dim // 2
    if inv_freq is None:
        i = torch.arange(half, dtype=torch.float64, device=device)
        inv_freq = float(base) ** (-2.0 * i / rotary_dim)
    inv_freq = torch.as_tensor(inv_freq, device=device).to(torch.float64)
    if inv_freq.shape != (half,):
        raise ValueError("inv_freq must have rotary_dim / 2 entries")
    angle = torch.arange(max_positions, dtype=torch.float64, device=inv_freq.device)[:, None] * inv_freq
    return torch.cat([angle.cos(), angle.sin()], 1).to(torch.float32).contiguous()


def _rows(t, name, dtype, device, heads, dim):
    """Checks a [T, heads, dim] tensor whose rows may be apart (a slice of a
    packed projection); returns the elements between one row and the next."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 3 or t.shape[2] != dim or (heads is not None and t.shape[1] != heads):
        raise ValueError(f"{name} must have shape [T, {'H' if heads is None else heads}, {dim}], "
                         f"got {tuple(t.shape)}")
    if not t.is_cuda or t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.stride(2) != 1 or (t.shape[1] > 1 and t.stride(1) != dim):
        raise ValueError(f"{name}: the heads of a row must be adjacent and contiguous")
    stride = t.stride(0) if t.shape[0] > 1 else t.shape[1] * dim
    if stride % 8:
        raise ValueError(f"{name}: rows must start on 16-byte boundaries")
    return stride


def rope_and_cache(q_out, q, k, v, k_cache, v_cache, positions, cos_sin, slot_mapping,
                   interleaved=False, stream=None):
    """Rotate q and k by their tokens' positions, write q to q_out and append k
    and v to the caches at slot_mapping (pa_rope_and_cache).

    q, q_out [T, Hq, D] and k, v [T, H, D] may be slices of a packed projection
    (rows apart, heads of a row adjacent); q_out may be q itself.  k_cache,
    v_cache [N, H, B, D]; positions, slot_mapping int32 [T]; cos_sin float32
    [max_positions, rotary_dim] as rope_table makes it, rotary_dim a multiple
    of 16 up to D.  interleaved pairs dims (2 i, 2 i + 1) instead of
    (i, i + rotary_dim / 2).  slot < 0 skips the token's k and v, a negative
    position the whole token."""
    import torch
    pa = _pa()
    pa._element_dtype(k_cache)
    et = k_cache.dtype
    pa._need(k_cache, "k_cache", et, 4)
    dev = k_cache.device
    pa._need(v_cache, "v_cache", et, 4, dev)
    N, H, B, D = k_cache.shape
    if v_cache.shape != k_cache.shape:
        raise ValueError("rope_and_cache: inconsistent cache shapes")
    qs = _rows(q, "q", et, dev, None, D)
    Hq, T = q.shape[1], q.shape[0]
    os_ = _rows(q_out, "q_out", et, dev, Hq, D)
    ks, vs = _rows(k, "k", et, dev, H, D), _rows(v, "v", et, dev, H, D)
    pa._need(positions, "positions", torch.int32, 1, dev)
    pa._need(slot_mapping, "slot_mapping", torch.int32, 1, dev)
    pa._need(cos_sin, "cos_sin", torch.float32, 2, dev)
    if any(t.shape[0] != T for t in (q_out, k, v, positions, slot_mapping)):
        raise ValueError("rope_and_cache: inconsistent numbers of tokens")
    if T > 1 and os_ < Hq * D:
        raise ValueError("q_out: rows overlap")
    if T:
        _refuse_overlap(q_out, os_, q, qs, "q", T, D, same_ok=True)
        _refuse_overlap(q_out, os_, k, ks, "k", T, D)
        _refuse_overlap(q_out, os_, v, vs, "v", T, D)
    dims = pa._cache_dims(k_cache)
    sh, _ = pa._stream_handle(dev, stream)
    with torch.cuda.device(dev):
        rc = pa.lib().pa_rope_and_cache(
            pa._ptr(q_out), pa._ptr(q), pa._ptr(k), pa._ptr(v), pa._ptr(k_cache), pa._ptr(v_cache),
            pa._ptr(positions), pa._ptr(cos_sin), pa._ptr(slot_mapping), T, Hq, qs, ks, vs, os_,
            cos_sin.shape[1], cos_sin.shape[0], 1 if interleaved else 0, ctypes.byref(dims), sh)
    pa._check(rc, "pa_rope_and_cache")
    return q_out


def _refuse_overlap(out, out_stride, x, x_stride, name, T, D, same_ok=False):
    """Refuses an input that shares elements with q_out (q itself excepted).
    Slices of one packed tensor that interleave without sharing are fine."""
    size = 2
    a0, a_row = out.data_ptr(), out.shape[1] * D * size
    b0, b_row = x.data_ptr(), x.shape[1] * D * size
    if same_ok and a0 == b0 and (out_stride == x_stride or T == 1):
        return
    a1, b1 = a0 + (T - 1) * out_stride * size + a_row, b0 + (T - 1) * x_stride * size + b_row
    if a1 <= b0 or b1 <= a0:
        return
    if out_stride == x_stride and T > 1:
        # rows of one stride: apart iff the offset leaves room on both sides
        off = (b0 - a0) % (out_stride * size)
        if off >= a_row and off + b_row <= out_stride * size:
            return
    raise ValueError(f"q_out overlaps {name}")


# Per (device, stream): zeroed counters, which every successful call leaves
# zeroed, and a workspace; both grow on demand.
_buffers: dict = {}


def _buffers_for(device, stream, counters_bytes, workspace_bytes):
    import torch
    pa = _pa()
    with torch.cuda.stream(stream):
        if torch.cuda.is_current_stream_capturing():
            return (torch.zeros(counters_bytes // 4, dtype=torch.int32, device=device),
                    torch.empty(max(workspace_bytes, 16), dtype=torch.uint8, device=device))
        key = (device.index, stream.cuda_stream)
        with pa._buf_lock:
            ctr, ws = _buffers.get(key, (None, None))
            if ctr is None or ctr.numel() * 4 < counters_bytes:
                ctr = torch.zeros(max(counters_bytes, 1 << 14) // 4, dtype=torch.int32, device=device)
            if ws is None or ws.numel() < workspace_bytes:
                ws = torch.empty(max(workspace_bytes, 16), dtype=torch.uint8, device=device)
            _buffers[key] = (ctr, ws)
            return ctr, ws


def reset_counters():
    """Zero every cached counter buffer (needed after a device error)."""
    with _pa()._buf_lock:
        for ctr, _ in _buffers.values():
            ctr.zero_()


def _attention_args(what, out, q, k_cache, v_cache, block_tables, context_lens, softcap,
                    alibi_slopes, window, prefix_lens):
    import torch
    pa = _pa()
    pa._element_dtype(k_cache)
    et = k_cache.dtype
    pa._need(k_cache, "k_cache", et, 4)
    dev = k_cache.device
    pa._need(v_cache, "v_cache", et, 4, dev)
    pa._need(q, "q", et, 3, dev)
    pa._need(out, "out", et, 3, dev)
    pa._need(block_tables, "block_tables", torch.int32, 2, dev)
    pa._need(context_lens, "context_lens", torch.int32, 1, dev)
    S, Hq = context_lens.shape[0], q.shape[1]
    H, D = k_cache.shape[1], k_cache.shape[3]
    if v_cache.shape != k_cache.shape or out.shape != q.shape or q.shape[2] != D \
            or block_tables.shape[0] != S:
        raise ValueError(f"{what}: inconsistent shapes")
    if H == 0 or Hq == 0 or Hq % H:
        raise ValueError(f"{what}: query heads must be a multiple of the cache's heads")
    if alibi_slopes is not None:
        pa._need(alibi_slopes, "alibi_slopes", torch.float32, 1, dev)
        if alibi_slopes.shape[0] != Hq:
            raise ValueError(f"{what}: alibi_slopes must have one entry per query head")
    if prefix_lens is not None:
        pa._need(prefix_lens, "prefix_lens", torch.int32, 1, dev)
        if prefix_lens.shape[0] != S:
            raise ValueError(f"{what}: prefix_lens must have one entry per sequence")
    opts = AttnOpts(float(softcap or 0.0), int(window or 0),
                    None if alibi_slopes is None else alibi_slopes.data_ptr(),
                    None if prefix_lens is None else prefix_lens.data_ptr())
    return dev, S, Hq, pa._cache_dims(k_cache, S), opts


def _pick_buffers(dev, st, need_ctr, need_ws, counters, workspace):
    import torch
    pa = _pa()
    if counters is None or (workspace is None and need_ws):
        c2, w2 = _buffers_for(dev, st, need_ctr, need_ws)
        counters = c2 if counters is None else counters
        workspace = w2 if workspace is None else workspace
    pa._need(counters, "counters", torch.int32, 1, dev)
    if workspace is not None:
        pa._need(workspace, "workspace", torch.uint8, 1, dev)
    ws_ptr = pa._ptr(workspace) if workspace is not None else ctypes.c_void_p(0)
    return counters, workspace, ws_ptr, workspace.numel() if workspace is not None else 0


def decode_grouped_workspace_bytes(num_q_heads, num_kv_heads, head_dim, block_size) -> int:
    """Bytes of workspace decode_grouped needs, for any batch."""
    pa = _pa()
    dims = pa.Dims(0, num_kv_heads, head_dim, block_size, 1)
    n = pa.lib().pa_decode_grouped_workspace_bytes(ctypes.byref(dims), num_q_heads)
    if n == pa._SIZE_ERROR:
        raise pa.PaError(-2, "pa_decode_grouped_workspace_bytes: invalid sizes")
    return n


def decode_grouped_counters_bytes(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size) -> int:
    """Bytes of the (zeroed, reusable) counters decode_grouped needs."""
    pa = _pa()
    dims = pa.Dims(num_seqs, num_kv_heads, head_dim, block_size, 1)
    n = pa.lib().pa_decode_grouped_counters_bytes(ctypes.byref(dims), num_q_heads)
    if n == 0:
        raise pa.PaError(-2, "pa_decode_grouped_counters_bytes: invalid sizes")
    return n


def prefill_grouped_workspace_bytes(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                                    max_query_len) -> int:
    """Bytes of workspace prefill_grouped needs (0: none)."""
    pa = _pa()
    dims = pa.Dims(num_seqs, num_kv_heads, head_dim, block_size, 1)
    n = pa.lib().pa_prefill_grouped_workspace_bytes(ctypes.byref(dims), num_q_heads, max_query_len)
    if n == pa._SIZE_ERROR:
        raise pa.PaError(-2, "pa_prefill_grouped_workspace_bytes: invalid sizes")
    return n


def prefill_grouped_counters_bytes(num_q_heads, num_kv_heads, head_dim, block_size) -> int:
    """Bytes of the (zeroed, reusable) counters prefill_grouped needs."""
    pa = _pa()
    dims = pa.Dims(0, num_kv_heads, head_dim, block_size, 1)
    n = pa.lib().pa_prefill_grouped_counters_bytes(ctypes.byref(dims), num_q_heads)
    if n == 0:
        raise pa.PaError(-2, "pa_prefill_grouped_counters_bytes: invalid sizes")
    return n


def decode_grouped(out, q, k_cache, v_cache, block_tables, context_lens, scale, softcap=0.0,
                   alibi_slopes=None, window=0, prefix_lens=None, workspace=None, counters=None,
                   stream=None):
    """Attention of one new token per sequence over its paged history, with
    query heads that share K/V heads (pa_decode_grouped).

    q, out [S, Hq, D]; k_cache, v_cache [N, H, B, D] with Hq a multiple of H;
    block_tables [S, MB] int32; context_lens [S] int32.  softcap > 0 caps the
    scores (softcap * tanh(s / softcap)); alibi_slopes [Hq] float32 subtracts
    slope * distance; window > 0 sees only the last `window` keys, the token's
    own among them, and the first prefix_lens[s] (int32 [S]).  workspace
    (uint8) and counters (zeroed int32): see the _bytes functions; by default
    cached per stream, or taken from the graph's pool inside a capture."""
    import torch
    pa = _pa()
    dev, S, Hq, dims, opts = _attention_args("decode_grouped", out, q, k_cache, v_cache,
                                             block_tables, context_lens, softcap, alibi_slopes,
                                             window, prefix_lens)
    if q.shape[0] != S:
        raise ValueError("decode_grouped: inconsistent shapes")
    sh, st = pa._stream_handle(dev, stream)
    l = pa.lib()
    with torch.cuda.device(dev):
        need_ws = l.pa_decode_grouped_workspace_bytes(ctypes.byref(dims), Hq)
        need_ctr = l.pa_decode_grouped_counters_bytes(ctypes.byref(dims), Hq)
        if need_ws == pa._SIZE_ERROR or need_ctr == 0:
            raise pa.PaError(-3, "decode_grouped: unsupported head_dim or block_size")
        counters, workspace, ws_ptr, ws_n = _pick_buffers(dev, st, need_ctr, need_ws, counters,
                                                          workspace)
        rc = l.pa_decode_grouped(pa._ptr(out), pa._ptr(q), pa._ptr(k_cache), pa._ptr(v_cache),
                                 pa._ptr(block_tables), pa._ptr(context_lens), float(scale),
                                 block_tables.shape[1], ctypes.byref(dims), Hq, ctypes.byref(opts),
                                 ws_ptr, ws_n, pa._ptr(counters), counters.numel() * 4, sh)
    pa._check(rc, "pa_decode_grouped")
    return out


def prefill_grouped(out, q, k_cache, v_cache, block_tables, context_lens, query_start, scale,
                    max_query_len=None, softcap=0.0, alibi_slopes=None, window=0, prefix_lens=None,
                    workspace=None, counters=None, stream=None):
    """Attention of the last q_len_s tokens of each sequence over its paged
    keys, with query heads that share K/V heads (pa_prefill_grouped).

    q, out [total_q, Hq, D]; query_start [S + 1] int32; max_query_len bounds
    every q_len_s (computed from query_start, with a device sync, when None).
    The rest as decode_grouped; a query at position p sees keys up to p, and
    the first prefix_lens[s] keys wherever it stands."""
    import torch
    pa = _pa()
    dev, S, Hq, dims, opts = _attention_args("prefill_grouped", out, q, k_cache, v_cache,
                                             block_tables, context_lens, softcap, alibi_slopes,
                                             window, prefix_lens)
    pa._need(query_start, "query_start", torch.int32, 1, dev)
    if query_start.shape[0] != S + 1:
        raise ValueError("prefill_grouped: inconsistent shapes")
    if max_query_len is None:
        max_query_len = int((query_start[1:] - query_start[:-1]).max()) if S else 0
    sh, st = pa._stream_handle(dev, stream)
    l = pa.lib()
    with torch.cuda.device(dev):
        need_ws = l.pa_prefill_grouped_workspace_bytes(ctypes.byref(dims), Hq, int(max_query_len))
        need_ctr = l.pa_prefill_grouped_counters_bytes(ctypes.byref(dims), Hq)
        if need_ws == pa._SIZE_ERROR or need_ctr == 0:
            raise pa.PaError(-3, "prefill_grouped: unsupported head_dim, block_size or heads, or "
                                 "a negative max_query_len")
        counters, workspace, ws_ptr, ws_n = _pick_buffers(dev, st, need_ctr, need_ws, counters,
                                                          workspace)
        rc = l.pa_prefill_grouped(pa._ptr(out), pa._ptr(q), pa._ptr(k_cache), pa._ptr(v_cache),
                                  pa._ptr(block_tables), pa._ptr(context_lens),
                                  pa._ptr(query_start), q.shape[0], int(max_query_len),
                                  float(scale), block_tables.shape[1], ctypes.byref(dims), Hq,
                                  ctypes.byref(opts), ws_ptr, ws_n, pa._ptr(counters),
                                  counters.numel() * 4, sh)
    pa._check(rc, "pa_prefill_grouped")
    return out
