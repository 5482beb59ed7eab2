"""The 8-bit paged cache: its append, its read-back and the attention over it.

The binding of pa_norm_rope_and_cache, pa_gather_cache_q8, pa_decode_grouped_q8
and pa_prefill_grouped_q8.  An 8-bit cache is two float8_e4m3fn tensors
[N, H, B, D] with two float32 tensors of H scales; a value is its number times
its head's scale.  Like the rest of the package it only marshals arguments;
workspaces and counters are those of the 16-bit grouped calls, kept and shared
in the same way.
"""
from __future__ import annotations

import ctypes

from . import grouped as _g


class AppendOpts(ctypes.Structure):
    _fields_ = [("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p), ("eps", ctypes.c_float),
                ("k_scales", ctypes.c_void_p), ("v_scales", ctypes.c_void_p)]


def declare(l, dims_p):
    vp, i32, i64, sz, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
    op = ctypes.POINTER(_g.AttnOpts)
    l.pa_norm_rope_and_cache.argtypes = [vp] * 9 + [i32, i32, i64, i64, i64, i64, i32, i32, i32, dims_p,
                                                    ctypes.POINTER(AppendOpts), vp]
    l.pa_gather_cache_q8.argtypes = [vp] * 7 + [i32, dims_p, vp]
    l.pa_decode_grouped_q8.argtypes = [vp] * 8 + [f32, i32, dims_p, i32, op, vp, sz, vp, sz, vp]
    l.pa_prefill_grouped_q8.argtypes = [vp] * 9 + [i32, i32, f32, i32, dims_p, i32, op, vp, sz, vp, sz, vp]
    for name in ("pa_norm_rope_and_cache", "pa_gather_cache_q8", "pa_decode_grouped_q8", "pa_prefill_grouped_q8"):
        getattr(l, name).restype = ctypes.c_int


def _scales(k_scales, v_scales, index, dev, H):
    """Checks the scales; returns their pointers."""
    k_p = _g._plain(k_scales, "k_scales", _g._F32, 1, index, dev)
    v_p = _g._plain(v_scales, "v_scales", _g._F32, 1, index, dev)
    if k_scales.shape[0] != H or v_scales.shape[0] != H:
        raise ValueError("k_scales and v_scales must have one entry per head of the cache")
    return k_p, v_p


def _caches_q8(k_cache, v_cache, like, name):
    """Checks 8-bit caches that are used with a 16-bit tensor; returns what
    grouped._caches does, the dtype being that tensor's."""
    pa = _g._pa()
    torch = pa._torch()
    e4m3 = torch.float8_e4m3fn
    if not isinstance(like, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if like.dtype not in (torch.float16, torch.bfloat16):
        raise TypeError(f"{name} must be float16 or bfloat16, got {like.dtype}")
    pa._need(k_cache, "k_cache", e4m3, 4)
    pa._need(v_cache, "v_cache", e4m3, 4, k_cache.device)
    if v_cache.shape != k_cache.shape:
        raise ValueError("k_cache and v_cache must have one shape")
    code = pa.DTYPE_BF16 if like.dtype is torch.bfloat16 else pa.DTYPE_F16
    return k_cache.get_device(), k_cache.device, code, like.dtype, k_cache.shape


def norm_rope_and_cache(q_out, q, k, v, k_cache, v_cache, positions, cos_sin, slot_mapping, q_weight=None,
                        k_weight=None, eps=1e-6, interleaved=False, k_scales=None, v_scales=None, stream=None):
    """Norm the heads of q and k, rotate both by their tokens' positions, write q
    to q_out and append k and v to the caches at slot_mapping
    (pa_norm_rope_and_cache).

    q_weight, k_weight float32 [D]: each head row is divided by the root of its
    mean square (plus eps) and multiplied by the weights before the rotation;
    None leaves it as it is.  k_cache, v_cache [N, H, B, D] of q's dtype, or
    float8_e4m3fn with k_scales, v_scales float32 [H]: then the number nearest
    to value / scale is stored, values past 448 scales at 448.

    The rest as rope_and_cache, except that cos_sin may be None (no rotation;
    positions too, if no token is padding) and q with q_out (k and v alone)."""
    pa = _g._pa()
    if _g._marshal is not None:
        device = _g._get_device()
        rc = _g._marshal.norm_rope(q_out, q, k, v, k_cache, v_cache, positions, cos_sin, slot_mapping, interleaved,
                                   device, _g._raw_stream(device) if stream is None else stream.cuda_stream,
                                   q_weight, k_weight, eps, k_scales, v_scales,
                                   _g._addresses["pa_norm_rope_and_cache"])
        if rc == 0:
            return q_out
        if rc is not None:
            pa._check(rc, "pa_norm_rope_and_cache")
    torch = pa._torch()
    q8 = k_scales is not None or v_scales is not None
    if q8:
        index, dev, code, et, (N, H, B, D) = _caches_q8(k_cache, v_cache, k, "k")
    else:
        index, dev, code, et, (N, H, B, D) = _g._caches(k_cache, v_cache)
    if torch.cuda.current_device() != index:
        with torch.cuda.device(index):
            return norm_rope_and_cache(q_out, q, k, v, k_cache, v_cache, positions, cos_sin, slot_mapping, q_weight,
                                       k_weight, eps, interleaved, k_scales, v_scales, stream)
    opts = AppendOpts(None, None, float(eps), None, None)
    if q8:
        opts.k_scales, opts.v_scales = _scales(k_scales, v_scales, index, dev, H)
    for name, t in (("q_weight", q_weight), ("k_weight", k_weight)):
        if t is not None:
            setattr(opts, name, _g._plain(t, name, _g._F32, 1, index, dev))
            if t.shape[0] != D:
                raise ValueError(f"{name} must have one entry per dim of a head")
    k_p, (T, _, _), ks = _g._rows(k, "k", et, index, dev, H, D)
    v_p, v_shape, vs = _g._rows(v, "v", et, index, dev, H, D)
    slot_p = _g._plain(slot_mapping, "slot_mapping", _g._I32, 1, index, dev)
    if v_shape[0] != T or slot_mapping.shape[0] != T:
        raise ValueError("norm_rope_and_cache: inconsistent numbers of tokens")
    q_p = o_p = pos_p = cs_p = None
    Hq = qs = os_ = rotary_dim = max_positions = 0
    if (q is None) != (q_out is None):
        raise ValueError("norm_rope_and_cache: q and q_out go together")
    if q is not None:
        q_p, q_shape, qs = _g._rows(q, "q", et, index, dev, None, D)
        Hq = q_shape[1]
        o_p, o_shape, os_ = _g._rows(q_out, "q_out", et, index, dev, Hq, D)
        if q_shape[0] != T or o_shape[0] != T:
            raise ValueError("norm_rope_and_cache: inconsistent numbers of tokens")
        if T > 1 and os_ < Hq * D:
            raise ValueError("q_out: rows overlap")
        if T:
            if o_p != q_p or (os_ != qs and T > 1):
                _g._refuse_overlap(o_p, os_, Hq * D, q_p, qs, Hq * D, T, "q")
            _g._refuse_overlap(o_p, os_, Hq * D, k_p, ks, H * D, T, "k")
            _g._refuse_overlap(o_p, os_, Hq * D, v_p, vs, H * D, T, "v")
    if cos_sin is not None:
        cs_p = _g._plain(cos_sin, "cos_sin", _g._F32, 2, index, dev)
        max_positions, rotary_dim = cos_sin.shape
        if rotary_dim == 0:
            raise ValueError("cos_sin has no columns: pass None for no rotation")
    if positions is not None:
        pos_p = _g._plain(positions, "positions", _g._I32, 1, index, dev)
        if positions.shape[0] != T:
            raise ValueError("norm_rope_and_cache: inconsistent numbers of tokens")
    elif cos_sin is not None:
        raise ValueError("norm_rope_and_cache: a rotation needs positions")
    rc = pa.lib().pa_norm_rope_and_cache(
        o_p, q_p, k_p, v_p, k_cache.data_ptr(), v_cache.data_ptr(), pos_p, cs_p, slot_p, T, Hq, qs, ks, vs, os_,
        rotary_dim, max_positions, 1 if interleaved else 0, ctypes.byref(pa.Dims(0, H, D, B, N, code)),
        ctypes.byref(opts), _g._raw_stream(index) if stream is None else stream.cuda_stream)
    if rc:
        pa._check(rc, "pa_norm_rope_and_cache")
    return q_out


def reshape_and_cache_q8(k, v, k_cache, v_cache, k_scales, v_scales, slot_mapping, stream=None):
    """reshape_and_cache into an 8-bit cache: every token's k and v [T, H, D] as
    the e4m3 numbers nearest to value / scale (norm_rope_and_cache without q, norm
    and rotation)."""
    if k_scales is None or v_scales is None:
        raise TypeError("k_scales and v_scales must be tensors")
    norm_rope_and_cache(None, None, k, v, k_cache, v_cache, None, None, slot_mapping, k_scales=k_scales,
                        v_scales=v_scales, stream=stream)


def gather_cache_q8(k_out, v_out, k_cache, v_cache, k_scales, v_scales, slots, stream=None):
    """Read tokens of an 8-bit cache back (pa_gather_cache_q8): row i of k_out and
    v_out [T, H, D] (float16 or bfloat16) is what slots[i] (int32 [T]) holds, in
    any order and any number of times; slots[i] < 0 leaves the row as it is.
    Returns (k_out, v_out)."""
    pa = _g._pa()
    if _g._marshal is not None:
        device = _g._get_device()
        rc = _g._marshal.gather_q8(k_out, v_out, k_cache, v_cache, k_scales, v_scales, slots, device,
                                   _g._raw_stream(device) if stream is None else stream.cuda_stream,
                                   _g._addresses["pa_gather_cache_q8"])
        if rc == 0:
            return k_out, v_out
        if rc is not None:
            pa._check(rc, "pa_gather_cache_q8")
    torch = pa._torch()
    index, dev, code, et, (N, H, B, D) = _caches_q8(k_cache, v_cache, k_out, "k_out")
    ks_p, vs_p = _scales(k_scales, v_scales, index, dev, H)
    ko_p = _g._plain(k_out, "k_out", et, 3, index, dev)
    vo_p = _g._plain(v_out, "v_out", et, 3, index, dev)
    s_p = _g._plain(slots, "slots", _g._I32, 1, index, dev)
    T = slots.shape[0]
    if k_out.shape != (T, H, D) or v_out.shape != (T, H, D):
        raise ValueError("gather_cache_q8: inconsistent shapes")
    if T and abs(ko_p - vo_p) < T * H * D * 2:
        raise ValueError("k_out overlaps v_out")
    with torch.cuda.device(index):
        rc = pa.lib().pa_gather_cache_q8(
            ko_p, vo_p, k_cache.data_ptr(), v_cache.data_ptr(), ks_p, vs_p, s_p, T,
            ctypes.byref(pa.Dims(0, H, D, B, N, code)), _g._raw_stream(index) if stream is None else stream.cuda_stream)
    if rc:
        pa._check(rc, "pa_gather_cache_q8")
    return k_out, v_out


def decode_grouped_q8(out, q, k_cache, v_cache, k_scales, v_scales, block_tables, context_lens, scale, softcap=0.0,
                      alibi_slopes=None, window=0, prefix_lens=None, workspace=None, counters=None, stream=None):
    """decode_grouped over an 8-bit cache (pa_decode_grouped_q8): k_cache, v_cache
    float8_e4m3fn [N, H, B, D], k_scales, v_scales float32 [H]; q and out [S, Hq, D]
    float16 or bfloat16.  The rest as decode_grouped, workspace and counters too."""
    pa = _g._pa()
    if _g._marshal is not None:
        device, handle, counters_, workspace_ = _g._known_buffers(stream, counters, workspace)
        if counters_ is not None:
            rc = _g._marshal.decode_q8(out, q, k_cache, v_cache, block_tables, context_lens, scale, softcap,
                                       alibi_slopes, window, prefix_lens, counters_, workspace_, device, handle,
                                       k_scales, v_scales, _g._addresses["pa_decode_grouped_q8"],
                                       _g._addresses["pa_decode_grouped_workspace_bytes"],
                                       _g._addresses["pa_decode_grouped_counters_bytes"])
            if rc == 0:
                return out
            if rc is not None:
                pa._check(rc, "pa_decode_grouped_q8")
    torch = pa._torch()
    caches = _caches_q8(k_cache, v_cache, q, "q")
    scales = _scales(k_scales, v_scales, caches[0], caches[1], caches[4][1])
    index, dev, S, Hq, sizes, MB, rows, head, dims, opts = _g._attention_args(
        "decode_grouped_q8", out, q, k_cache, v_cache, block_tables, context_lens, softcap, alibi_slopes, window,
        prefix_lens, caches)
    if rows != S:
        raise ValueError("decode_grouped_q8: inconsistent shapes")
    if torch.cuda.current_device() != index:
        with torch.cuda.device(index):
            return decode_grouped_q8(out, q, k_cache, v_cache, k_scales, v_scales, block_tables, context_lens, scale,
                                     softcap, alibi_slopes, window, prefix_lens, workspace, counters, stream)
    need_ws, need_ctr = _g._decode_needs(S, Hq, *sizes)
    if need_ws == pa._SIZE_ERROR or need_ctr == 0:
        raise pa.PaError(-3, "decode_grouped_q8: unsupported head_dim or block_size")
    w_p, w_n, c_p, c_n = _g._pick_buffers(index, dev, stream, need_ctr, need_ws, counters, workspace)
    rc = pa.lib().pa_decode_grouped_q8(
        *head[:4], *scales, *head[4:], float(scale), MB, ctypes.byref(dims), Hq, opts, w_p, w_n, c_p, c_n,
        _g._raw_stream(index) if stream is None else stream.cuda_stream)
    if rc:
        pa._check(rc, "pa_decode_grouped_q8")
    return out


def prefill_grouped_q8(out, q, k_cache, v_cache, k_scales, v_scales, block_tables, context_lens, query_start, scale,
                       max_query_len=None, softcap=0.0, alibi_slopes=None, window=0, prefix_lens=None, workspace=None,
                       counters=None, stream=None):
    """prefill_grouped over an 8-bit cache (pa_prefill_grouped_q8): k_cache,
    v_cache float8_e4m3fn [N, H, B, D], k_scales, v_scales float32 [H]; q and out
    [total_q, Hq, D] float16 or bfloat16.  The rest as prefill_grouped, workspace
    and counters too."""
    pa = _g._pa()
    if _g._marshal is not None and max_query_len is not None:
        device, handle, counters_, workspace_ = _g._known_buffers(stream, counters, workspace)
        if counters_ is not None:
            rc = _g._marshal.prefill_q8(out, q, k_cache, v_cache, block_tables, context_lens, scale, softcap,
                                        alibi_slopes, window, prefix_lens, counters_, workspace_, device, handle,
                                        k_scales, v_scales, query_start, max_query_len,
                                        _g._addresses["pa_prefill_grouped_q8"],
                                        _g._addresses["pa_prefill_grouped_workspace_bytes"],
                                        _g._addresses["pa_prefill_grouped_counters_bytes"])
            if rc == 0:
                return out
            if rc is not None:
                pa._check(rc, "pa_prefill_grouped_q8")
    torch = pa._torch()
    caches = _caches_q8(k_cache, v_cache, q, "q")
    scales = _scales(k_scales, v_scales, caches[0], caches[1], caches[4][1])
    index, dev, S, Hq, sizes, MB, rows, head, dims, opts = _g._attention_args(
        "prefill_grouped_q8", out, q, k_cache, v_cache, block_tables, context_lens, softcap, alibi_slopes, window,
        prefix_lens, caches)
    qs_p = _g._plain(query_start, "query_start", _g._I32, 1, index, dev)
    if query_start.shape[0] != S + 1:
        raise ValueError("prefill_grouped_q8: inconsistent shapes")
    if torch.cuda.current_device() != index:
        with torch.cuda.device(index):
            return prefill_grouped_q8(out, q, k_cache, v_cache, k_scales, v_scales, block_tables, context_lens,
                                      query_start, scale, max_query_len, softcap, alibi_slopes, window, prefix_lens,
                                      workspace, counters, stream)
    if max_query_len is None:
        with torch.cuda.stream(stream):      # the one that query_start is ready on
            max_query_len = int((query_start[1:] - query_start[:-1]).max()) if S else 0
    max_query_len = _g._bound(max_query_len, "max_query_len")
    need_ws, need_ctr = _g._prefill_needs(S, Hq, *sizes, max_query_len)
    if need_ws == pa._SIZE_ERROR or need_ctr == 0:
        raise pa.PaError(-3, "prefill_grouped_q8: unsupported head_dim, block_size or heads, or "
                             "a negative max_query_len")
    w_p, w_n, c_p, c_n = _g._pick_buffers(index, dev, stream, need_ctr, need_ws, counters, workspace)
    rc = pa.lib().pa_prefill_grouped_q8(
        *head[:4], *scales, *head[4:], qs_p, rows, max_query_len, float(scale), MB, ctypes.byref(dims), Hq, opts, w_p,
        w_n, c_p, c_n, _g._raw_stream(index) if stream is None else stream.cuda_stream)
    if rc:
        pa._check(rc, "pa_prefill_grouped_q8")
    return out
