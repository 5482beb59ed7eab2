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
import functools
import importlib.util
import threading
import warnings

torch = Tensor = _I32 = _F32 = _U8 = _raw_stream = _package = None
_marshal = None        # the compiled marshalling module: one call per operator
_get_device = _capturing = None
_addresses: dict = {}  # of the library's functions, for _marshal


_init_lock = threading.Lock()


def _init():
    """Imports what the calls need, at the first one (the package itself, with
    its block manager, works without torch).  _package is set last: a thread that
    finds it finds the rest, and one that comes before waits."""
    global torch, Tensor, _I32, _F32, _U8, _raw_stream, _package, _marshal, _get_device, _capturing
    with _init_lock:
        if _package is not None:
            return
        import torch as torch_
        import paged_kv_cache_269_gb300 as package
        torch, Tensor = torch_, torch_.Tensor
        _I32, _F32, _U8 = torch.int32, torch.float32, torch.uint8
        c = torch._C
        if all(hasattr(c, n) for n in ("_cuda_getCurrentRawStream", "_cuda_getDevice",
                                       "_cuda_isCurrentStreamCapturing")) and torch.cuda.is_available():
            torch.cuda.init()
            _raw_stream, _get_device = c._cuda_getCurrentRawStream, c._cuda_getDevice
            _capturing = c._cuda_isCurrentStreamCapturing
            l = package.lib()
            for name in ("pa_rope_and_cache", "pa_decode_grouped", "pa_decode_grouped_workspace_bytes",
                         "pa_decode_grouped_counters_bytes", "pa_prefill_grouped",
                         "pa_prefill_grouped_workspace_bytes", "pa_prefill_grouped_counters_bytes"):
                _addresses[name] = ctypes.cast(getattr(l, name), ctypes.c_void_p).value
            try:
                _marshal = _load_marshal(package._build.build_marshal())
            except (RuntimeError, OSError, ImportError) as e:
                # once: every call then takes the Python checks, slower by 9 us
                warnings.warn(f"the grouped calls' marshalling module is missing, their arguments are checked "
                              f"in Python: {e}", RuntimeWarning, stacklevel=4)
        # (without CUDA the checks refuse every tensor)
        _package = package


def _load_marshal(path):
    spec = importlib.util.spec_from_file_location("pa_marshal", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


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
    if _package is None:
        _init()
    return _package


# The checks below are made on every call, so they touch each tensor as little
# as they can; one that fails is left to _need, which says what is wrong.
def _plain(t, name, dtype, ndim, index, device):
    """Checks a contiguous tensor on the given device; returns its pointer."""
    if not (isinstance(t, Tensor) and t.dtype is dtype and t.dim() == ndim and t.get_device() == index
            and t.is_contiguous()):
        _pa()._need(t, name, dtype, ndim, device)
    return t.data_ptr()


def _caches(k_cache, v_cache):
    """Checks the caches; returns (device index, device, dtype code, dtype, shape)."""
    pa = _pa()
    if not isinstance(k_cache, Tensor):
        raise TypeError("k_cache must be a torch.Tensor")
    code, et = pa._element_dtype(k_cache), k_cache.dtype
    index = k_cache.get_device()
    if index < 0 or k_cache.dim() != 4 or not k_cache.is_contiguous():
        pa._need(k_cache, "k_cache", et, 4)
    device = k_cache.device
    _plain(v_cache, "v_cache", et, 4, index, device)
    shape = k_cache.shape
    if v_cache.shape != shape:
        raise ValueError("k_cache and v_cache must have one shape")
    return index, device, code, et, shape


_I32_MAX = 0x7fffffff


def _bound(value, name):
    """An upper bound (a window, the longest query) for a 32-bit argument, which
    would otherwise keep its low 32 bits: one past them bounds nothing."""
    n = int(value)
    if n != value:
        raise ValueError(f"{name} must be a whole number, got {value}")
    return max(-1, min(n, _I32_MAX))


def _cap(softcap):
    """The softcap as the fp32 number the library gets; one that would become 0
    there, which means none, is refused."""
    cap = ctypes.c_float(softcap or 0.0).value
    if cap == 0.0 and softcap:
        raise ValueError(f"softcap {softcap} is out of range")
    return cap


# What the library needs for given sizes (pure functions of them).
@functools.lru_cache(maxsize=4096)
def _decode_needs(S, Hq, H, D, B, code):
    pa, l = _pa(), _pa().lib()
    d = ctypes.byref(pa.Dims(S, H, D, B, 1, code))
    return l.pa_decode_grouped_workspace_bytes(d, Hq), l.pa_decode_grouped_counters_bytes(d, Hq)


@functools.lru_cache(maxsize=4096)
def _prefill_needs(S, Hq, H, D, B, code, max_query_len):
    pa, l = _pa(), _pa().lib()
    d = ctypes.byref(pa.Dims(S, H, D, B, 1, code))
    return (l.pa_prefill_grouped_workspace_bytes(d, Hq, max_query_len),
            l.pa_prefill_grouped_counters_bytes(d, Hq))


def rope_table(max_positions, rotary_dim, base=10000.0, inv_freq=None, device=None):
    """The fp32 [max_positions, rotary_dim] table rope_and_cache takes: row p
    holds cos(p f_i), then sin(p f_i), i < rotary_dim / 2, with
    f_i = base^(-2 i / rotary_dim) or the given inv_freq [rotary_dim / 2].
    Angles are taken in 64 bits, so far positions keep their phase.  Made once,
    when a model is loaded."""
    _pa()
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


def _rows(t, name, dtype, index, device, heads, dim):
    """Checks a [T, heads, dim] tensor whose rows may be apart (a slice of a
    packed projection); returns its pointer, its shape and the elements between
    one row and the next."""
    if not isinstance(t, Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    shape = t.shape
    if len(shape) != 3 or shape[2] != dim or (heads is not None and shape[1] != heads):
        raise ValueError(f"{name} must have shape [T, {'H' if heads is None else heads}, {dim}], "
                         f"got {tuple(shape)}")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    stride = t.stride()
    if stride[2] != 1 or (shape[1] > 1 and stride[1] != dim):
        raise ValueError(f"{name}: the heads of a row must be adjacent and contiguous")
    step = stride[0] if shape[0] > 1 else shape[1] * dim
    if step % 8:
        raise ValueError(f"{name}: rows must start on 16-byte boundaries")
    return t.data_ptr(), shape, step


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
    pa = _pa()
    if _marshal is not None:
        device = _get_device()
        rc = _marshal.rope(q_out, q, k, v, k_cache, v_cache, positions, cos_sin, slot_mapping, interleaved,
                           device, _raw_stream(device) if stream is None else stream.cuda_stream,
                           _addresses["pa_rope_and_cache"])
        if rc == 0:
            return q_out
        if rc is not None:
            pa._check(rc, "pa_rope_and_cache")
    index, dev, code, et, (N, H, B, D) = _caches(k_cache, v_cache)
    if torch.cuda.current_device() != index:
        with torch.cuda.device(index):
            return rope_and_cache(q_out, q, k, v, k_cache, v_cache, positions, cos_sin, slot_mapping,
                                  interleaved, stream)
    q_p, (T, Hq, _), qs = _rows(q, "q", et, index, dev, None, D)
    o_p, o_shape, os_ = _rows(q_out, "q_out", et, index, dev, Hq, D)
    k_p, k_shape, ks = _rows(k, "k", et, index, dev, H, D)
    v_p, v_shape, vs = _rows(v, "v", et, index, dev, H, D)
    pos_p = _plain(positions, "positions", _I32, 1, index, dev)
    slot_p = _plain(slot_mapping, "slot_mapping", _I32, 1, index, dev)
    cs_p = _plain(cos_sin, "cos_sin", _F32, 2, index, dev)
    if not (o_shape[0] == k_shape[0] == v_shape[0] == positions.shape[0] == slot_mapping.shape[0] == T):
        raise ValueError("rope_and_cache: inconsistent numbers of tokens")
    if T > 1 and os_ < Hq * D:
        raise ValueError("q_out: rows overlap")
    if T:
        row, kv_row = Hq * D, H * D
        if o_p != q_p or (os_ != qs and T > 1):
            _refuse_overlap(o_p, os_, row, q_p, qs, row, T, "q")
        _refuse_overlap(o_p, os_, row, k_p, ks, kv_row, T, "k")
        _refuse_overlap(o_p, os_, row, v_p, vs, kv_row, T, "v")
    max_positions, rotary_dim = cos_sin.shape
    rc = pa.lib().pa_rope_and_cache(
        o_p, q_p, k_p, v_p, k_cache.data_ptr(), v_cache.data_ptr(), pos_p, cs_p, slot_p, T, Hq, qs, ks,
        vs, os_, rotary_dim, max_positions, 1 if interleaved else 0, ctypes.byref(pa.Dims(0, H, D, B, N, code)),
        _raw_stream(index) if stream is None else stream.cuda_stream)
    if rc:
        pa._check(rc, "pa_rope_and_cache")
    return q_out


def _refuse_overlap(a0, a_step, a_row, b0, b_step, b_row, T, name):
    """Refuses an input of T rows at b0 that shares elements with q_out at a0
    (pointers in bytes; steps and rows in elements of 2 bytes).  Slices of one
    packed tensor that interleave without sharing are fine."""
    if a0 + 2 * ((T - 1) * a_step + a_row) <= b0 or b0 + 2 * ((T - 1) * b_step + b_row) <= a0:
        return
    if a_step == b_step and T > 1:
        # rows of one step: apart iff the offset leaves room on both sides
        off = (b0 - a0) % (2 * a_step)
        if off >= 2 * a_row and off + 2 * b_row <= 2 * a_step:
            return
    raise ValueError(f"q_out overlaps {name}")


# Per (device, stream): zeroed counters, which every successful call leaves
# zeroed, and a workspace; both grow on demand.
_buffers: dict = {}


def _buffers_for(index, stream, counters_bytes, workspace_bytes):
    pa = _pa()
    if stream is None:
        capturing = torch.cuda.is_current_stream_capturing()
        key = (index, _raw_stream(index))
    else:
        with torch.cuda.stream(stream):
            capturing = torch.cuda.is_current_stream_capturing()
        key = (index, stream.cuda_stream)
    if not capturing:
        got = _buffers.get(key)
        if got is not None and got[2] >= counters_bytes and got[3] >= workspace_bytes:
            return got[:2]
    with torch.cuda.stream(stream):          # no change where stream is None
        if capturing:
            return (torch.zeros(counters_bytes // 4, dtype=_I32, device=index),
                    torch.empty(max(workspace_bytes, 16), dtype=_U8, device=index))
        with pa._buf_lock:
            ctr, ws, nc, nw = _buffers.get(key, (None, None, 0, 0))
            if nc < counters_bytes:
                nc = max(counters_bytes, 1 << 14)
                ctr = torch.zeros(nc // 4, dtype=_I32, device=index)
            if ws is None or nw < workspace_bytes:
                nw = max(workspace_bytes, 16)
                ws = torch.empty(nw, dtype=_U8, device=index)
            _buffers[key] = (ctr, ws, nc, nw)
            return ctr, ws


def _known_buffers(stream, counters, workspace):
    """(device, stream handle, counters, workspace) for a call that can be
    marshalled as it stands: the caller's buffers, or the stream's cached ones
    outside a capture; counters None otherwise."""
    device = _get_device()
    handle = _raw_stream(device) if stream is None else stream.cuda_stream
    if counters is None or workspace is None:
        got = _buffers.get((device, handle))
        if got is None or stream is not None or _capturing():
            return device, handle, None, None
        return (device, handle, got[0] if counters is None else counters,
                got[1] if workspace is None else workspace)
    return device, handle, counters, workspace


def reset_counters():
    """Zero every cached counter buffer (needed after a device error), with no
    call in flight on any of their streams."""
    if _package is None:
        return             # no call was made
    with _package._buf_lock:
        devices = {index for index, _ in _buffers}
        for index in devices:
            torch.cuda.synchronize(index)
        for got in _buffers.values():
            got[0].zero_()
        for index in devices:
            torch.cuda.synchronize(index)


def _attention_args(what, out, q, k_cache, v_cache, block_tables, context_lens, softcap,
                    alibi_slopes, window, prefix_lens):
    index, dev, code, et, (N, H, B, D) = _caches(k_cache, v_cache)
    q_p = _plain(q, "q", et, 3, index, dev)
    o_p = _plain(out, "out", et, 3, index, dev)
    t_p = _plain(block_tables, "block_tables", _I32, 2, index, dev)
    l_p = _plain(context_lens, "context_lens", _I32, 1, index, dev)
    shape = q.shape
    Hq, (S, MB) = shape[1], block_tables.shape
    if out.shape != shape or shape[2] != D or context_lens.shape[0] != S:
        raise ValueError(f"{what}: inconsistent shapes")
    if H == 0 or Hq == 0 or Hq % H:
        raise ValueError(f"{what}: query heads must be a multiple of the cache's heads")
    opts = None
    cap, span = _cap(softcap), _bound(window or 0, "window")
    if MB > _I32_MAX:
        raise ValueError(f"{what}: block_tables are too wide")
    if cap or span or alibi_slopes is not None or prefix_lens is not None:
        a_p = x_p = None
        if alibi_slopes is not None:
            a_p = _plain(alibi_slopes, "alibi_slopes", _F32, 1, index, dev)
            if alibi_slopes.shape[0] != Hq:
                raise ValueError(f"{what}: alibi_slopes must have one entry per query head")
        if prefix_lens is not None:
            x_p = _plain(prefix_lens, "prefix_lens", _I32, 1, index, dev)
            if prefix_lens.shape[0] != S:
                raise ValueError(f"{what}: prefix_lens must have one entry per sequence")
        opts = ctypes.byref(AttnOpts(cap, span, a_p, x_p))
    head = (o_p, q_p, k_cache.data_ptr(), v_cache.data_ptr(), t_p, l_p)
    return index, dev, S, Hq, (H, D, B, code), MB, shape[0], head, _pa().Dims(S, H, D, B, N, code), opts


def _pick_buffers(index, dev, stream, need_ctr, need_ws, counters, workspace):
    """(workspace pointer, bytes, counters pointer, bytes): the caller's, or
    the cached ones."""
    if counters is None or (workspace is None and need_ws):
        c2, w2 = _buffers_for(index, stream, need_ctr, need_ws)
        if counters is None:
            counters = c2
        if workspace is None:
            workspace = w2
    c_p = _plain(counters, "counters", _I32, 1, index, dev)
    if workspace is None:
        return None, 0, c_p, counters.numel() * 4
    w_p = _plain(workspace, "workspace", _U8, 1, index, dev)
    return w_p, workspace.numel(), c_p, counters.numel() * 4


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
    pa = _pa()
    if _marshal is not None:
        device, handle, counters_, workspace_ = _known_buffers(stream, counters, workspace)
        if counters_ is not None:
            rc = _marshal.decode(out, q, k_cache, v_cache, block_tables, context_lens, scale, softcap,
                                 alibi_slopes, window, prefix_lens, counters_, workspace_, device, handle,
                                 _addresses["pa_decode_grouped"],
                                 _addresses["pa_decode_grouped_workspace_bytes"],
                                 _addresses["pa_decode_grouped_counters_bytes"])
            if rc == 0:
                return out
            if rc is not None:
                pa._check(rc, "pa_decode_grouped")
    index, dev, S, Hq, sizes, MB, rows, head, dims, opts = _attention_args(
        "decode_grouped", out, q, k_cache, v_cache, block_tables, context_lens, softcap, alibi_slopes,
        window, prefix_lens)
    if rows != S:
        raise ValueError("decode_grouped: inconsistent shapes")
    if torch.cuda.current_device() != index:
        with torch.cuda.device(index):
            return decode_grouped(out, q, k_cache, v_cache, block_tables, context_lens, scale, softcap,
                                  alibi_slopes, window, prefix_lens, workspace, counters, stream)
    need_ws, need_ctr = _decode_needs(S, Hq, *sizes)
    if need_ws == pa._SIZE_ERROR or need_ctr == 0:
        raise pa.PaError(-3, "decode_grouped: unsupported head_dim or block_size")
    w_p, w_n, c_p, c_n = _pick_buffers(index, dev, stream, need_ctr, need_ws, counters, workspace)
    rc = pa.lib().pa_decode_grouped(
        *head, float(scale), MB, ctypes.byref(dims), Hq, opts, w_p, w_n, c_p, c_n,
        _raw_stream(index) if stream is None else stream.cuda_stream)
    if rc:
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
    pa = _pa()
    if _marshal is not None and max_query_len is not None:
        device, handle, counters_, workspace_ = _known_buffers(stream, counters, workspace)
        if counters_ is not None:
            rc = _marshal.prefill(out, q, k_cache, v_cache, block_tables, context_lens, scale, softcap,
                                  alibi_slopes, window, prefix_lens, counters_, workspace_, device, handle,
                                  query_start, max_query_len, _addresses["pa_prefill_grouped"],
                                  _addresses["pa_prefill_grouped_workspace_bytes"],
                                  _addresses["pa_prefill_grouped_counters_bytes"])
            if rc == 0:
                return out
            if rc is not None:
                pa._check(rc, "pa_prefill_grouped")
    index, dev, S, Hq, sizes, MB, rows, head, dims, opts = _attention_args(
        "prefill_grouped", out, q, k_cache, v_cache, block_tables, context_lens, softcap, alibi_slopes,
        window, prefix_lens)
    qs_p = _plain(query_start, "query_start", _I32, 1, index, dev)
    if query_start.shape[0] != S + 1:
        raise ValueError("prefill_grouped: inconsistent shapes")
    if torch.cuda.current_device() != index:
        with torch.cuda.device(index):
            return prefill_grouped(out, q, k_cache, v_cache, block_tables, context_lens, query_start,
                                   scale, max_query_len, softcap, alibi_slopes, window, prefix_lens,
                                   workspace, counters, stream)
    if max_query_len is None:
        with torch.cuda.stream(stream):      # the one that query_start is ready on
            max_query_len = int((query_start[1:] - query_start[:-1]).max()) if S else 0
    max_query_len = _bound(max_query_len, "max_query_len")
    need_ws, need_ctr = _prefill_needs(S, Hq, *sizes, max_query_len)
    if need_ws == pa._SIZE_ERROR or need_ctr == 0:
        raise pa.PaError(-3, "prefill_grouped: unsupported head_dim, block_size or heads, or "
                             "a negative max_query_len")
    w_p, w_n, c_p, c_n = _pick_buffers(index, dev, stream, need_ctr, need_ws, counters, workspace)
    rc = pa.lib().pa_prefill_grouped(
        *head, qs_p, rows, max_query_len, float(scale), MB, ctypes.byref(dims), Hq, opts, w_p, w_n, c_p,
        c_n, _raw_stream(index) if stream is None else stream.cuda_stream)
    if rc:
        pa._check(rc, "pa_prefill_grouped")
    return out
