"""GPU tests of the grouped calls at the edges of their buffers, and of what may
not reach their outputs; references and bounds as in grouped_ref."""
import pytest
import torch

import paged_kv_cache_269_gb300 as pa
from grouped_ref import TINY, U, make_case, reference, seen_mask
from test_gpu_grouped import check, run_decode, run_prefill, to_dev

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    d = torch.device("cuda", 0)
    torch.cuda.set_device(d)
    pa.lib()
    pa.device_errors()
    return d


# ------------------------------------------------------------------ buffers

@pytest.mark.parametrize("S,H,group,D", [(63, 1, 4, 128), (127, 1, 4, 64), (21, 3, 2, 128), (64, 1, 4, 128),
                                         (9, 7, 1, 64), (63, 1, 9, 256), (7, 3, 40, 64)])
def test_decode_counters_of_the_stated_size(dev, S, H, group, D):
    """Counters of exactly the stated size inside a larger tensor, at numbers of
    tickets that fill it (or pass it by one): the last context, which several CTAs
    share, is joined, and the words around the buffer stay as they were."""
    ctx = [1 + 13 * s % 40 for s in range(S)]
    ctx[-1] = 6000
    c = make_case(101, ctx, [1] * S, H * group, H, D, 16, F16)
    d = to_dev(c, dev)
    n = pa.decode_grouped_counters_bytes(S, H * group, H, D, 16) // 4
    guarded = torch.full((n + 128,), 0x5A5A5A5A, dtype=torch.int32, device=dev)
    guarded[64:64 + n] = 0
    ws = torch.empty(pa.decode_grouped_workspace_bytes(H * group, H, D, 16), dtype=torch.uint8, device=dev)
    for _ in range(3):
        out = run_decode(c, d, counters=guarded[64:64 + n], workspace=ws)
        assert pa.device_errors() == 0
        check(c, out, False)
        assert not guarded[64:64 + n].any()
        assert (guarded[:64] == 0x5A5A5A5A).all() and (guarded[64 + n:] == 0x5A5A5A5A).all()


@pytest.mark.parametrize("S", [63, 127])
def test_decode_counters_of_a_captured_call(dev, S):
    """A captured call takes counters of the stated size from the graph's pool."""
    ctx = [1 + 13 * s % 40 for s in range(S)]
    ctx[-1] = 6000
    c = make_case(102, ctx, [1] * S, 4, 1, 128, 16, BF16)
    d = to_dev(c, dev)
    out = torch.empty_like(d["q"])
    run_decode(c, d, out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run_decode(c, d, out)
    for _ in range(3):
        out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        check(c, out, False)
    assert pa.device_errors() == 0


# ------------------------------------------------------------------ prefill's roles

@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("D,group,alibi", [(64, 4, False), (64, 4, True), (64, 1, False), (128, 4, False)])
def test_prefill_tiles_of_unequal_pace(dev, dtype, D, group, alibi):
    """Second query tiles whose softmax is slow at every key tile (an outlier past
    the cap's polynomial), items whose second tile is empty behind them, and a last
    key tile that ends inside a block: each tile masks with its own blocks."""
    per = 128 // group
    new = [per * (1 + 2 * (i % 4)) + i % 3 for i in range(60)]
    ctx = [n + (997 - 13 * i) % 700 + 200 for i, n in enumerate(new)]
    c = make_case(103, ctx, new, group, 1, D, 16, dtype, cap=10.0, alibi=alibi)
    for s, n in enumerate(new):
        for first in range(per, n, 2 * per):          # one token of every second tile
            c.q[c.starts_list[s] + first] *= 40.0
    d = to_dev(c, dev)
    want, bound = (x.to(dev) for x in reference(c, True))
    for _ in range(20):
        got = run_prefill(c, d)
        assert pa.device_errors() == 0
        assert ((got.double() - want).abs() <= bound).all()


# ------------------------------------------------------------------ what no query sees

def _unseen_keys(c):
    """[N, B] bool: slots of the pool that no query sees."""
    seen = torch.zeros(c.k_cache.shape[0], c.B, dtype=torch.bool)
    for s, ctx in enumerate(c.ctx):
        if c.new[s]:
            for j in seen_mask(c, s).any(0).nonzero().flatten().tolist():
                seen[int(c.tables[s, j // c.B]), j % c.B] = True
    return ~seen


def _same_whatever_is_unseen(c, dev, run, weights16):
    """One result, to the bit, whatever the unseen key rows hold and whatever a call
    before has left in the shared memory of boxes that are not loaded."""
    d = to_dev(c, dev)
    unseen = _unseen_keys(c).to(dev)[:, None, :, None]
    dirty = make_case(1, [128] * 320, [1] * 320, c.q_heads, c.kv_heads, c.D, c.B, c.dtype)
    dd = to_dev(dirty, dev)
    dd["v_cache"].zero_()
    first = None
    for value in (0.0, float("nan"), 6e4, -6e4, float("inf")):
        k = torch.where(unseen, torch.full_like(d["k_cache"], value), d["k_cache"])
        dd["k_cache"].fill_(value)
        for _ in range(3):
            run(dirty, dd)
            got = run(c, dict(d, k_cache=k))
            first = got if first is None else first
            assert torch.equal(first, got), f"unseen keys of {value}"
    assert pa.device_errors() == 0
    check(c, first, weights16)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("D,B,group", [(64, 16, 2), (64, 8, 8), (64, 32, 9), (128, 16, 4), (128, 32, 8), (256, 8, 2)])
def test_capped_decode_ignores_unseen_keys(dev, dtype, D, B, group):
    ctx = [10, 45, 300, 17, 1, 130]
    c = make_case(104, ctx, [1] * 6, 2 * group, 2, D, B, dtype, cap=50.0, window=37, prefix=[0, 3, 0, 17, 1, 40])
    _same_whatever_is_unseen(c, dev, run_decode, False)
    c = make_case(105, ctx, [1] * 6, 2 * group, 2, D, B, dtype, cap=20.0, alibi=True)
    _same_whatever_is_unseen(c, dev, run_decode, False)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("D,B,alibi", [(64, 16, False), (64, 8, True), (128, 16, False), (128, 32, True)])
def test_capped_prefill_ignores_unseen_keys(dev, dtype, D, B, alibi):
    ctx, new = [10, 45, 300, 17, 200], [4, 45, 30, 1, 130]
    c = make_case(106, ctx, new, 8, 2, D, B, dtype, cap=50.0, window=37, prefix=[0, 3, 0, 17, 40], alibi=alibi)
    _same_whatever_is_unseen(c, dev, run_prefill, True)
    c = make_case(107, ctx, new, 8, 2, D, B, dtype, cap=20.0, alibi=alibi)
    _same_whatever_is_unseen(c, dev, run_prefill, True)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("D,group", [(128, 3), (64, 3), (128, 4), (64, 5), (128, 12)])
@pytest.mark.parametrize("cap", [0.0, 20.0])
def test_prefill_rows_of_others_do_not_round(dev, dtype, D, group, cap):
    """A sequence's result is the same to the bit whatever the queries of its
    neighbours in the pack and the rows behind the last sequence hold: rows of a tile
    that are not the sequence's, and rows that no query fills when the heads do not
    divide 128, decide nothing."""
    S = 100
    new = [1 + (37 * s) % 90 for s in range(S)]
    ctx = [n + (53 * s) % 150 for s, n in enumerate(new)]
    c = make_case(108, ctx, new, 2 * group, 2, D, 16, dtype, cap=cap)
    d = to_dev(c, dev)
    rows = c.starts_list[-1]
    mine = torch.zeros(rows, dtype=torch.bool)
    for s in range(0, S, 2):
        mine[c.starts_list[s]:c.starts_list[s + 1]] = True
    mine = mine.to(dev)
    first = None
    for value in (None, 0.0, float("nan"), 300.0, -300.0, float("inf")):
        q = torch.cat([d["q"], torch.zeros(40, 2 * group, D, dtype=dtype, device=dev)])
        if value is not None:
            q[:rows][~mine] = value
            q[rows:] = value
        for _ in range(3):
            got = torch.full_like(q, 7.0)
            run_prefill(c, dict(d, q=q), got)
            assert (got[rows:] == 7.0).all()
            if first is None:
                check(c, got[:rows], True)
                first = got[:rows][mine]
            assert torch.equal(first, got[:rows][mine]), f"other queries of {value}"
    assert pa.device_errors() == 0


# ------------------------------------------------------------------ caps

def _capped_reference(c, weights16, share):
    """As grouped_ref.reference for a capped call without biases, but each score is
    off by 2^-20 of itself where it was 2^-20 of the cap (share: 2^-20 of the
    cap, for one score in four).  The cap's slope is at most 1, so the dot
    product's error passes through it undiminished at most."""
    out, bound = torch.zeros(c.q.shape).double(), torch.zeros(c.q.shape).double()
    G, u = c.q_heads // c.kv_heads, U[c.dtype]
    for s, ctx in enumerate(c.ctx):
        r = slice(c.starts_list[s], c.starts_list[s + 1])
        seen = seen_mask(c, s)
        blk, off = c.tables[s, torch.arange(ctx) // c.B].long(), torch.arange(ctx) % c.B
        for hq in range(c.q_heads):
            K, V = c.k_cache[blk, hq // G, off].double(), c.v_cache[blk, hq // G, off].double()
            q = c.q[r, hq].double()
            x = c.cap * torch.tanh(q @ K.T * c.scale / c.cap)
            d = c.D * 2.0 ** -23 * abs(c.scale) * (q.abs() @ K.abs().T)
            d = d + 2.0 ** -20 * (c.cap if share else x.abs()) + 2.0 ** -21 * x.abs()
            x = x.masked_fill(~seen, float("-inf"))
            w = torch.softmax(x, -1)
            mag = w @ V.abs()
            d = torch.where(x >= x.amax(-1, keepdim=True) - 28.0, d, torch.zeros_like(d))
            n = seen.sum(-1, keepdim=True).double()
            rel = 2.1 * d.amax(-1, keepdim=True) + (64 + n / 16) * 2.0 ** -23 + (u if weights16 else 2.0 ** -16)
            out[r, hq] = w @ V
            bound[r, hq] = (u * out[r, hq].abs() + rel * mag) * 1.001 + TINY[c.dtype]
    return out, bound


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("cap", [3.0, 128.0, 129.0, 1e3, 1025.0, 1e5, 1e7, 1e25])
def test_caps_of_any_size_keep_the_scores(dev, dtype, cap):
    """A cap far above the scores changes nothing, one among them bends them, and
    neither costs a score more than 2^-20 of itself (prefill: 2^-20 of a cap up to 128
    in fp16, 1024 in bf16)."""
    for D, group in ((128, 4), (64, 2)):
        c = make_case(109, [90, 300], [1, 1], 2 * group, 2, D, 16, dtype, cap=cap, q_scale=3.0)
        got = run_decode(c, to_dev(c, dev)).cpu().double()
        want, bound = _capped_reference(c, False, False)
        assert ((got - want).abs() <= bound).all()
        c = make_case(110, [90, 300, 70], [90, 200, 3], 2 * group, 2, D, 16, dtype, cap=cap, q_scale=3.0)
        got = run_prefill(c, to_dev(c, dev)).cpu().double()
        want, bound = _capped_reference(c, True, cap <= (128.0 if dtype == F16 else 1024.0))
        assert ((got - want).abs() <= bound).all()
    assert pa.device_errors() == 0


# ------------------------------------------------------------------ the binding's numbers

def test_bounds_past_32_bits(dev):
    """A window or a longest query that 32 bits do not hold limits nothing."""
    c = make_case(111, [90, 300], [1, 1], 4, 2, 128, 16, F16)
    d = to_dev(c, dev)
    first = run_decode(c, d)
    for window in (2 ** 31, 2 ** 32 + 5, 2 ** 63 - 1):
        c.window = window
        assert torch.equal(first, run_decode(c, d))
    c.window, c.cap = 0, 1e-50
    with pytest.raises(ValueError):
        run_decode(c, d)
    c = make_case(112, [90, 300], [90, 30], 4, 2, 128, 16, F16)
    d = to_dev(c, dev)
    first = run_prefill(c, d)
    c.window = 2 ** 32 + 5
    assert torch.equal(first, run_prefill(c, d))
    c.window = 0
    many = make_case(112, [1, 2] * 40, [1] * 80, 128, 64, 64, 16, F16)
    for longest in (2 ** 32 + 5, 2 ** 33):     # more work items than there can be
        with pytest.raises(pa.PaError):
            run_prefill(many, to_dev(many, dev), max_query_len=longest)
    assert pa.device_errors() == 0


# ------------------------------------------------------------------ large numbers

@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("base", [2.0, 2.5])
def test_scores_of_a_large_step(dev, dtype, D, base):
    """Scores near 2^26, where fp32 counts in steps of 8: keys a step apart, the larger
    ones last, give a finite softmax of them (the weights' ratio is 2^-8)."""
    c = make_case(113, [200, 100], [1, 1], 8, 2, D, 16, dtype, scale=0.6931471805599453)
    big = 4096.0 * 2 if dtype == F16 else 8192.0
    for s, n in enumerate(c.ctx):
        for j in range(n):
            k = c.k_cache[int(c.tables[s, j // 16]), :, j % 16]
            k[:] = 0.0
            k[:, 0] = big * base / 2
            k[:, 1] = 1.0 if j < 64 else 2.0
    c.q[:] = 0.0
    c.q[:, :, 0], c.q[:, :, 1] = big, 8.0            # scores of 2^26 base / 2 + 8 or 16, in log2 units
    for run in (run_decode, run_prefill):
        got = run(c, to_dev(c, dev)).cpu().double()
        assert torch.isfinite(got).all()
        for s, n in enumerate(c.ctx):
            V = torch.stack([c.v_cache[int(c.tables[s, j // 16]), :, j % 16].double() for j in range(n)])   # [n, H, D]
            w = torch.where(torch.arange(n) < 64, 2.0 ** -8, 1.0).double()
            want = torch.einsum("n,nhd->hd", w / w.sum(), V).repeat_interleave(4, 0)
            # a score that is off by a step moves the early keys' part of the output,
            # at most 64 / n of the weights, between two means of the same values
            share = 2.0 * 64 / n * V.abs().amax()
            assert ((got[s] - want).abs() <= share + U[dtype] * V.abs().amax()).all()
    assert pa.device_errors() == 0


# ------------------------------------------------------------------ streams

def test_calls_on_a_given_stream(dev):
    """stream= orders the whole call, the search for the longest query among it, and
    has buffers of its own, in a capture too."""
    side = torch.cuda.Stream(dev)
    c = make_case(114, [700, 90, 3000], [64, 90, 5], 8, 2, 128, 16, F16)
    d = to_dev(c, dev)
    want = run_prefill(c, d)
    starts = d["starts"].clone()
    busy = torch.randn(4096, 4096, device=dev)
    torch.cuda.synchronize()
    for _ in range(3):
        late = torch.zeros_like(starts)
        out = torch.zeros_like(d["q"])
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            for _ in range(40):
                busy @ busy
            late.copy_(starts)
        run_prefill(c, dict(d, starts=late), out, max_query_len=None, stream=side)
        side.synchronize()
        assert torch.equal(want, out)
    e = make_case(115, [700, 3000, 9], [1] * 3, 8, 2, 128, 16, BF16)
    de = to_dev(e, dev)
    want = run_decode(e, de)
    torch.cuda.synchronize()
    out = torch.zeros_like(want)
    run_decode(e, de, out, stream=side)
    side.synchronize()
    assert torch.equal(want, out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        run_decode(e, de, out, stream=side)
        run_decode(e, de, out, stream=side)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(want, out)
    assert pa.device_errors() == 0


# ------------------------------------------------------------------ batches

@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("D,group,kw", [(128, 4, {}), (64, 3, dict(alibi=True)), (128, 8, dict(window=200, cap=30.0))])
def test_prefill_a_chunk_beside_single_tokens(dev, dtype, D, group, kw):
    """A prompt's chunk and the next tokens of running sequences in one call: most
    work items of the call are empty."""
    ctx = [1500] + [17 + 41 * s % 700 for s in range(63)]
    c = make_case(116, ctx, [600] + [1] * 63, 2 * group, 2, D, 16, dtype, **kw)
    got = run_prefill(c, to_dev(c, dev))
    assert pa.device_errors() == 0
    check(c, got, True)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_unseen_keys_and_values_stay_out(dev, dtype, D):
    """NaN and infinities in keys and values behind a decode's window, and in keys
    behind a prompt's, with the bound of grouped_ref."""
    ctx = [300, 77, 40]
    for run, new, weights16 in ((run_decode, [1, 1, 1], False), (run_prefill, [60, 5, 40], True)):
        if run is run_prefill and D == 256:
            continue
        c = make_case(117, ctx, new, 8, 2, D, 16, dtype, window=33)
        unseen = _unseen_keys(c)[:, None, :, None]
        c.k_cache = torch.where(unseen, torch.full_like(c.k_cache, float("inf")), c.k_cache)
        if run is run_decode:
            c.v_cache = torch.where(unseen, torch.full_like(c.v_cache, float("nan")), c.v_cache)
        got = run(c, to_dev(c, dev))
        assert pa.device_errors() == 0
        check(c, got, weights16)
