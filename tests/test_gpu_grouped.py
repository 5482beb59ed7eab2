"""GPU parity of rope_and_cache, decode_grouped and prefill_grouped against the
fp64 reference of grouped_ref, within the bounds derived there."""
import pytest
import torch

import paged_kv_cache_269_gb300 as pa
from paged_kv_cache_269_gb300 import grouped
from grouped_ref import make_case, reference, rope_bound, rotate

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module", params=["marshalled", "checked"])
def dev(request):
    """Each test runs through the compiled marshalling module, and through the
    Python checks that take over from it."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    d = torch.device("cuda", 0)
    torch.cuda.set_device(d)
    pa.lib()
    pa.device_errors()
    grouped._pa()
    known = grouped._marshal
    assert known is not None
    if request.param == "checked":
        grouped._marshal = None
    yield d
    grouped._marshal = known


def to_dev(c, dev):
    d = {n: getattr(c, n).to(dev) for n in ("q", "k_cache", "v_cache", "tables", "lens", "starts")}
    d["slopes"] = None if c.slopes is None else c.slopes.to(dev)
    d["prefix"] = None if c.prefix is None else c.prefix.to(dev)
    return d


def run_decode(c, d, out=None, **kw):
    out = torch.full_like(d["q"], float("nan")) if out is None else out
    pa.decode_grouped(out, d["q"], d["k_cache"], d["v_cache"], d["tables"], d["lens"], c.scale,
                      softcap=c.cap, alibi_slopes=d["slopes"], window=c.window,
                      prefix_lens=d["prefix"], **kw)
    return out


def run_prefill(c, d, out=None, **kw):
    out = torch.full_like(d["q"], float("nan")) if out is None else out
    kw.setdefault("max_query_len", max(c.new))
    pa.prefill_grouped(out, d["q"], d["k_cache"], d["v_cache"], d["tables"], d["lens"], d["starts"],
                       c.scale, softcap=c.cap, alibi_slopes=d["slopes"], window=c.window,
                       prefix_lens=d["prefix"], **kw)
    return out


def check(c, got, weights16, what=""):
    want, bound = reference(c, weights16)
    got = got.cpu().double()
    assert torch.isfinite(got).all(), f"{what}: non-finite output"
    worst = ((got - want).abs() / bound.clamp(min=1e-300)).max().item() if got.numel() else 0.0
    assert worst <= 1.0, f"{what}: error {worst:.3g} x the bound"


def decode(c, dev, what=""):
    got = run_decode(c, to_dev(c, dev))
    assert pa.device_errors() == 0
    check(c, got, False, what)


def prefill(c, dev, what=""):
    got = run_prefill(c, to_dev(c, dev))
    assert pa.device_errors() == 0
    check(c, got, True, what)


# ------------------------------------------------------------------ decode

@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("B", [8, 16, 32])
def test_decode_shapes(dev, dtype, D, B):
    ctx = [1, 2, 7, 15, 16, 17, 31, 33, 64, 100, 257]
    decode(make_case(11, ctx, [1] * len(ctx), 8, 2, D, B, dtype), dev)


@pytest.mark.parametrize("group", [1, 2, 3, 5, 7, 8, 9, 16, 17, 40, 71])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_decode_groups(dev, group, D):
    decode(make_case(12, [40, 1, 300, 0], [1, 1, 1, 1], 3 * group, 3, D, 16, BF16), dev)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("window,prefix", [(0, None), (1, None), (5, None), (64, None), (100, [4] * 6),
                                           (17, [0, 1, 16, 33, 200, 999]), (0, [3] * 6), (1, [1, -5, 0, 40, 63, 64])])
@pytest.mark.parametrize("cap,alibi", [(0.0, False), (20.0, False), (0.0, True), (5.0, True)])
def test_decode_options(dev, dtype, window, prefix, cap, alibi):
    ctx = [1, 16, 63, 128, 500, 1023]
    c = make_case(13, ctx, [1] * 6, 12, 4, 128, 16, dtype, window=window, prefix=prefix, cap=cap, alibi=alibi,
                  q_scale=2.0)
    decode(c, dev)


@pytest.mark.parametrize("D,B", [(64, 8), (64, 32), (256, 16), (256, 8)])
def test_decode_options_other_shapes(dev, D, B):
    ctx = [9, 130, 1, 700, 65]
    c = make_case(14, ctx, [1] * 5, 14, 2, D, B, BF16, window=70, prefix=[3, 40, 0, 9, 64], cap=15.0, alibi=True)
    decode(c, dev)


def test_decode_long_contexts(dev):
    decode(make_case(15, [9000, 3, 20011], [1] * 3, 8, 1, 64, 16, F16), dev)
    decode(make_case(16, [12345], [1], 6, 2, 128, 32, BF16, alibi=True), dev)


def test_decode_many_short_sequences(dev):
    g = torch.Generator().manual_seed(5)
    ctx = torch.randint(0, 40, (3000,), generator=g).tolist()
    decode(make_case(17, ctx, [1] * 3000, 2, 1, 64, 16, F16), dev)


def test_decode_negative_and_zero_scale(dev):
    decode(make_case(18, [50, 300], [1, 1], 8, 2, 128, 16, BF16, scale=-0.09), dev)
    decode(make_case(18, [50, 300], [1, 1], 8, 2, 128, 16, BF16, scale=0.0), dev)


def test_decode_score_profiles(dev):
    # scores that rise, fall and spike along the context: the running maximum moves
    for kind in range(4):
        c = make_case(19, [600, 33], [1, 1], 8, 2, 128, 16, F16)
        j = torch.arange(600).float()
        prof = [j / 20, 30 - j / 20, torch.where(j == 577, 30.0, 0.0), (j % 64) / 2][kind]
        for i in range(600):
            blk = int(c.tables[0, i // 16])
            c.k_cache[blk, :, i % 16, 0] = prof[i]
        c.q[0, :, 0] = 11.0
        decode(c, dev, f"profile {kind}")


def test_decode_context_errors_and_bad_entries(dev):
    c = make_case(20, [50, 64, 33], [1] * 3, 4, 2, 128, 16, F16)
    d = to_dev(c, dev)
    d["lens"] = torch.tensor([-3, c.tables.shape[1] * 16 + 1, 33], dtype=torch.int32, device=dev)
    got = run_decode(c, d)
    assert pa.device_errors() == pa.DEVERR_CONTEXT
    assert (got[:2] == 0).all()
    want, bound = reference(c, False)
    assert ((got[2].cpu().double() - want[2]).abs() <= bound[2]).all()
    # a bad entry inside a context: its keys are left out
    c = make_case(21, [64], [1], 4, 2, 128, 16, F16)
    d = to_dev(c, dev)
    d["tables"][0, 1] = c.k_cache.shape[0]
    got = run_decode(c, d)
    assert pa.device_errors() == pa.DEVERR_TABLE
    c2 = make_case(21, [64], [1], 4, 2, 128, 16, F16)
    keep = [0, 2, 3]
    c2.tables[0, :3] = c.tables[0, keep]
    c2.ctx, c2.lens = [48], torch.tensor([48], dtype=torch.int32)
    check(c2, got, False, "bad entry")


def test_decode_on_a_side_stream_and_in_graphs(dev):
    # two graphs captured on one stream, replayed at once on two streams, and
    # an eager call in between: none shares buffers with another
    cases = [make_case(22 + i, [700 + 50 * i, 3000], [1, 1], 8, 1, 128, 16, BF16) for i in range(2)]
    ds = [to_dev(c, dev) for c in cases]
    outs = [torch.zeros_like(d["q"]) for d in ds]
    side = torch.cuda.Stream(dev)
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(side):
        for c, d, o in zip(cases, ds, outs):
            run_decode(c, d, o)
    side.synchronize()
    for c, d, o in zip(cases, ds, outs):
        check(c, o, False, "side stream")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            run_decode(c, d, o)
        graphs.append(g)
    streams = [torch.cuda.Stream(dev) for _ in range(2)]
    eager = torch.zeros_like(outs[0])
    torch.cuda.synchronize()
    for _ in range(20):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        run_decode(cases[0], ds[0], eager)
        torch.cuda.synchronize()
        for c, o in zip(cases, outs):
            check(c, o, False, "graph")
        check(cases[0], eager, False, "eager")
    assert pa.device_errors() == 0


def test_decode_is_reproducible_and_leaves_counters_zero(dev):
    c = make_case(24, [5000, 40, 900], [1] * 3, 16, 2, 128, 16, BF16)
    d = to_dev(c, dev)
    ctr = torch.zeros(pa.decode_grouped_counters_bytes(3, 16, 2, 128, 16) // 4, dtype=torch.int32, device=dev)
    ws = torch.empty(pa.decode_grouped_workspace_bytes(16, 2, 128, 16), dtype=torch.uint8, device=dev)
    first = run_decode(c, d, counters=ctr, workspace=ws)
    for _ in range(10):
        ws.fill_(255)
        assert torch.equal(first, run_decode(c, d, counters=ctr, workspace=ws))
        assert not ctr.any()
    with pytest.raises(pa.PaError):
        run_decode(c, d, counters=ctr[:0].clone(), workspace=ws)


# ------------------------------------------------------------------ prefill

CTX = [1, 15, 16, 17, 64, 65, 127, 128, 129, 300, 513]


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("D,B", [(64, 8), (64, 16), (64, 32), (128, 8), (128, 16), (128, 32)])
@pytest.mark.parametrize("mode", ["whole", "chunk", "single"])
def test_prefill_ragged(dev, dtype, D, B, mode):
    new = {"whole": CTX, "chunk": [min(c, n) for c, n in zip(CTX, [1, 7, 16, 5, 64, 1, 100, 128, 129, 200, 257])],
           "single": [1] * len(CTX)}[mode]
    prefill(make_case(31, CTX, new, 4, 2, D, B, dtype), dev)


@pytest.mark.parametrize("group", [1, 3, 5, 7, 8, 16, 33, 64, 100, 128])
@pytest.mark.parametrize("D", [64, 128])
def test_prefill_groups(dev, group, D):
    prefill(make_case(32, [40, 1, 150, 0], [40, 1, 70, 0], 2 * group if group < 64 else group,
                      2 if group < 64 else 1, D, 16, BF16), dev)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("window,prefix", [(0, None), (1, None), (100, None), (300, [4] * 5), (0, [0, 1, 40, 200, 999]),
                                           (33, [0, 17, 16, 300, 130])])
@pytest.mark.parametrize("cap,alibi", [(0.0, False), (20.0, False), (0.0, True), (5.0, True)])
def test_prefill_options(dev, dtype, window, prefix, cap, alibi):
    ctx, new = [1, 130, 64, 400, 700], [1, 130, 20, 333, 150]
    c = make_case(33, ctx, new, 6, 2, 128, 16, dtype, window=window, prefix=prefix, cap=cap, alibi=alibi,
                  q_scale=2.0)
    prefill(c, dev)


@pytest.mark.parametrize("B", [8, 32])
def test_prefill_options_other_shapes(dev, B):
    c = make_case(34, [9, 500, 260], [9, 300, 2], 10, 2, 64, B, F16, window=120, prefix=[3, 200, 50], cap=8.0,
                  alibi=True)
    prefill(c, dev)


def test_prefill_few_queries_of_long_contexts(dev):
    prefill(make_case(35, [9000, 5000], [3, 5], 8, 1, 128, 16, BF16), dev)
    prefill(make_case(36, [7001], [130], 4, 2, 64, 32, F16, window=2000, prefix=[5]), dev)


def test_prefill_many_short_prompts(dev):
    g = torch.Generator().manual_seed(6)
    ctx = torch.randint(0, 130, (96,), generator=g).tolist()
    c = make_case(37, ctx, ctx, 8, 4, 128, 16, BF16)
    d = to_dev(c, dev)
    for _ in range(3):
        got = run_prefill(c, d)
        assert pa.device_errors() == 0
    check(c, got, True)


def test_prefill_scales_and_profiles(dev):
    prefill(make_case(38, [300], [300], 4, 2, 128, 16, F16, scale=-0.1), dev)
    prefill(make_case(38, [300], [300], 4, 2, 128, 16, F16, scale=0.0), dev)
    for kind in range(4):
        c = make_case(39, [600], [200], 4, 2, 128, 16, F16)
        j = torch.arange(600).float()
        prof = [j / 20, 30 - j / 20, torch.where(j == 577, 30.0, 0.0), (j % 64) / 2][kind]
        for i in range(600):
            c.k_cache[int(c.tables[0, i // 16]), :, i % 16, 0] = prof[i]
        c.q[:, :, 0] = 11.0
        prefill(c, dev, f"profile {kind}")


def test_prefill_leaves_other_rows_alone(dev):
    c = make_case(40, [40, 90, 20], [40, 30, 20], 4, 2, 128, 16, BF16)
    d = to_dev(c, dev)
    want, bound = reference(c, True)
    # rows behind the last sequence, and rows of a sequence with a bad length
    q = torch.cat([d["q"], torch.full((7, 4, 128), float("nan"), dtype=BF16, device=dev)])
    out = torch.full_like(q, 7.0)
    d["lens"][1] = 29                                  # fewer keys than queries
    pa.prefill_grouped(out, q, d["k_cache"], d["v_cache"], d["tables"], d["lens"], d["starts"], c.scale,
                       max_query_len=40)
    assert pa.device_errors() == pa.DEVERR_CONTEXT
    assert (out[90:] == 7.0).all() and (out[40:70] == 7.0).all()
    for r in (slice(0, 40), slice(70, 90)):
        assert ((out[r].cpu().double() - want[r]).abs() <= bound[r]).all()
    # an understated max_query_len
    out.fill_(7.0)
    d["lens"][1] = 90
    pa.prefill_grouped(out, q, d["k_cache"], d["v_cache"], d["tables"], d["lens"], d["starts"], c.scale,
                       max_query_len=30)
    assert pa.device_errors() == pa.DEVERR_CONTEXT
    assert (out[:40] == 7.0).all() and (out[40:90] != 7.0).any()
    # query_start out of range
    out.fill_(7.0)
    bad = torch.tensor([0, 40, 30, 500], dtype=torch.int32, device=dev)
    pa.prefill_grouped(out, q, d["k_cache"], d["v_cache"], d["tables"], d["lens"], bad, c.scale,
                       max_query_len=40)
    assert pa.device_errors() == pa.DEVERR_CONTEXT
    assert (out[40:] == 7.0).all() and (out[:40] != 7.0).any()


def test_prefill_bad_entry_is_left_out(dev):
    c = make_case(41, [64], [10], 4, 2, 128, 16, F16)
    d = to_dev(c, dev)
    d["tables"][0, 1] = c.k_cache.shape[0]
    got = run_prefill(c, d)
    assert pa.device_errors() == pa.DEVERR_TABLE
    # the same attention without keys 16 .. 31, over a table without that block
    # (every query sits past them, so only the positions shift)
    c2 = make_case(41, [64], [10], 4, 2, 128, 16, F16)
    c2.tables[0, :3] = c.tables[0, [0, 2, 3]]
    c2.ctx, c2.lens = [48], torch.tensor([48], dtype=torch.int32)
    check(c2, got, True, "bad entry")


def test_prefill_in_graphs_and_reproducible(dev):
    cases = [make_case(42 + i, [500, 3000], [200, 4], 8, 2, 128, 16, BF16) for i in range(2)]
    ds = [to_dev(c, dev) for c in cases]
    outs = [torch.zeros_like(d["q"]) for d in ds]
    first = [run_prefill(c, d) for c, d in zip(cases, ds)]
    side = torch.cuda.Stream(dev)
    torch.cuda.synchronize()
    graphs = []
    for c, d, o in zip(cases, ds, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            run_prefill(c, d, o)
        graphs.append(g)
    streams = [torch.cuda.Stream(dev) for _ in range(2)]
    for _ in range(10):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for f, o in zip(first, outs):
            assert torch.equal(f, o)
    for c, f in zip(cases, first):
        check(c, f, True)
    assert pa.device_errors() == 0


# ------------------------------------------------------------------ extremes

@pytest.mark.parametrize("cap", [0.5, 1000.0, 1e6])
def test_small_and_large_caps(dev, cap):
    """Scores far past a small cap, and a cap so large that it does nothing."""
    decode(make_case(70, [90, 300], [1, 1], 8, 2, 128, 16, F16, cap=cap, q_scale=3.0), dev)
    prefill(make_case(71, [90, 300], [90, 40], 8, 2, 128, 16, BF16, cap=cap, q_scale=3.0), dev)


@pytest.mark.parametrize("window", [2 ** 31 - 1, 1023, 1024])
def test_windows_as_long_as_the_context(dev, window):
    c = make_case(72, [1024, 700, 3], [1] * 3, 6, 2, 64, 16, F16, window=window)
    decode(c, dev)
    prefill(make_case(73, [1024, 300], [600, 300], 6, 2, 64, 16, F16, window=window), dev)


def test_values_that_no_query_sees(dev):
    """NaN and infinities in keys outside a decode's window, in slots past the
    context, and (keys) in front of a prompt's later rows."""
    c = make_case(74, [300], [1], 8, 2, 128, 16, BF16, window=40)
    for j in range(260):
        blk = int(c.tables[0, j // 16])
        if blk >= 0:
            c.k_cache[blk, :, j % 16] = float("nan")
            c.v_cache[blk, :, j % 16] = float("inf")
    got = run_decode(c, to_dev(c, dev))
    assert pa.device_errors() == 0
    keep = torch.arange(260, 300)
    blk, off = c.tables[0, keep // 16].long(), keep % 16
    for h in range(2):
        K, V = c.k_cache[blk, h, off].double(), c.v_cache[blk, h, off].double()
        for g in range(4):
            w = torch.softmax(c.q[0, 4 * h + g].double() @ K.T * c.scale, -1)
            o, mag = w @ V, w @ V.abs()
            # the fp32 dot product's part of the bound, and the output's rounding
            tol = 2.0 ** -8 * o.abs() + 2e-3 * mag
            assert ((got[0, 4 * h + g].cpu().double() - o).abs() <= tol).all()


def test_nan_queries_stay_in_their_rows(dev):
    c = make_case(75, [70, 200], [70, 33], 6, 2, 128, 16, F16)
    d = to_dev(c, dev)
    d["q"][10, 3] = float("nan")
    got = run_prefill(c, d)
    assert torch.isnan(got[10, 3]).all()
    got[10, 3] = run_prefill(c, to_dev(c, dev))[10, 3]
    check(c, got, True)
    c = make_case(76, [70, 200], [1, 1], 6, 2, 128, 16, F16)
    d = to_dev(c, dev)
    d["q"][1, 2] = float("nan")
    got = run_decode(c, d)
    assert torch.isnan(got[1, 2]).all()
    got[1, 2] = run_decode(c, to_dev(c, dev))[1, 2]
    check(c, got, False)


def test_caches_past_32_bit_offsets(dev):
    """Blocks at the end of a pool of more than 2^32 bytes and 2^31 elements."""
    H, B, D = 8, 16, 128
    N = 2 ** 31 // (H * B * D) + 64
    kc = torch.empty(N, H, B, D, dtype=F16, device=dev)
    vc = torch.empty(N, H, B, D, dtype=F16, device=dev)
    assert kc.numel() > 2 ** 31
    c = make_case(77, [50, 90], [1, 33], 16, H, D, B, F16, extra_blocks=0)
    n = c.k_cache.shape[0]
    kc[N - n:], vc[N - n:] = c.k_cache.to(dev), c.v_cache.to(dev)
    d = to_dev(c, dev)
    d["k_cache"], d["v_cache"] = kc, vc
    d["tables"] = torch.where((d["tables"] >= 0) & (d["tables"] < n), d["tables"] + (N - n), d["tables"])
    got = run_prefill(c, d)
    check(c, got, True)
    c2 = make_case(77, [50, 90], [1, 1], 16, H, D, B, F16, extra_blocks=0)
    d2 = dict(d, q=c2.q.to(dev))
    c2.k_cache, c2.v_cache, c2.tables = c.k_cache, c.v_cache, c.tables
    check(c2, run_decode(c2, d2), False)
    q = torch.randn(3, 16, D, device=dev).to(F16)
    k, v = torch.randn(3, H, D, device=dev).to(F16), torch.randn(3, H, D, device=dev).to(F16)
    slots = torch.tensor([N * B - 1, N * B - 17, (N - 1) * B], dtype=torch.int32, device=dev)
    pos = torch.zeros(3, dtype=torch.int32, device=dev)             # angle 0: K as it is
    pa.rope_and_cache(torch.empty_like(q), q, k, v, kc, vc, pos, pa.rope_table(4, 128, device=dev), slots)
    assert torch.equal(kc[N - 1, :, 15], k[0]) and torch.equal(vc[N - 2, :, 15], v[1])
    assert torch.equal(kc[N - 1, :, 0], k[2])
    assert pa.device_errors() == 0


def test_decode_at_the_edges_of_a_cta_s_piece(dev):
    """Every way a context can meet the pieces: many of one tile, one of many,
    sequences of no tokens between them."""
    g = torch.Generator().manual_seed(8)
    for seed, S in ((80, 33), (81, 600)):
        ctx = [0 if torch.rand(1, generator=g) < 0.3 else int(torch.randint(1, 90, (1,), generator=g)) for _ in range(S)]
        ctx[S // 2] = 5000
        decode(make_case(seed, ctx, [1] * S, 4, 2, 128, 16, F16), dev)
    decode(make_case(82, [0, 0, 0], [1] * 3, 4, 2, 128, 16, F16), dev)


def test_single_tokens_prefill_like_decode(dev):
    """One new token per sequence through both calls."""
    c = make_case(83, [1, 64, 65, 700], [1] * 4, 8, 2, 128, 16, F16, alibi=True)
    d = to_dev(c, dev)
    a, b = run_decode(c, d), run_prefill(c, d)
    check(c, a, False)
    check(c, b, True)


# ------------------------------------------------------------------ rope

def rope_inputs(seed, T, Hq, H, D, B, rot, dtype, packed, far=5000):
    g = torch.Generator().manual_seed(seed)
    if packed:
        qkv = torch.randn(T, (Hq + 2 * H) * D, generator=g).to(dtype)
    else:
        qkv = [torch.randn(T, h * D, generator=g).to(dtype) for h in (Hq, H, H)]
    pos = torch.randint(0, far, (T,), generator=g).to(torch.int32)
    N = -(-T // B) + 2
    slots = torch.randperm(N * B, generator=g)[:T].to(torch.int32)
    return qkv, pos, slots, N, pa.rope_table(far, rot)


def split(qkv, Hq, H, D, packed):
    if packed:
        T = qkv.shape[0]
        x = qkv.view(T, Hq + 2 * H, D)
        return x[:, :Hq], x[:, Hq:Hq + H], x[:, Hq + H:]
    return tuple(t.view(t.shape[0], -1, D) for t in qkv)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,Hq,H,D,B,rot,packed", [
    (1, 32, 8, 128, 16, 128, True), (1, 1, 1, 64, 8, 16, False), (33, 6, 2, 64, 32, 64, True),
    (257, 7, 1, 256, 16, 256, True), (100, 12, 4, 64, 16, 32, False), (5, 71, 1, 64, 16, 48, True),
    (64, 8, 8, 128, 8, 80, False), (2000, 4, 2, 128, 16, 128, True), (1500, 24, 8, 64, 16, 64, False)])
def test_rope(dev, dtype, interleaved, T, Hq, H, D, B, rot, packed):
    qkv, pos, slots, N, table = rope_inputs(50, T, Hq, H, D, B, rot, dtype, packed)
    if T > 4:
        slots[3] = -1              # no K / V
        pos[1] = -1                # padding
        pos[2], slots[2] = -4, -1
    dq = qkv.to(dev) if packed else [t.to(dev) for t in qkv]
    q, k, v = split(dq, Hq, H, D, packed)
    kc = torch.full((N, H, B, D), 3.0, dtype=dtype, device=dev)
    vc = torch.full((N, H, B, D), 5.0, dtype=dtype, device=dev)
    qo = torch.full((T, Hq, D), 9.0, dtype=dtype, device=dev)
    pa.rope_and_cache(qo, q, k, v, kc, vc, pos.to(dev), table.to(dev), slots.to(dev), interleaved=interleaved)
    assert pa.device_errors() == 0
    q64, k64, v64 = (x.double() for x in split(qkv, Hq, H, D, packed))
    live = pos >= 0
    cs = table[pos.clamp(min=0).long()].double()
    wq, mq = rotate(q64, cs[:, :rot // 2], cs[:, rot // 2:], interleaved)
    wk, mk = rotate(k64, cs[:, :rot // 2], cs[:, rot // 2:], interleaved)
    bq, bk = rope_bound(wq, mq, dtype), rope_bound(wk, mk, dtype)
    wq[~live], bq[~live] = 9.0, 0.0
    got = qo.cpu().double()
    assert ((got - wq).abs() <= bq).all()
    assert torch.equal(got[live][..., rot:], q64[live][..., rot:])
    want_k, bound_k = torch.full((N * B, H, D), 3.0).double(), torch.zeros(N * B, H, D).double()
    want_v = torch.full((N * B, H, D), 5.0).double()
    keep = live & (slots >= 0)
    at = slots[keep].long()
    want_k[at], bound_k[at], want_v[at] = wk[keep], bk[keep], v64[keep]
    flat = lambda c: c.cpu().double().permute(0, 2, 1, 3).reshape(N * B, H, D)
    assert ((flat(kc) - want_k).abs() <= bound_k).all()
    assert torch.equal(flat(vc), want_v)
    # in place gives the same bits
    pa.rope_and_cache(q, q, k, v, kc, vc, pos.to(dev), table.to(dev), slots.to(dev), interleaved=interleaved)
    assert torch.equal(q[live.to(dev)], qo[live.to(dev)])


def test_rope_errors(dev):
    qkv, pos, slots, N, table = rope_inputs(51, 8, 4, 2, 64, 16, 64, F16, True)
    pos[5], slots[6] = 5000, N * 16
    q, k, v = split(qkv.to(dev), 4, 2, 64, True)
    kc = torch.zeros(N, 2, 16, 64, dtype=F16, device=dev)
    vc, qo = torch.zeros_like(kc), torch.full((8, 4, 64), 9.0, dtype=F16, device=dev)
    args = (kc, vc, pos.to(dev), table.to(dev), slots.to(dev))
    pa.rope_and_cache(qo, q, k, v, *args)
    assert pa.device_errors() == pa.DEVERR_POSITION | pa.DEVERR_SLOT
    assert (qo[5] == 9.0).all() and (qo[6] != 9.0).any() and (qo[4] != 9.0).any()
    x = qkv.to(dev).view(8, 8, 64)
    with pytest.raises(ValueError):
        pa.rope_and_cache(x[:, 2:6], x[:, :4], k, v, *args)        # overlaps q
    with pytest.raises(ValueError):
        pa.rope_and_cache(x[:, 4:], x[:, :4], x[:, 4:6], x[:, 6:], *args)     # overlaps k and v
    with pytest.raises(ValueError):
        pa.rope_and_cache(qo, q, k, v[:4], *args)
    with pytest.raises(ValueError):
        pa.rope_and_cache(qo, q.transpose(0, 1), k, v, *args)
    with pytest.raises(TypeError):
        pa.rope_and_cache(qo, q.float(), k, v, *args)
    with pytest.raises(pa.PaError):
        pa.rope_and_cache(qo, q, k, v, kc, vc, args[2], pa.rope_table(5000, 24, device=dev), args[4])


def test_marshalled_calls_leave_odd_ones_to_the_checks(dev):
    """What the marshalling module does not take as it stands gets the Python
    checks' answer: an error, or the call made another way."""
    c = make_case(60, [40, 7], [1, 1], 4, 2, 64, 16, F16)
    d = to_dev(c, dev)
    out = torch.empty_like(d["q"])
    args = [out, d["q"], d["k_cache"], d["v_cache"], d["tables"], d["lens"], c.scale]

    def refused(kind, i, value, **kw):
        bad = list(args)
        bad[i] = value
        with pytest.raises(kind):
            pa.decode_grouped(*bad, **kw)

    refused(ValueError, 0, out[:1])
    refused(TypeError, 1, d["q"].float())
    refused(ValueError, 1, c.q)                                    # on the host
    refused(TypeError, 2, d["k_cache"].float())
    refused(ValueError, 3, d["v_cache"][:-1])
    refused(ValueError, 3, d["v_cache"].transpose(2, 3))
    refused(TypeError, 4, d["tables"].long())
    refused(ValueError, 5, d["lens"][:1])
    refused(ValueError, 5, d["lens"].repeat(4)[::4])               # strided
    refused(TypeError, 5, None)
    refused(ValueError, 6, c.scale, alibi_slopes=torch.ones(3, device=dev))
    refused(TypeError, 6, c.scale, prefix_lens=torch.zeros(2, device=dev))
    refused(pa.PaError, 6, c.scale, window=-1)
    refused(pa.PaError, 6, c.scale, softcap=-2.0)
    refused(pa.PaError, 6, float("nan"))
    refused(pa.PaError, 6, c.scale, workspace=torch.empty(16, dtype=torch.uint8, device=dev),
            counters=torch.zeros(8192, dtype=torch.int32, device=dev))
    empty = [t[:0] for t in (out, d["q"])] + args[2:4] + [d["tables"][:0], d["lens"][:0], c.scale]
    assert pa.decode_grouped(*empty).shape[0] == 0
    assert pa.device_errors() == 0
    check(c, run_decode(c, d), False)
    none = torch.empty(0, 4, 64, dtype=F16, device=dev)
    kv = torch.empty(0, 2, 64, dtype=F16, device=dev)
    i0 = torch.empty(0, dtype=torch.int32, device=dev)
    pa.rope_and_cache(none, none, kv, kv, d["k_cache"], d["v_cache"], i0, pa.rope_table(8, 64, device=dev), i0)
    pa.prefill_grouped(none, none, d["k_cache"], d["v_cache"], d["tables"][:0], d["lens"][:0],
                       torch.zeros(1, dtype=torch.int32, device=dev), c.scale)
    assert pa.device_errors() == 0


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("dtype,window,cap", [(F16, 0, 0.0), (BF16, 48, 30.0)])
def test_prompt_then_tokens(dev, dtype, window, cap):
    """A layer's prompt and its next tokens, through the block manager: append
    with rotation and prefill, then one token at a time with decode, against
    fp64 attention over what the caches hold."""
    Hq, H, D, B, rot = 8, 2, 128, 16, 128
    mgr = pa.KVManager(64, B, 16, shuffle_seed=3)
    lens = [37, 100, 5]
    ids = [mgr.add_sequence(n) for n in lens]
    g = torch.Generator().manual_seed(9)
    kc = torch.full((64, H, B, D), float("nan"), dtype=dtype, device=dev)
    vc = kc.clone()
    table = pa.rope_table(400, rot, device=dev)
    scale = D ** -0.5

    def append(T, pos, slots):
        qkv = torch.randn(T, Hq + 2 * H, D, generator=g).to(dtype).to(dev)
        q = torch.empty(T, Hq, D, dtype=dtype, device=dev)
        pa.rope_and_cache(q, qkv[:, :Hq], qkv[:, Hq:Hq + H], qkv[:, Hq + H:], kc, vc,
                          torch.tensor(pos, dtype=torch.int32, device=dev), table,
                          torch.tensor(slots, dtype=torch.int32, device=dev))
        return q

    def verify(q, out, new, weights16, what):
        c = make_case(0, [1], [1], Hq, H, D, B, dtype)
        tb, ln = mgr.block_tables(ids)
        c.ctx, c.new = ln.tolist(), new
        c.starts_list = [0]
        for n in new:
            c.starts_list.append(c.starts_list[-1] + n)
        c.tables, c.q, c.window, c.cap, c.scale = torch.from_numpy(tb), q.cpu(), window, cap, scale
        c.k_cache, c.v_cache = kc.cpu(), vc.cpu()
        check(c, out, weights16, what)

    pos = [p for n in lens for p in range(n)]
    q = append(sum(lens), pos, [mgr.slot(i, t) for i, n in zip(ids, lens) for t in range(n)])
    tb, ln = mgr.block_tables(ids)
    starts = torch.tensor([0, 37, 137, 142], dtype=torch.int32, device=dev)
    out = torch.empty_like(q)
    pa.prefill_grouped(out, q, kc, vc, torch.from_numpy(tb).to(dev), torch.from_numpy(ln).to(dev), starts, scale,
                       max_query_len=100, softcap=cap, window=window)
    assert pa.device_errors() == 0
    verify(q, out, lens, True, "prompt")
    for step in range(20):
        slots = []
        for i in ids:
            slot, src, dst = mgr.append(i)
            slots.append(slot)
        tb, ln = mgr.block_tables(ids)
        q = append(3, (ln - 1).tolist(), slots)
        out = torch.empty_like(q)
        pa.decode_grouped(out, q, kc, vc, torch.from_numpy(tb).to(dev), torch.from_numpy(ln).to(dev), scale,
                          softcap=cap, window=window)
        assert pa.device_errors() == 0
        verify(q, out, [1, 1, 1], False, f"step {step}")
