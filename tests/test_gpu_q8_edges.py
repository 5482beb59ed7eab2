"""GPU tests of the 8-bit cache's calls at the ends of their ranges and where their
kernels change form.  References and bounds as in q8_ref and grouped_ref."""
import math

import pytest
import torch

import paged_kv_cache_269_gb300 as pa
import test_gpu_grouped
from grouped_ref import make_case
from paged_kv_cache_269_gb300 import grouped
from q8_ref import E4M3, make_q8_case, refresh, scales_for
from test_gpu_q8 import check, decode, prefill, run_prefill, to_dev

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16
BYTE = torch.uint8


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    d = torch.device("cuda", 0)
    torch.cuda.set_device(d)
    pa.lib()
    pa.device_errors()
    return d


def processors(dev):
    return torch.cuda.get_device_properties(dev).multi_processor_count


# ------------------------------------------------------------------ sizes of queries

# Rows of about 2^-down: fp32 holds the power of two that brings them to fp16's range down
# to 2^-116; bf16 numbers end at 2^-133.
DOWN = [88, 100, 110, 117, 124, 126, 128, 130]


def small_queries(seed, ctx, new, heads, down, cap=0.0, **kw):
    """Rows of about 2^-down, with scales that give scores of the usual size: the softmax
    scale is 2^90 times the usual one (past 2^100 it is refused), K's the rest."""
    c = make_q8_case(seed, ctx, new, *heads, 128, 16, BF16, cap=cap, **kw)
    c.q = torch.ldexp(c.q.double(), torch.tensor(-down)).to(BF16)
    c.scale = 128 ** -0.5 * 2.0 ** min(90, down)
    c.ks = c.ks * 2.0 ** max(down - 90, 0)
    refresh(c)
    assert (c.ks >= 2.0 ** -60).all() and (c.ks <= 2.0 ** 60).all() and c.q.abs().max() < 2.0 ** (4 - down)
    return c


@pytest.mark.parametrize("down", DOWN)
@pytest.mark.parametrize("cap", [0.0, 12.0])
def test_decode_of_the_smallest_queries(dev, down, cap):
    decode(small_queries(201, [50, 300, 1], [1] * 3, (8, 2), down, cap), dev)
    c = small_queries(202, [400, 77], [1] * 2, (12, 2), down, cap, alibi=True)
    c.q[0, 3] = 0.0
    c.q[1, 2, 5] = 2.0 ** (7 - down)                  # one element far above the others
    decode(c, dev)


@pytest.mark.parametrize("down", DOWN)
@pytest.mark.parametrize("cap", [0.0, 12.0])
def test_prefill_of_the_smallest_queries(dev, down, cap):
    prefill(small_queries(203, [300, 77], [300, 5], (8, 2), down, cap), dev)
    c = small_queries(204, [200], [150], (4, 2), down, cap, alibi=True)
    c.q[7] = 0.0
    c.q[11, 2, 5] = 2.0 ** (7 - down)
    prefill(c, dev)


# ------------------------------------------------------------------ appends without q or a rotation

class Watched:
    """The marshalling module, with what its append returned."""

    def __init__(self, module):
        self.module, self.seen = module, []

    def norm_rope(self, *args):
        self.seen.append(self.module.norm_rope(*args))
        return self.seen[-1]


@pytest.mark.parametrize("q8", [True, False])
@pytest.mark.parametrize("T", [1, 45])
@pytest.mark.parametrize("with_q,turn,placed", [(False, False, False), (False, False, True), (False, True, True),
                                                (True, False, False), (True, False, True), (True, True, True)])
def test_append_without_q_or_rotation_is_marshalled(dev, monkeypatch, q8, T, with_q, turn, placed):
    """These forms go through the compiled marshalling too, and do what they do through the
    Python checks, bit for bit."""
    H, D, B, N = 2, 64, 16, 5
    g = torch.Generator().manual_seed(T)
    x = torch.randn(T, 3 + 2 * H, D, generator=g).to(BF16).to(dev)
    pos = torch.randint(-1, 50, (T,), generator=g).to(torch.int32).to(dev) if placed else None
    table = pa.rope_table(50, 32, device=dev) if turn else None
    slots = torch.randperm(N * B, generator=g)[:T].to(torch.int32).to(dev)
    w = (1.0 + 0.1 * torch.randn(D, generator=g)).to(dev)
    s = scales_for(1, H).to(dev) if q8 else None
    pa.device_errors()
    grouped._pa()
    watched, got = Watched(grouped._marshal), []
    for module in (watched, None):
        monkeypatch.setattr(grouped, "_marshal", module)
        out = torch.full((T, 3, D), 7.0, dtype=BF16, device=dev) if with_q else None
        kc, vc = (torch.zeros(N, H, B, D, dtype=BYTE if q8 else BF16, device=dev) for _ in range(2))
        a, b = (c.view(E4M3) if q8 else c for c in (kc, vc))
        r = pa.norm_rope_and_cache(out, x[:, :3] if with_q else None, x[:, 3:3 + H], x[:, 3 + H:], a, b, pos, table, slots,
                                   w if with_q else None, w, 1e-5, True, s, s)
        assert r is out and pa.device_errors() == 0
        got.append((kc.view(BYTE), vc.view(BYTE)) + (() if out is None else (out.view(BYTE),)))
    assert watched.seen == [0]
    assert all(torch.equal(m, p) for m, p in zip(*got)) and got[0][0].any()


def test_append_without_q_or_rotation_refuses(dev):
    H, D = 2, 64
    x = torch.zeros(4, 2 * H + 3, D, dtype=F16, device=dev)
    kc, vc = (torch.zeros(3, H, 16, D, dtype=BYTE, device=dev).view(E4M3) for _ in range(2))
    s, slots = torch.ones(H, device=dev), torch.arange(4, dtype=torch.int32, device=dev)
    table = pa.rope_table(9, D, device=dev)
    base = dict(q_out=None, q=None, k=x[:, :H], v=x[:, H:2 * H], k_cache=kc, v_cache=vc, positions=None, cos_sin=None,
                slot_mapping=slots, k_scales=s, v_scales=s)
    for kind, kw in ((ValueError, dict(q=x[:, 2 * H:])), (ValueError, dict(q_out=x[:, 2 * H:])),
                     (ValueError, dict(cos_sin=table)), (ValueError, dict(positions=slots[:3])),
                     (TypeError, dict(positions=slots.long())), (TypeError, dict(cos_sin=table.double(), positions=slots)),
                     (ValueError, dict(cos_sin=table[:, :0], positions=slots)), (TypeError, dict(k=None)),
                     (ValueError, dict(v=x[:3, :H])), (TypeError, dict(slot_mapping=None)), (TypeError, dict(v_scales=None))):
        with pytest.raises(kind):
            pa.norm_rope_and_cache(**{**base, **kw})
    for name in ("q", "k", "v"):                      # the rotary append takes none of them away
        full = dict(q_out=x[:, 4:].clone(), q=x[:, 4:], k=x[:, :H], v=x[:, H:2 * H])
        c16 = torch.zeros(3, H, 16, D, dtype=F16, device=dev)
        with pytest.raises(TypeError):
            pa.rope_and_cache(**{**full, name: None}, k_cache=c16, v_cache=c16.clone(), positions=slots, cos_sin=table,
                              slot_mapping=slots)
    with pytest.raises(TypeError):
        pa.rope_and_cache(x[:, 4:].clone(), x[:, 4:], x[:, :H], x[:, H:2 * H], c16, c16.clone(), slots, None, slots)
    assert pa.norm_rope_and_cache(**base) is None and pa.device_errors() == 0


# ------------------------------------------------------------------ short contexts

@pytest.mark.parametrize("group,D,tiles", [(1, 64, 12), (4, 128, 8), (4, 256, 20), (8, 128, 12), (16, 64, 12),
                                           (16, 128, 8)])
@pytest.mark.parametrize("rounds", [1, 2, 3])
def test_decode_of_short_contexts_around_full_rounds(dev, group, D, tiles, rounds):
    """As many units as CTAs (two or three a processor) and a sequence more, twice and three
    times as many, and less than a round: cut or whole, each context's rows are right."""
    H, TK = 4, 4096 // D
    full = rounds * processors(dev) * (3 if D <= 128 and group <= 8 else 2) // H
    for S in (full, full * 9 // 10) if rounds == 2 else (full + 1,):
        g = torch.Generator().manual_seed(S)
        ctx = torch.randint(TK * tiles * 7 // 10, TK * tiles + 1, (S,), generator=g).tolist()
        ctx[S // 3] = TK * tiles
        decode(make_q8_case(231, ctx, [1] * S, H * group, H, D, 16, BF16), dev)


# ------------------------------------------------------------------ the prefill's queue

def items(c):
    """Work items of a prefill without key splits: pairs of tiles of the longest query, for
    every sequence and K/V head."""
    pair = 2 * (128 // (c.q_heads // c.kv_heads))
    return -(-max(c.new) // pair) * len(c.ctx) * c.kv_heads


def assert_ordered(c, dev, ordered=True):
    """Items are taken by falling numbers of keys with up to 32 sequences, no distance bias
    and one to four rounds of processors."""
    n, sms = items(c), processors(dev)
    assert (sms < n <= 4 * sms and 1 < len(c.ctx) <= 32) == ordered and n > sms, (n, sms)


CTX = [900, 1500, 33, 1500, 0, 1200, 700]
NEW = [900, 300, 33, 1500, 0, 257, 1]


@pytest.mark.parametrize("heads,B,dtype", [((8, 8), 16, F16), ((12, 4), 8, BF16), ((14, 7), 32, BF16)])
def test_prefill_in_order_of_keys(dev, heads, B, dtype):
    c = make_q8_case(211, CTX, NEW, *heads, 64, B, dtype)
    assert_ordered(c, dev)
    prefill(c, dev)
    c = make_q8_case(212, CTX, NEW, *heads, 128, B, dtype, window=300, prefix=[0, 40, 5, 0, 0, 1000, 3], cap=9.0)
    assert_ordered(c, dev)
    prefill(c, dev)


@pytest.mark.parametrize("heads", [(16, 16), (24, 8)])
def test_prefill_by_levels_past_four_rounds(dev, heads):
    c = make_q8_case(213, CTX, NEW, *heads, 64, 16, F16)
    assert_ordered(c, dev, ordered=False)
    prefill(c, dev)


@pytest.mark.parametrize("ctx,new", [
    ([512] * 5, [512] * 5),                                     # every end in every sequence
    ([0, 700, 700, 0, 444, 700, 0], [0, 700, 444, 0, 444, 1, 0]),   # the first and the last are empty
    ([768, 512, 1024, 256, 1280], [768, 512, 1024, 256, 1280]),     # whole pairs: all ends meet
    ([2000, 1, 1999, 1], [1000, 1, 999, 1])])
def test_prefill_in_order_of_ends_that_meet(dev, ctx, new):
    S = len(ctx)
    H = -(-(processors(dev) + 1) // (-(-max(new) // 256) * S))
    c = make_q8_case(214, ctx, new, H, H, 64, 16, BF16)
    assert_ordered(c, dev)
    prefill(c, dev)


def test_prefill_in_order_of_32_sequences(dev):
    g = torch.Generator().manual_seed(5)
    ctx = torch.randint(1, 200, (32,), generator=g).tolist()
    ctx[31] = 500
    new = [min(c, int(n)) for c, n in zip(ctx, torch.randint(0, 200, (32,), generator=g))]
    new[31] = 500
    c = make_q8_case(215, ctx, new, 4, 2, 64, 16, F16)
    assert_ordered(c, dev)
    prefill(c, dev)


@pytest.mark.parametrize("who", [0, 3, 6])
@pytest.mark.parametrize("fault", ["short", "long", "rows", "longest"])
def test_prefill_in_order_with_a_rejected_sequence(dev, who, fault):
    """A sequence whose lengths are inconsistent is flagged and its rows are left; the
    others' rows are what they are without it, to the bit."""
    ctx = [900, 1500, 33, 1300, 0, 1200, 1000]
    new = [700, 300, 33, 701, 0, 257, 650]
    if fault == "longest":
        new[who] = 768                                # alone past max_query_len
    c = make_q8_case(216, ctx, new, 12, 12, 64, 16, BF16)
    d = to_dev(c, dev)
    assert_ordered(c, dev)
    good = run_prefill(c, d).cpu()
    assert pa.device_errors() == 0
    check(c, good, True)
    last = len(ctx) - 1
    kw = {}
    lost = {who}
    if fault == "short":
        d["lens"][who] = new[who] - 1
    elif fault == "long":
        d["lens"][who] = d["tables"].shape[1] * 16 + 1
    elif fault == "longest":
        kw["max_query_len"] = 767
    elif who == last:
        d["starts"][last + 1] += 1                    # a row past the last
    else:                                             # an end before its start, and what follows from it
        d["starts"][who + 1] = d["starts"][who] - 1
        lost = {who, who + 1}
        d["lens"][who + 1] = min(ctx[who + 1], new[who])    # shorter than the rows it now has
    out = torch.full_like(d["q"], 5.0)
    run_prefill(c, d, out, **kw)
    assert pa.device_errors() == pa.DEVERR_CONTEXT
    pa.reset_workspaces()
    out = out.cpu()
    for s in range(len(ctx)):
        r0, r1 = c.starts_list[s], c.starts_list[s + 1]
        assert (out[r0:r1] == 5).all() if s in lost else torch.equal(out[r0:r1], good[r0:r1]), s


# ------------------------------------------------------------------ joins of key splits

def parts(ctx, splits):
    """Parts that the item of a few queries over ctx keys is split into: one for every
    sqrt(n / 2) of its n tiles of 128 keys, of two such tiles at least."""
    count = -(-ctx // 64)
    per = math.ceil(2 * max(2.0, math.sqrt(count / 4)))
    return min(splits, -(-count // per))


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("cap,alibi", [(0.0, False), (20.0, True)])
def test_prefill_joins_few_and_many_splits(dev, bits, dtype, D, cap, alibi):
    """Up to four parts are joined in one round trip, more in a loop: items of 1 to 7 parts in
    one call, rows that end within a warp's, several warps' and a second tile's."""
    ctx = [60, 512, 700, 1024, 1300, 1600, 2300, 3200]
    assert [parts(n, 152 // len(ctx)) for n in ctx] == [1, 2, 3, 4, 5, 5, 6, 7]
    for new, heads in (([3, 1, 5, 2, 6, 1, 4, 5], (5, 1)), ([60, 43, 1, 40, 17, 33, 5, 16], (3, 1))):
        if bits == 8:
            prefill(make_q8_case(221, ctx, new, *heads, D, 16, dtype, cap=cap, alibi=alibi), dev)
        else:
            c = make_case(222, ctx, new, *heads, D, 16, dtype, cap=cap, alibi=alibi)
            got = test_gpu_grouped.run_prefill(c, test_gpu_grouped.to_dev(c, dev))
            assert pa.device_errors() == 0
            check(c, got, True)


# ------------------------------------------------------------------ read-backs that fill the device

def gather_case(seed, T, H, D, B, dtype, offset, dev, bad=None):
    """Random codes and slots, outputs that start `offset` elements past a 256-byte line;
    checked bit for bit against the definition, and what must not be written."""
    g = torch.Generator(device=dev).manual_seed(seed)
    N = 37
    kc, vc = (torch.randint(0, 256, (N, H, B, D), generator=g, device=dev).to(BYTE).view(E4M3) for _ in range(2))
    ks, vs = scales_for(1, H).to(dev), scales_for(2, H).to(dev)
    slots = torch.randint(-3, N * B, (T,), generator=g, device=dev).to(torch.int32)
    if bad is not None:
        slots[bad] = N * B
    base = [torch.full((T * H * D + 128,), -3.5, dtype=dtype, device=dev) for _ in range(2)]
    assert all(b.data_ptr() % 256 == 0 for b in base)
    ko, vo = (b[offset:offset + T * H * D].view(T, H, D) for b in base)
    pa.gather_cache_q8(ko, vo, kc, vc, ks, vs, slots)
    assert pa.device_errors() == (0 if bad is None else pa.DEVERR_SLOT)
    keep = (slots >= 0) & (slots < N * B)
    at = slots.clamp(0, N * B - 1).long()
    for o, b, c, s in ((ko, base[0], kc, ks), (vo, base[1], vc, vs)):
        want = (c.view(BYTE)[at // B, :, at % B].view(E4M3).float() * s[:, None]).to(dtype)
        want[~keep] = -3.5
        assert torch.equal(o.isnan(), want.isnan())
        assert torch.equal(o.nan_to_num(0.0).view(torch.int16), want.nan_to_num(0.0).view(torch.int16))
        assert (b[:offset] == -3.5).all() and (b[offset + T * H * D:] == -3.5).all()


def full_tokens(dev, H, D):
    """The tokens past which a read-back takes four chunks of 16 numbers a thread: the device
    is full of threads (8 CTAs of 256 a processor) by then."""
    return 8 * 256 * processors(dev) * 16 // (2 * H * D)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("H,D,B", [(1, 64, 16), (3, 64, 8), (5, 128, 16), (8, 128, 32), (3, 256, 32), (8, 256, 8), (40, 128, 16)])
@pytest.mark.parametrize("offset", [0, 8, 16, 24])
def test_gather_that_fills_the_device(dev, dtype, H, D, B, offset):
    # (offsets of 8 and 24 elements: rows on 16-byte and not on 32-byte lines)
    T = full_tokens(dev, H, D) + 1
    assert 2 * T * H * D // 16 > 8 * 256 * processors(dev)
    gather_case(1, T + 36, H, D, B, dtype, offset, dev, bad=T)
    if offset == 0:
        gather_case(2, T, H, D, B, dtype, offset, dev)
        gather_case(3, T - 1, H, D, B, dtype, offset, dev)      # the last with one chunk


@pytest.mark.parametrize("offset", [0, 8, 16, 24])
@pytest.mark.parametrize("T", [1, 7, 301])
def test_gather_to_any_aligned_output(dev, T, offset):
    gather_case(4, T, 3, 64, 16, F16, offset, dev)
    gather_case(5, T, 2, 128, 16, BF16, offset, dev, bad=T - 1)
