"""GPU parity of norm_rope_and_cache, reshape_and_cache_q8, gather_cache_q8,
decode_grouped_q8 and prefill_grouped_q8 against fp64, within the bounds derived
in q8_ref and grouped_ref."""
import pytest
import torch

import paged_kv_cache_269_gb300 as pa
from paged_kv_cache_269_gb300 import grouped
from grouped_ref import U, reference
from q8_ref import (E4M3, assert_codes, assert_rows, codes, make_q8_case, norm_rotate, refresh, scales_for, to_e4m3)

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16
BYTE = torch.uint8


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


# ------------------------------------------------------------------ append

class Append:
    """Inputs of an append on the CPU, and what it should leave behind."""

    def __init__(self, seed, T, Hq, H, D, B, dtype, rotary=None, norm=True, q8=True, interleaved=False, packed=True,
                 in_place=False, slots=None, positions=None, x_scale=1.0, eps=1e-6):
        g = torch.Generator().manual_seed(seed)
        self.T, self.Hq, self.H, self.D, self.B, self.dtype = T, Hq, H, D, B, dtype
        self.q8, self.interleaved, self.in_place, self.eps, self.packed = q8, interleaved, in_place, eps, packed
        self.qkv = (torch.randn(T, Hq + 2 * H, D, generator=g) * x_scale).to(dtype)
        rotary = D if rotary is None else rotary
        self.most = 300
        self.table = pa.rope_table(self.most, rotary) if rotary else None
        self.qw = 1.0 + 0.3 * torch.randn(D, generator=g) if norm else None
        self.kw = 1.0 + 0.3 * torch.randn(D, generator=g) if norm else None
        self.ks, self.vs = scales_for(seed, H, 0.004, 0.02), scales_for(seed + 1, H, 0.004, 0.02)
        self.N = -(-T // B) + 3
        self.slots = torch.randperm(self.N * B, generator=g)[:T].to(torch.int32) if slots is None else \
            torch.tensor(slots, dtype=torch.int32)
        self.positions = torch.randint(0, self.most, (T,), generator=g).to(torch.int32) if positions is None else \
            torch.tensor(positions, dtype=torch.int32)

    def run(self, dev, **kw):
        t = lambda x: None if x is None else x.to(dev)
        Hq, H = self.Hq, self.H
        qkv = self.qkv.to(dev)
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + H], qkv[:, Hq + H:]
        if not self.packed:
            q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
        out = q if self.in_place else torch.full((self.T, Hq, self.D), -77.0, dtype=self.dtype, device=dev)
        shape = (self.N, H, self.B, self.D)
        if self.q8:
            kc, vc = (torch.full(shape, 0x55, dtype=BYTE, device=dev).view(E4M3) for _ in range(2))
        else:
            kc, vc = (torch.full(shape, -55.0, dtype=self.dtype, device=dev) for _ in range(2))
        got = pa.norm_rope_and_cache(out, q, k, v, kc, vc, t(self.positions), t(self.table), t(self.slots), t(self.qw),
                                     t(self.kw), self.eps, self.interleaved, *((t(self.ks), t(self.vs)) if self.q8 else ()),
                                     **kw)
        assert got is out
        return out.cpu(), kc.cpu(), vc.cpu()

    def check(self, dev, flags=0, **kw):
        out, kc, vc = self.run(dev, **kw)
        assert pa.device_errors() == flags
        Hq, H, B = self.Hq, self.H, self.B
        pos_ok = (self.positions >= 0) & (self.positions < self.most)
        want, err = norm_rotate(self.qkv[:, :Hq], self.qw, self.eps, self.table, self.positions, self.interleaved)
        assert_rows(out[pos_ok], want[pos_ok], err[pos_ok], self.dtype, "q")
        left = self.qkv[:, :Hq] if self.in_place else torch.full_like(out, -77.0)
        assert torch.equal(out[~pos_ok], left[~pos_ok])
        keep = pos_ok & (self.slots >= 0) & (self.slots < self.N * B)
        at = self.slots[keep].long()
        kw_, ke = norm_rotate(self.qkv[:, Hq:Hq + H], self.kw, self.eps, self.table, self.positions, self.interleaved)
        v = self.qkv[:, Hq + H:]
        raw = BYTE if self.q8 else torch.int16
        for name, cache in (("k", kc), ("v", vc)):
            got = cache.view(raw)[at // B, :, at % B].view(cache.dtype)
            if name == "k" and self.q8:
                assert_codes(got, kw_[keep], ke[keep], self.ks, "k")
            elif name == "k":
                assert_rows(got, kw_[keep], ke[keep], self.dtype, "k")
            elif self.q8:     # the definition in fp32, bit for bit
                exact = (v[keep].float() / self.vs[:, None]).clamp(-448, 448).to(E4M3)
                assert torch.equal(got.view(BYTE), exact.view(BYTE))
            else:
                assert torch.equal(got.view(raw), v[keep].contiguous().view(raw))
            untouched = torch.ones(self.N * B, dtype=torch.bool)
            untouched[at] = False
            rest = cache.view(raw).permute(0, 2, 1, 3).reshape(self.N * B, H, self.D)[untouched]
            fill = 0x55 if self.q8 else torch.tensor([-55.0], dtype=self.dtype).view(raw).item()
            assert (rest == fill).all()


@pytest.mark.parametrize("q8", [True, False])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("D,B", [(64, 8), (64, 32), (128, 16), (128, 8), (256, 16), (256, 32)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_shapes(dev, q8, dtype, D, B, interleaved):
    Append(1, 37, 6, 2, D, B, dtype, q8=q8, interleaved=interleaved).check(dev)


@pytest.mark.parametrize("rotary", [0, 16, 48, 112, 128])
@pytest.mark.parametrize("norm,q8", [(True, True), (False, True), (True, False), (False, False)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_part_of_the_head(dev, rotary, norm, q8, interleaved):
    Append(2, 19, 5, 5, 128, 16, BF16, rotary=rotary, norm=norm, q8=q8, interleaved=interleaved).check(dev)


@pytest.mark.parametrize("heads", [(1, 1), (8, 1), (3, 3), (71, 1), (12, 4)])
@pytest.mark.parametrize("T", [1, 2, 130])
def test_append_heads_and_tokens(dev, heads, T):
    Append(3, T, *heads, 64, 16, F16, packed=False).check(dev)


def test_append_many_tokens(dev):
    # past 8 tokens a processor a block takes all rows of its token
    Append(4, 1300, 9, 3, 128, 16, BF16, rotary=64).check(dev)
    Append(4, 1300, 9, 3, 256, 16, F16, norm=False, interleaved=True).check(dev)


@pytest.mark.parametrize("q8", [True, False])
@pytest.mark.parametrize("heads,D", [((5, 1), 64), ((7, 3), 128)])
def test_append_many_tokens_skips_and_flags(dev, q8, heads, D):
    T, g = 1501, torch.Generator().manual_seed(2)
    a = Append(13, T, *heads, D, 16, BF16, q8=q8, rotary=48)
    a.slots[torch.rand(T, generator=g) < 0.2] = -1
    a.slots[7::97] = a.N * 16
    a.positions[torch.rand(T, generator=g) < 0.2] = -5
    a.positions[3::101] = a.most
    a.check(dev, flags=pa.DEVERR_SLOT | pa.DEVERR_POSITION)
    a.slots[:], a.positions[:] = -1, -1                      # nothing to do for any token
    a.check(dev)


def test_append_many_tokens_of_k_and_v_alone(dev):
    T = 1400
    a = Append(14, T, 1, 3, 128, 8, F16, rotary=0, norm=False)
    a.slots[5::9] = -1
    kc, vc = (torch.zeros(a.N, 3, 8, 128, dtype=BYTE, device=dev).view(E4M3) for _ in range(2))
    pa.reshape_and_cache_q8(a.qkv[:, 1:4].to(dev), a.qkv[:, 4:].to(dev), kc, vc, a.ks.to(dev), a.vs.to(dev),
                            a.slots.to(dev))
    assert pa.device_errors() == 0
    keep = a.slots >= 0
    at = a.slots[keep].long()
    for cache, x, s in ((kc, a.qkv[:, 1:4], a.ks), (vc, a.qkv[:, 4:], a.vs)):
        want = (x[keep].float() / s[:, None]).clamp(-448, 448).to(E4M3).view(BYTE)
        assert torch.equal(cache.cpu().view(BYTE)[at // 8, :, at % 8], want)


@pytest.mark.parametrize("heads,D", [((40, 8), 256), ((100, 1), 256), ((226, 2), 256), ((250, 2), 256)])
def test_append_many_tokens_of_long_rows(dev, heads, D):
    # rows for which fewer CTAs fit a processor, and none: the same as in shorter calls
    Hq, H = heads
    T = 1300
    g = torch.Generator(device=dev).manual_seed(1)
    qkv = torch.randn(T, Hq + 2 * H, D, generator=g, device=dev).to(BF16)
    slots = torch.randperm(T, generator=g, device=dev).to(torch.int32)
    pos = torch.randint(0, 500, (T,), generator=g, device=dev).to(torch.int32)
    table, w = pa.rope_table(500, D, device=dev), 1 + 0.1 * torch.randn(D, generator=g, device=dev)
    s = scales_for(3, H).to(dev)
    got = []
    for step in (T, 600):
        out = torch.zeros(T, Hq, D, dtype=BF16, device=dev)
        kc, vc = (torch.zeros(-(-T // 16), H, 16, D, dtype=BYTE, device=dev).view(E4M3) for _ in range(2))
        for i in range(0, T, step):
            x = qkv[i:i + step]
            pa.norm_rope_and_cache(out[i:i + step], x[:, :Hq], x[:, Hq:Hq + H], x[:, Hq + H:], kc, vc, pos[i:i + step],
                                   table, slots[i:i + step], w, w, k_scales=s, v_scales=s)
        got.append((out, kc.view(BYTE), vc.view(BYTE)))
    assert pa.device_errors() == 0
    for x, y in zip(*got):
        assert torch.equal(x, y)


@pytest.mark.parametrize("packed", [True, False])
@pytest.mark.parametrize("q8", [True, False])
def test_append_in_place(dev, packed, q8):
    Append(5, 33, 8, 2, 128, 16, BF16, in_place=True, packed=packed, q8=q8).check(dev)
    Append(5, 1400, 4, 2, 64, 16, BF16, in_place=True, packed=packed, q8=q8).check(dev)


@pytest.mark.parametrize("q8", [True, False])
def test_append_skips_and_flags(dev, q8):
    n = 3 * 16 * 1       # slots of a pool of 4 blocks of 16
    a = Append(6, 12, 4, 2, 128, 16, F16, q8=q8, slots=[3, -1, 17, 9999, 0, 40, -5, 33, 12, 50, 51, 52],
               positions=[0, 5, -1, 7, 300, 299, 3, -9, 0, 1, 2, 3])
    assert a.N * 16 > 52 > n
    a.check(dev, flags=pa.DEVERR_SLOT | pa.DEVERR_POSITION)


def test_append_one_weight_only(dev):
    a = Append(7, 21, 4, 2, 128, 16, BF16)
    a.qw = None
    a.check(dev)
    a = Append(8, 21, 4, 2, 128, 16, BF16)
    a.kw = None
    a.check(dev)


@pytest.mark.parametrize("x_scale", [1e-4, 300.0])
def test_append_sizes_of_values(dev, x_scale):
    # norms of small rows (eps counts) and large ones; without them numbers that saturate
    Append(9, 40, 4, 2, 128, 16, F16, x_scale=x_scale, eps=1e-6).check(dev)
    Append(9, 40, 4, 2, 128, 16, BF16, x_scale=x_scale, norm=False).check(dev)
    Append(9, 40, 4, 2, 128, 16, BF16, x_scale=x_scale, norm=True, eps=0.0, q8=False).check(dev)


def test_append_infinities_and_nan(dev):
    inf, nan = float("inf"), float("nan")
    k = torch.zeros(1, 1, 64, dtype=BF16, device=dev)
    k[0, 0, :6] = torch.tensor([inf, -inf, nan, 3e38, -3e38, 1e-38], dtype=BF16)
    kc, vc = (torch.zeros(1, 1, 8, 64, dtype=BYTE, device=dev).view(E4M3) for _ in range(2))
    s = torch.tensor([0.013], device=dev)
    pa.reshape_and_cache_q8(k, k, kc, vc, s, s, torch.tensor([2], dtype=torch.int32, device=dev))
    assert pa.device_errors() == 0
    for cache in (kc, vc):
        row = cache.cpu()[0, 0, 2].float()
        assert row[:6].nan_to_num(7.0).tolist() == [448.0, -448.0, 7.0, 448.0, -448.0, 0.0]
        assert row[2].isnan() and (row[6:] == 0).all()


def test_every_16bit_number_gets_its_code(dev):
    """All finite fp16 and bf16 numbers, over scales of many sizes: the code is that
    of value / scale in fp32."""
    for dtype in (F16, BF16):
        x = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(dtype)
        x = x[x.isfinite()]
        x = x[: x.numel() // 512 * 512].view(-1, 8, 64).contiguous()
        T = x.shape[0]
        for exp in (-20, -9, -6, 0, 7):
            s = (2.0 ** exp) * (1.0 + torch.arange(8).float() / 9.1)
            kc, vc = (torch.zeros(-(-T // 16), 8, 16, 64, dtype=BYTE, device=dev).view(E4M3) for _ in range(2))
            sd = s.to(dev)
            pa.reshape_and_cache_q8(x.to(dev), x.to(dev), kc, vc, sd, sd, torch.arange(T, dtype=torch.int32, device=dev))
            want = (x.float() / s[:, None]).clamp(-448, 448).to(E4M3).view(BYTE)
            for cache in (kc, vc):
                got = cache.view(BYTE).permute(0, 2, 1, 3).reshape(-1, 8, 64)[:T].cpu()
                assert torch.equal(got, want), f"{dtype} 2^{exp}"


def test_append_without_norms_is_rope_and_cache(dev):
    a = Append(10, 50, 8, 2, 128, 16, BF16, norm=False, q8=False)
    out, kc, vc = a.run(dev)
    qkv = a.qkv.to(dev)
    o2 = torch.zeros(50, 8, 128, dtype=BF16, device=dev)
    k2, v2 = (torch.full((a.N, 2, 16, 128), -55.0, dtype=BF16, device=dev) for _ in range(2))
    pa.rope_and_cache(o2, qkv[:, :8], qkv[:, 8:10], qkv[:, 10:], k2, v2, a.positions.to(dev), a.table.to(dev),
                      a.slots.to(dev))
    assert torch.equal(out, o2.cpu()) and torch.equal(kc, k2.cpu()) and torch.equal(vc, v2.cpu())


def test_append_without_q_or_rotation(dev):
    a = Append(11, 20, 3, 2, 64, 16, F16, rotary=0, norm=False)
    k, v = a.qkv[:, 3:5].to(dev), a.qkv[:, 5:].to(dev)      # slices: rows apart
    kc, vc = (torch.zeros(a.N, 2, 16, 64, dtype=BYTE, device=dev).view(E4M3) for _ in range(2))
    pos = a.positions.clone()
    pos[4] = -1
    assert pa.norm_rope_and_cache(None, None, k, v, kc, vc, pos.to(dev), None, a.slots.to(dev), k_scales=a.ks.to(dev),
                                  v_scales=a.vs.to(dev)) is None
    assert pa.device_errors() == 0
    at = a.slots.long()
    for cache, x, s in ((kc, k, a.ks), (vc, v, a.vs)):
        want = (x.cpu().float() / s[:, None]).clamp(-448, 448).to(E4M3).view(BYTE)
        want[4] = 0
        assert torch.equal(cache.cpu().view(BYTE)[at // 16, :, at % 16], want)


def test_append_refuses(dev):
    a = Append(12, 4, 4, 2, 128, 16, BF16)
    t = lambda x: x.to(dev)
    q, k, v = (x.contiguous() for x in (t(a.qkv)[:, :4], t(a.qkv)[:, 4:6], t(a.qkv)[:, 6:]))
    c8 = torch.zeros(4, 2, 16, 128, dtype=BYTE, device=dev).view(E4M3)
    c16 = torch.zeros(4, 2, 16, 128, dtype=BF16, device=dev)
    base = dict(q_out=torch.empty_like(q), q=q, k=k, v=v, k_cache=c8, v_cache=c8.clone(), positions=t(a.positions),
                cos_sin=t(a.table), slot_mapping=t(a.slots), k_scales=t(a.ks), v_scales=t(a.vs))

    def refused(kind, **kw):
        with pytest.raises(kind):
            pa.norm_rope_and_cache(**{**base, **kw})

    refused(TypeError, k_cache=c16)
    refused(TypeError, k_scales=None)
    refused(TypeError, v_scales=None)
    refused(TypeError, k_scales=None, v_scales=None)              # e4m3 caches need scales
    refused(ValueError, k_scales=t(a.ks)[:1])
    refused(TypeError, v_scales=t(a.vs).double())
    refused(ValueError, k_scales=a.ks)                            # on the CPU
    refused(TypeError, q_weight=t(a.qw).to(BF16))
    refused(ValueError, k_weight=t(a.kw)[:64])
    refused(ValueError, q_out=k.expand(4, 2, 128))
    refused(ValueError, q_out=None)
    refused(ValueError, q=None)
    refused(ValueError, positions=None)
    refused(ValueError, slot_mapping=t(a.slots)[:3])
    refused(TypeError, q=q.half())
    refused(pa.PaError, eps=-1.0)
    refused(pa.PaError, eps=float("nan"))
    refused(pa.PaError, cos_sin=pa.rope_table(300, 8, device=dev))
    big = torch.zeros(4, 8, 128, dtype=BF16, device=dev)
    refused(ValueError, q_out=big[:, 1:5], q=big[:, 0:4])         # overlapping rows
    refused(ValueError, q_out=big[:, 1:5], q=q, k=big[:, 4:6])
    assert pa.norm_rope_and_cache(**{**base, "q_weight": t(a.qw)}) is base["q_out"]
    assert pa.device_errors() == 0


def test_append_nothing(dev):
    e = torch.zeros(0, 4, 128, dtype=BF16, device=dev)
    c8 = torch.zeros(4, 2, 16, 128, dtype=BYTE, device=dev).view(E4M3)
    s, i = torch.ones(2, device=dev), torch.zeros(0, dtype=torch.int32, device=dev)
    pa.norm_rope_and_cache(e, e, e[:, :2], e[:, :2], c8, c8.clone(), i, pa.rope_table(9, 64, device=dev), i, k_scales=s,
                           v_scales=s)
    assert pa.device_errors() == 0


# ------------------------------------------------------------------ gather

@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("H,D,B", [(1, 64, 8), (3, 64, 32), (8, 128, 16), (5, 256, 8), (2, 256, 32)])
@pytest.mark.parametrize("T", [1, 7, 300])
def test_gather(dev, dtype, H, D, B, T):
    g = torch.Generator().manual_seed(T + D)
    N = 11
    kc, vc = (torch.randint(0, 256, (N, H, B, D), generator=g).to(BYTE).view(E4M3) for _ in range(2))
    ks, vs = scales_for(1, H), scales_for(2, H)
    slots = torch.randint(-2, N * B, (T,), generator=g).to(torch.int32)   # some twice, some skipped
    ko, vo = (torch.full((T, H, D), -3.5, dtype=dtype, device=dev) for _ in range(2))
    got = pa.gather_cache_q8(ko, vo, kc.to(dev), vc.to(dev), ks.to(dev), vs.to(dev), slots.to(dev))
    assert got[0] is ko and got[1] is vo and pa.device_errors() == 0
    keep = slots >= 0
    at = slots[keep].long()
    for o, c, s in ((ko.cpu(), kc, ks), (vo.cpu(), vc, vs)):
        want = (c.view(BYTE)[at // B, :, at % B].view(E4M3).float() * s[:, None]).to(dtype)
        assert torch.equal(o[keep].isnan(), want.isnan())
        assert torch.equal(o[keep].nan_to_num(0.0), want.nan_to_num(0.0))
        assert (o[~keep] == -3.5).all()


def test_gather_flags_and_refuses(dev):
    c = torch.zeros(2, 1, 16, 64, dtype=BYTE, device=dev).view(E4M3)
    s = torch.ones(1, device=dev)
    o, o2 = (torch.full((3, 1, 64), 9.0, dtype=F16, device=dev) for _ in range(2))
    slots = torch.tensor([32, 31, 2 ** 31 - 1], dtype=torch.int32, device=dev)
    pa.gather_cache_q8(o, o2, c, c, s, s, slots)
    assert pa.device_errors() == pa.DEVERR_SLOT
    assert (o[[0, 2]] == 9).all() and (o[1] == 0).all() and (o2[[0, 2]] == 9).all()
    for kind, args in ((ValueError, (o, o, c, c, s, s, slots)), (ValueError, (o, o2[:2], c, c, s, s, slots)),
                       (TypeError, (o, o2.to(BF16), c, c, s, s, slots)), (TypeError, (o, o2, o[None], c, s, s, slots)),
                       (TypeError, (o.float(), o2, c, c, s, s, slots)), (ValueError, (o, o2, c, c, s[:0], s, slots)),
                       (TypeError, (o, o2, c, c, s, s, slots.long())), (ValueError, (o, o2, c, c[:1], s, s, slots))):
        with pytest.raises(kind):
            pa.gather_cache_q8(*args)
    pa.gather_cache_q8(o[:0], o2[:0], c, c, s, s, slots[:0])
    assert pa.device_errors() == 0


# ------------------------------------------------------------------ blocks

@pytest.mark.parametrize("H,D,B", [(1, 64, 8), (3, 64, 8), (5, 128, 16), (2, 256, 32)])
def test_copy_blocks(dev, H, D, B):
    g = torch.Generator().manual_seed(4)
    kc, vc = (torch.randint(0, 256, (9, H, B, D), generator=g).to(BYTE) for _ in range(2))
    a, b = kc.to(dev).view(E4M3), vc.to(dev).view(E4M3)
    pairs = torch.tensor([[0, 7], [3, 8], [1, 99]], dtype=torch.int32, device=dev)
    pa.copy_blocks(a, b, a, b, pairs)
    assert pa.device_errors() == pa.DEVERR_TABLE
    host = torch.empty(4, H, B, D, dtype=BYTE).pin_memory().view(E4M3)
    assert host.is_pinned()
    pa.copy_blocks(a, b, host, host, torch.tensor([[7, 1]], dtype=torch.int32, device=dev)[:0])
    host_k, host_v = (torch.zeros(4, H, B, D, dtype=BYTE).pin_memory().view(E4M3) for _ in range(2))
    pa.copy_blocks(a, b, host_k, host_v, torch.tensor([[7, 1], [8, 3]], dtype=torch.int32, device=dev))
    assert pa.device_errors() == 0
    for cache, was, out in ((a, kc, host_k), (b, vc, host_v)):
        want = was.clone()
        want[7], want[8] = was[0], was[3]
        assert torch.equal(cache.view(BYTE).cpu(), want)
        assert torch.equal(out.view(BYTE)[1], was[0]) and torch.equal(out.view(BYTE)[3], was[3])
        assert (out.view(BYTE)[[0, 2]] == 0).all()


# ------------------------------------------------------------------ attention

def to_dev(c, dev):
    d = {n: getattr(c, n).to(dev) for n in ("q", "k8", "v8", "ks", "vs", "tables", "lens", "starts")}
    d["slopes"] = None if c.slopes is None else c.slopes.to(dev)
    d["prefix"] = None if c.prefix is None else c.prefix.to(dev)
    return d


def run_decode(c, d, out=None, **kw):
    out = torch.full_like(d["q"], float("nan")) if out is None else out
    pa.decode_grouped_q8(out, d["q"], d["k8"], d["v8"], d["ks"], d["vs"], d["tables"], d["lens"], c.scale,
                         softcap=c.cap, alibi_slopes=d["slopes"], window=c.window, prefix_lens=d["prefix"], **kw)
    return out


def run_prefill(c, d, out=None, **kw):
    out = torch.full_like(d["q"], float("nan")) if out is None else out
    kw.setdefault("max_query_len", max(c.new))
    pa.prefill_grouped_q8(out, d["q"], d["k8"], d["v8"], d["ks"], d["vs"], d["tables"], d["lens"], d["starts"], c.scale,
                          softcap=c.cap, alibi_slopes=d["slopes"], window=c.window, prefix_lens=d["prefix"], **kw)
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


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("B", [8, 16, 32])
def test_decode_shapes(dev, dtype, D, B):
    ctx = [1, 2, 7, 15, 16, 17, 31, 33, 64, 65, 100, 257]
    decode(make_q8_case(21, ctx, [1] * len(ctx), 8, 2, D, B, dtype), dev)


@pytest.mark.parametrize("group", [1, 2, 3, 4, 5, 8, 9, 16, 17, 40])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_decode_groups(dev, group, D):
    decode(make_q8_case(22, [40, 1, 300, 0], [1] * 4, 3 * group, 3, D, 16, BF16), dev)
    decode(make_q8_case(23, [77, 200], [1] * 2, 2 * group, 2, D, 8, F16), dev)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("window,prefix", [(0, None), (1, None), (64, None), (100, [4] * 6),
                                           (17, [0, 1, 16, 33, 200, 999]), (1, [1, -5, 0, 40, 63, 64])])
@pytest.mark.parametrize("cap,alibi", [(0.0, False), (20.0, False), (0.0, True), (5.0, True)])
def test_decode_options(dev, dtype, window, prefix, cap, alibi):
    ctx = [1, 16, 63, 128, 500, 1023]
    decode(make_q8_case(24, ctx, [1] * 6, 12, 4, 128, 16, dtype, window=window, prefix=prefix, cap=cap, alibi=alibi,
                        q_scale=2.0), dev)


@pytest.mark.parametrize("D,B", [(64, 8), (64, 32), (256, 16), (256, 8), (256, 32), (128, 32)])
def test_decode_options_other_shapes(dev, D, B):
    ctx = [9, 130, 1, 700, 65]
    decode(make_q8_case(25, ctx, [1] * 5, 14, 2, D, B, BF16, window=70, prefix=[3, 40, 0, 9, 64], cap=15.0, alibi=True),
           dev)


def test_decode_long_and_many(dev):
    decode(make_q8_case(26, [9000, 3, 20011], [1] * 3, 8, 1, 64, 16, F16), dev)
    decode(make_q8_case(27, [12345], [1], 6, 2, 128, 32, BF16, alibi=True), dev)
    decode(make_q8_case(28, [5000, 7001], [1, 1], 20, 2, 256, 16, BF16), dev)
    g = torch.Generator().manual_seed(5)
    ctx = torch.randint(0, 40, (3000,), generator=g).tolist()
    decode(make_q8_case(29, ctx, [1] * 3000, 2, 1, 64, 16, F16), dev)


@pytest.mark.parametrize("S,heads,lo,hi,D", [(50, (16, 8), 60, 100, 128), (150, (8, 4), 90, 100, 128),
                                             (500, (9, 3), 50, 64, 64), (512, (10, 1), 1, 33, 128),
                                             (31, (6, 2), 1, 320, 256), (90, (40, 8), 120, 130, 64)])
def test_decode_short_contexts(dev, S, heads, lo, hi, D):
    """Whole contexts to a CTA, one or several, some empty; and one that is too long for it."""
    g = torch.Generator().manual_seed(S)
    ctx = torch.randint(lo, hi + 1, (S,), generator=g).tolist()
    decode(make_q8_case(33, ctx, [1] * S, *heads, D, 16, BF16), dev)
    ctx[S // 2] = ctx[1] = 0
    c = make_q8_case(34, ctx, [1] * S, *heads, D, 16, F16, window=40, prefix=[3] * S, cap=9.0)
    decode(c, dev)
    ctx[S - 1] = 1500
    decode(make_q8_case(35, ctx, [1] * S, *heads, D, 16, F16, alibi=True), dev)
    d = to_dev(c, dev)
    d["lens"][:] = 0
    out = run_decode(c, d)
    assert pa.device_errors() == 0 and (out == 0).all()


@pytest.mark.parametrize("q_scale", [1e-30, 1e-3, 1e4, 1e30])
def test_decode_sizes_of_queries(dev, q_scale):
    """bf16 queries of any size go through fp16 products: a scale that undoes theirs
    gives the same scores."""
    c = make_q8_case(30, [50, 300], [1, 1], 8, 2, 128, 16, BF16, q_scale=q_scale, scale=128 ** -0.5 / q_scale)
    decode(c, dev)
    c = make_q8_case(30, [50, 300], [1, 1], 8, 2, 128, 16, BF16)
    c.q[0, 3] = 0.0                                   # a row of zeros
    c.q[1, 2, 5] = 3e4                                # one element far above the others
    c.scale = 1e-4
    decode(c, dev)


def test_decode_score_profiles(dev):
    for kind in range(4):
        c = make_q8_case(31, [600, 33], [1, 1], 8, 2, 128, 16, F16)
        j = torch.arange(600).float()
        prof = [j / 20, 30 - j / 20, torch.where(j == 577, 30.0, 0.0), (j % 64) / 2][kind]
        c.ks[:] = 0.1
        c.k8 = codes(c.k_cache * 1.0, c.ks)
        for i in range(600):
            blk = int(c.tables[0, i // 16])
            c.k8[blk, :, i % 16, 0] = to_e4m3(prof[i].double() / 0.1).float().to(E4M3)
        refresh(c)
        c.q[0, :, 0] = 11.0
        decode(c, dev, f"profile {kind}")


def test_decode_errors_and_bad_entries(dev):
    c = make_q8_case(32, [40, 100, 64], [1] * 3, 8, 2, 128, 16, BF16)
    good = run_decode(c, to_dev(c, dev)).cpu()
    pa.device_errors()
    d = to_dev(c, dev)
    d["lens"][1] = 9999
    got = run_decode(c, d).cpu()
    assert pa.device_errors() == pa.DEVERR_CONTEXT
    assert torch.equal(got[[0, 2]], good[[0, 2]]) and (got[1] == 0).all()
    pa.reset_workspaces()
    d = to_dev(c, dev)
    d["tables"][2, 1] = 2 ** 30
    got = run_decode(c, d).cpu()
    assert pa.device_errors() == pa.DEVERR_TABLE
    pa.reset_workspaces()
    assert torch.equal(got[:2], good[:2]) and torch.isfinite(got).all()


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B", [8, 16, 32])
def test_prefill_shapes(dev, dtype, D, B):
    ctx = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 200]
    prefill(make_q8_case(41, ctx, ctx, 4, 2, D, B, dtype), dev)
    prefill(make_q8_case(42, [130, 300, 77], [1, 130, 3], 8, 2, D, B, dtype), dev)


@pytest.mark.parametrize("group", [1, 2, 3, 5, 8, 16, 40, 128])
@pytest.mark.parametrize("D", [64, 128])
def test_prefill_groups(dev, group, D):
    prefill(make_q8_case(43, [70, 1, 150], [70, 1, 33], 2 * group, 2, D, 16, BF16), dev)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("window,prefix", [(0, None), (1, None), (64, None), (100, [4] * 4), (17, [0, 33, 200, 999]),
                                           (0, [300, 3, 70, 0])])
@pytest.mark.parametrize("cap,alibi", [(0.0, False), (20.0, False), (0.0, True), (5.0, True)])
def test_prefill_options(dev, dtype, window, prefix, cap, alibi):
    ctx, new = [300, 16, 129, 500], [300, 16, 40, 7]
    prefill(make_q8_case(44, ctx, new, 12, 4, 128, 16, dtype, window=window, prefix=prefix, cap=cap, alibi=alibi,
                         q_scale=2.0), dev)


@pytest.mark.parametrize("D,B", [(64, 8), (64, 32), (128, 32), (128, 8)])
def test_prefill_options_other_shapes(dev, D, B):
    prefill(make_q8_case(45, [260, 90, 700], [260, 9, 130], 6, 2, D, B, F16, window=70, prefix=[3, 40, 0], cap=15.0,
                         alibi=True), dev)


def test_prefill_long(dev):
    prefill(make_q8_case(46, [2100], [2100], 4, 1, 128, 16, BF16), dev)
    prefill(make_q8_case(47, [9000, 33], [5, 33], 8, 1, 128, 16, F16), dev)       # key splits
    prefill(make_q8_case(48, [6000, 5000], [64, 300], 8, 4, 64, 16, BF16, alibi=True), dev)


@pytest.mark.parametrize("heads,B", [((16, 16), 16), ((24, 8), 8)])
def test_prefill_more_items_than_processors(dev, heads, B):
    """Items are then taken by falling numbers of keys, whatever sequence they are of."""
    ctx = [900, 1500, 33, 1500, 0, 1200, 700]
    new = [900, 300, 33, 1500, 0, 257, 1]
    prefill(make_q8_case(51, ctx, new, *heads, 64, B, F16), dev)
    c = make_q8_case(52, ctx, new, *heads, 64, B, BF16, window=300, prefix=[0, 40, 5, 0, 0, 1000, 3])
    d = to_dev(c, dev)
    good = run_prefill(c, d).cpu()
    assert pa.device_errors() == 0
    check(c, good, True)
    d["lens"][3] = 1499                               # shorter than its queries
    out = torch.full_like(d["q"], 5.0)
    run_prefill(c, d, out)
    assert pa.device_errors() == pa.DEVERR_CONTEXT
    r0, r1 = c.starts_list[3], c.starts_list[4]
    out = out.cpu()
    assert (out[r0:r1] == 5).all()
    assert torch.equal(out[:r0], good[:r0]) and torch.equal(out[r1:], good[r1:])
    pa.reset_workspaces()


def test_prefill_many_sequences(dev):
    # past 32 sequences items go by levels of pairs
    g = torch.Generator().manual_seed(9)
    ctx = torch.randint(1, 90, (200,), generator=g).tolist()
    new = [min(c, int(n)) for c, n in zip(ctx, torch.randint(1, 90, (200,), generator=g))]
    prefill(make_q8_case(53, ctx, new, 4, 2, 64, 16, BF16), dev)


@pytest.mark.parametrize("q_scale", [1e-30, 1e-3, 1e4, 1e30])
@pytest.mark.parametrize("cap", [0.0, 12.0])
def test_prefill_sizes_of_queries(dev, q_scale, cap):
    """As for the decode; items follow one another on a processor, so that the rows of
    one are scaled while the item before is finished."""
    ctx = [300, 1100, 77]
    c = make_q8_case(54, ctx, ctx, 32, 16, 128, 16, BF16, q_scale=q_scale, scale=128 ** -0.5 / q_scale, cap=cap)
    if cap and c.scale / cap < 2.0 ** -100:           # the range of scale / softcap
        with pytest.raises(pa.PaError):
            run_prefill(c, to_dev(c, dev))
        return
    prefill(c, dev)
    c.q[7, 3] = 0.0
    c.q[250] = 0.0
    c.q[311, 2, 5] = 3e4 * q_scale
    c.scale = 1e-4 / q_scale
    prefill(c, dev)


def test_attention_of_keys_that_are_not_numbers(dev):
    """A NaN among one sequence's keys or values reaches that sequence's rows alone, and
    nothing at all from where no query sees it."""
    ctx, new = [200, 150, 90], [40, 150, 1]
    for D in (64, 128):
        c = make_q8_case(55, ctx, new, 8, 2, D, 16, F16, window=60)
        d = to_dev(c, dev)
        one = dict(d, q=d["q"][[39, 189, 190]].contiguous())
        good_d, good_p = run_decode(c, one).cpu(), run_prefill(c, d).cpu()
        assert torch.isfinite(good_d).all() and torch.isfinite(good_p).all()
        for name in ("k8", "v8"):
            x = d[name].clone()
            blk = int(c.tables[1, 9])                         # tokens 144 to 149 of sequence 1
            x[blk, 0, 2] = torch.tensor(float("nan"), device=dev).to(E4M3)
            got_d, got_p = run_decode(c, dict(one, **{name: x})).cpu(), run_prefill(c, dict(d, **{name: x})).cpu()
            assert pa.device_errors() == 0
            assert got_d[1, :4].isnan().any() and got_p[189, :4].isnan().any()
            assert torch.equal(got_d[[0, 2]], good_d[[0, 2]]) and torch.equal(got_d[1, 4:], good_d[1, 4:])
            assert torch.equal(got_p[:40], good_p[:40]) and torch.equal(got_p[190:], good_p[190:])
            assert torch.equal(got_p[:, 4:], good_p[:, 4:])
            if name == "k8":
                assert torch.equal(got_p[40:40 + 146], good_p[40:40 + 146])


def test_prefill_rows_left_alone_and_flags(dev):
    c = make_q8_case(49, [100, 50, 70], [20, 50, 1], 4, 2, 128, 16, BF16)
    d = to_dev(c, dev)
    good = run_prefill(c, d).cpu()
    assert pa.device_errors() == 0
    q = torch.cat([d["q"], d["q"][:5]])
    out = torch.full_like(q, 5.0)
    d2 = dict(d, q=q)
    run_prefill(c, d2, out)                           # five rows behind the last sequence
    assert torch.equal(out[:71].cpu(), good) and (out[71:] == 5).all()
    d["lens"][0] = 10                                 # shorter than its queries
    out = torch.full_like(d["q"], 5.0)
    run_prefill(c, d, out)
    assert pa.device_errors() == pa.DEVERR_CONTEXT
    assert (out[:20] == 5).all() and torch.equal(out[20:].cpu(), good[20:])
    pa.reset_workspaces()
    d = to_dev(c, dev)
    d["tables"][1, 1] = -3
    out = run_prefill(c, d)
    assert pa.device_errors() == pa.DEVERR_TABLE
    assert torch.isfinite(out).all() and torch.equal(out[:20].cpu(), good[:20])
    pa.reset_workspaces()


def test_attention_refuses(dev):
    c = make_q8_case(50, [40, 30], [1, 1], 8, 2, 128, 16, BF16)
    d = to_dev(c, dev)
    out = torch.empty_like(d["q"])
    names = ("q", "k8", "v8", "ks", "vs", "tables", "lens")
    half = torch.zeros(d["k8"].shape, dtype=BF16, device=dev)
    bad = [(TypeError, "q", d["q"].float()), (TypeError, "k8", half), (TypeError, "v8", half),
           (ValueError, "v8", d["v8"][1:]), (ValueError, "ks", d["ks"][:1]), (TypeError, "vs", d["vs"].double()),
           (ValueError, "vs", c.vs), (TypeError, "tables", d["tables"].long()), (ValueError, "lens", d["lens"][:1]),
           (ValueError, "q", d["q"][:, :7]), (TypeError, "ks", None)]
    for kind, name, value in bad:
        args = [dict(d, **{name: value})[n] for n in names]
        with pytest.raises(kind):
            pa.decode_grouped_q8(out, *args, c.scale)
        with pytest.raises(kind):
            pa.prefill_grouped_q8(out, *args, d["starts"], c.scale, max_query_len=1)
    with pytest.raises(TypeError):
        pa.decode_grouped_q8(out.half(), *[d[n] for n in names], c.scale)
    with pytest.raises(pa.PaError):
        pa.decode_grouped_q8(out, *[d[n] for n in names], float("nan"))
    with pytest.raises(ValueError):
        pa.prefill_grouped_q8(out, *[d[n] for n in names], d["starts"][:2], c.scale)
    with pytest.raises(TypeError):                    # the 16-bit calls do not take 8-bit caches
        pa.decode_grouped(out, d["q"], d["k8"], d["v8"], d["tables"], d["lens"], c.scale)
    assert pa.device_errors() == 0


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("dtype", [F16, BF16])
def test_a_layer_of_a_server(dev, dtype):
    """Two prompts appended and read in one call, then tokens one by one, against fp64
    on the cache as it was written; and what the cache holds read back."""
    Hq, H, D, B, N = 8, 2, 128, 16, 40
    g = torch.Generator().manual_seed(3)
    ks, vs = (scales_for(i, H).to(dev) for i in (1, 2))
    kc, vc = (torch.zeros(N, H, B, D, dtype=BYTE, device=dev).view(E4M3) for _ in range(2))
    table = pa.rope_table(512, D, device=dev)
    qw, kw = (1 + 0.2 * torch.randn(D, generator=g).to(dev) for _ in range(2))
    m = pa.KVManager(N, B, 20, shuffle_seed=7)
    lens = [100, 37]
    seqs = [m.add_sequence(n) for n in lens]

    def step(new):
        tables, ctx = m.block_tables(seqs, 20)
        T = sum(new)
        qkv = torch.randn(T, Hq + 2 * H, D, generator=g).to(dtype).to(dev)
        pos = torch.cat([torch.arange(n - k, n) for n, k in zip(lens, new)]).to(torch.int32)
        slots = torch.tensor([m.slot(s, int(p)) for s, n, k in zip(seqs, lens, new) for p in range(n - k, n)],
                             dtype=torch.int32)
        q = torch.empty(T, Hq, D, dtype=dtype, device=dev)
        pa.norm_rope_and_cache(q, qkv[:, :Hq], qkv[:, Hq:Hq + H], qkv[:, Hq + H:], kc, vc, pos.to(dev), table,
                               slots.to(dev), qw, kw, k_scales=ks, v_scales=vs)
        t = torch.as_tensor(tables, dtype=torch.int32).to(dev)
        c = torch.as_tensor(ctx, dtype=torch.int32).to(dev)
        out = torch.empty_like(q)
        starts = [0]
        for k in new:
            starts.append(starts[-1] + k)
        if max(new) == 1:
            pa.decode_grouped_q8(out, q, kc, vc, ks, vs, t, c, D ** -0.5)
        else:
            pa.prefill_grouped_q8(out, q, kc, vc, ks, vs, t, c, torch.tensor(starts, dtype=torch.int32, device=dev),
                                  D ** -0.5, max_query_len=max(new))
        assert pa.device_errors() == 0
        case = make_q8_case(1, lens, new, Hq, H, D, B, dtype)
        case.q, case.tables = q.cpu(), t.cpu()
        case.k8, case.v8, case.ks, case.vs = kc.cpu(), vc.cpu(), ks.cpu(), vs.cpu()
        refresh(case)
        check(case, out, max(new) > 1)

    step(list(lens))
    for _ in range(3):
        for i, s in enumerate(seqs):
            m.append(s)
            lens[i] += 1
        step([1, 1])
    slots = torch.tensor([m.slot(seqs[0], i) for i in range(lens[0])], dtype=torch.int32, device=dev)
    ko, vo = (torch.empty(lens[0], H, D, dtype=dtype, device=dev) for _ in range(2))
    pa.gather_cache_q8(ko, vo, kc, vc, ks, vs, slots)
    at = slots.cpu().long()
    for o, cch, s in ((ko, kc, ks), (vo, vc, vs)):
        want = cch.cpu().view(BYTE)[at // B, :, at % B].view(E4M3).float() * s.cpu()[:, None]
        assert ((o.cpu().float() - want).abs() <= U[dtype] * want.abs() + 2.0 ** -25).all()


def test_graph_capture_and_streams(dev):
    """Captured calls take buffers of their own, replay on new contents, and run on
    another stream than the default one."""
    c = make_q8_case(60, [3000, 200, 17], [1, 1, 1], 8, 2, 128, 16, BF16)
    p = make_q8_case(61, [3000, 200, 17], [40, 3, 1], 8, 2, 128, 16, BF16)
    d, e = to_dev(c, dev), to_dev(p, dev)
    want_d, want_p = run_decode(c, d).clone(), run_prefill(p, e).clone()
    out_d, out_p = torch.zeros_like(want_d), torch.zeros_like(want_p)
    s = torch.cuda.Stream(dev)
    s.wait_stream(torch.cuda.current_stream(dev))
    run_decode(c, d, out_d, stream=s)
    run_prefill(p, e, out_p, stream=s)
    s.synchronize()
    assert torch.equal(out_d, want_d) and torch.equal(out_p, want_p)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run_decode(c, d, out_d)
            run_prefill(p, e, out_p)
        graphs.append(g)
    for g in graphs:
        out_d.zero_(), out_p.zero_()
        for _ in range(3):
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out_d, want_d) and torch.equal(out_p, want_p)
    d["ks"] *= 0.5
    want = run_decode(c, dict(d, ks=d["ks"].clone()))
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(out_d, want) and pa.device_errors() == 0


def test_two_streams_at_once(dev):
    """Calls on two streams, each with its stream's buffers, over and over."""
    cases = [make_q8_case(70 + i, [2000, 300, 40, 5], [30, 300, 1, 5], 8, 2, 128, 16, BF16) for i in range(2)]
    ds = [to_dev(c, dev) for c in cases]
    ones = [dict(d, q=d["q"][[29, 329, 330, 335]].contiguous()) for d in ds]
    want = [(run_decode(c, o).clone(), run_prefill(c, d).clone()) for c, d, o in zip(cases, ds, ones)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(dev) for _ in range(2)]
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append((run_decode(cases[i], ones[i]), run_prefill(cases[i], ds[i])))
    torch.cuda.synchronize()
    assert pa.device_errors() == 0
    for g, w in zip(got, want):
        assert all(torch.equal(x, w[0]) and torch.equal(y, w[1]) for x, y in g)


def test_pools_past_2_31_bytes(dev):
    """Blocks at the far end of pools of more than 2^32 bytes."""
    H, D, B, N = 8, 256, 32, 70000
    assert N * H * B * D > 2 ** 32
    kc, vc = (torch.empty(N, H, B, D, dtype=BYTE, device=dev).view(E4M3) for _ in range(2))
    g = torch.Generator().manual_seed(1)
    T = 150
    far = torch.tensor([N - 1, N - 3, N // 2 + 7, N - 2, 1], dtype=torch.int32)
    x = torch.randn(T, 2 * H + 16, D, generator=g).to(BF16).to(dev)
    ks, vs = scales_for(1, H).to(dev), scales_for(2, H).to(dev)
    t = torch.arange(T)
    slots = (far[t // B].long() * B + t % B).to(torch.int32).to(dev)
    pa.reshape_and_cache_q8(x[:, :H], x[:, H:2 * H], kc, vc, ks, vs, slots)
    ko, vo = (torch.empty(T, H, D, dtype=BF16, device=dev) for _ in range(2))
    pa.gather_cache_q8(ko, vo, kc, vc, ks, vs, slots)
    tables, lens = far[None].to(dev), torch.tensor([T], dtype=torch.int32, device=dev)
    q = x[:1, 2 * H:].contiguous()
    out = torch.empty_like(q)
    pa.decode_grouped_q8(out, q, kc, vc, ks, vs, tables, lens, D ** -0.5)
    assert pa.device_errors() == 0
    # the same in a pool of five blocks
    k5, v5 = (torch.empty(5, H, B, D, dtype=BYTE, device=dev).view(E4M3) for _ in range(2))
    near = torch.arange(5, dtype=torch.int32)
    pa.reshape_and_cache_q8(x[:, :H], x[:, H:2 * H], k5, v5, ks, vs, torch.arange(T, dtype=torch.int32, device=dev))
    want = torch.empty_like(q)
    pa.decode_grouped_q8(want, q, k5, v5, ks, vs, near[None].to(dev), lens, D ** -0.5)
    assert torch.equal(out, want)
    for o, c, s in ((ko, k5, ks), (vo, v5, vs)):
        rows = c.view(BYTE).permute(0, 2, 1, 3).reshape(5 * B, H, D)[:T].view(E4M3).float() * s[:, None]
        assert torch.equal(o, rows.to(BF16))
    # and the prefill, at head_dim 128 (the same bytes as twice the heads)
    k2, v2 = kc.view(BYTE).view(N, 2 * H, B, 128).view(E4M3), vc.view(BYTE).view(N, 2 * H, B, 128).view(E4M3)
    assert k2.numel() > 2 ** 32
    s2 = torch.full((2 * H,), 0.01, device=dev)
    q2 = torch.randn(T, 2 * H, 128, generator=g).to(BF16).to(dev)
    xs = torch.randn(T, 2 * H, 128, generator=g).to(BF16).to(dev)
    pa.reshape_and_cache_q8(xs, xs, k2, v2, s2, s2, slots)
    k5, v5 = k5.view(BYTE).view(5, 2 * H, B, 128).view(E4M3), v5.view(BYTE).view(5, 2 * H, B, 128).view(E4M3)
    pa.reshape_and_cache_q8(xs, xs, k5, v5, s2, s2, torch.arange(T, dtype=torch.int32, device=dev))
    starts = torch.tensor([0, T], dtype=torch.int32, device=dev)
    a, b = torch.empty_like(q2), torch.empty_like(q2)
    pa.prefill_grouped_q8(a, q2, k2, v2, s2, s2, tables, lens, starts, 128 ** -0.5, max_query_len=T)
    pa.prefill_grouped_q8(b, q2, k5, v5, s2, s2, near[None].to(dev), lens, starts, 128 ** -0.5, max_query_len=T)
    assert pa.device_errors() == 0 and torch.equal(a, b)


def test_appended_then_read_in_one_stream(dev):
    """Each call reads what the one before wrote, without a wait in between."""
    H, D, B, N = 4, 128, 16, 64
    g = torch.Generator(device=dev).manual_seed(8)
    kc, vc = (torch.zeros(N, H, B, D, dtype=BYTE, device=dev).view(E4M3) for _ in range(2))
    s = torch.full((H,), 2.0 ** -5, device=dev)
    slots = torch.randperm(N * B, generator=g, device=dev).to(torch.int32)
    x = [torch.randn(N * B, 2 * H, D, generator=g, device=dev).to(BF16) for _ in range(40)]
    got = []
    for y in x:
        pa.reshape_and_cache_q8(y[:, :H], y[:, H:], kc, vc, s, s, slots)
        ko, vo = (torch.empty(N * B, H, D, dtype=BF16, device=dev) for _ in range(2))
        pa.gather_cache_q8(ko, vo, kc, vc, s, s, slots)
        got.append((ko, vo))
    assert pa.device_errors() == 0
    for y, (ko, vo) in zip(x, got):
        for o, r in ((ko, y[:, :H]), (vo, y[:, H:])):
            assert torch.equal(o, ((r.float() * 32).clamp(-448, 448).to(E4M3).float() / 32).to(BF16))
