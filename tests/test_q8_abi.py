"""Refusals of the 8-bit cache's calls, on the host: no CUDA call is reached, so
this runs without a GPU.  Also the fp64 test reference of the numbers, against
torch's own conversion."""
import ctypes

import pytest
import torch

import paged_kv_cache_269_gb300 as pa
from paged_kv_cache_269_gb300.grouped import AttnOpts
from paged_kv_cache_269_gb300.quantized import AppendOpts
from q8_ref import E4M3, to_e4m3

FAKE = ctypes.c_void_p(0x100000)     # never dereferenced: checks fail first
FAKE_P = 0x100000
ODD = ctypes.c_void_p(0x100008)
BIG = 1 << 30


@pytest.fixture(scope="module")
def lib():
    return pa.lib()


def dims(S=2, H=4, D=128, B=16, N=32, dtype=0):
    return pa.Dims(S, H, D, B, N, dtype)


def test_reference_rounding_is_the_types():
    every = torch.arange(256, dtype=torch.uint8).view(E4M3).float()
    every = every[every.isfinite()].double()
    assert torch.equal(to_e4m3(every), every)
    g = torch.Generator().manual_seed(1)
    x = torch.randn(200000, generator=g) * torch.exp2(torch.randint(-14, 8, (200000,), generator=g).float())
    edges = torch.unique(every)
    x = torch.cat([x, (edges[1:] + edges[:-1]).float() / 2]).clamp(-448, 448)   # ties too
    assert torch.equal(to_e4m3(x.double()), x.to(E4M3).float().double())


def append_opts(qw=None, kw=None, eps=1e-6, ks=FAKE_P, vs=FAKE_P):
    return AppendOpts(qw, kw, eps, ks, vs)


def test_append_rejects(lib):
    def call(d=None, q_out=FAKE, q=FAKE, k=FAKE, v=FAKE, kc=FAKE, pos=FAKE, cs=FAKE, slots=FAKE, T=4, Hq=8, qs=1024,
             ks=512, vs=512, os_=1024, rot=128, maxp=100, no_dims=False, o=None, no_opts=False):
        d = d or dims()
        o = o or append_opts()
        return lib.pa_norm_rope_and_cache(q_out, q, k, v, kc, FAKE, pos, cs, slots, T, Hq, qs, ks, vs, os_, rot, maxp, 0,
                                          None if no_dims else ctypes.byref(d), None if no_opts else ctypes.byref(o),
                                          None)
    assert call(no_dims=True) == -1
    assert call(d=dims(D=96)) == -3
    assert call(d=dims(B=12)) == -3
    assert call(d=dims(dtype=2)) == -3
    assert call(d=dims(H=0)) == -2
    assert call(Hq=-1) == -2
    assert call(T=-1) == -2
    assert call(T=0, k=None) == 0
    assert call(maxp=0) == -2
    assert call(rot=-16) == -2
    assert call(rot=144) == -2
    assert call(rot=24) == -3
    assert call(qs=-8) == -2
    assert call(qs=1025) == -4
    assert call(ks=513) == -4
    assert call(os_=512) == -2            # rows of q_out would overlap
    assert call(q_out=None) == -1
    assert call(q=None) == -1
    assert call(k=None) == -1
    assert call(v=None) == -1
    assert call(kc=None) == -1
    assert call(pos=None) == -1
    assert call(cs=None) == -1
    assert call(slots=None) == -1
    assert call(k=ODD) == -4
    assert call(kc=ODD) == -4
    assert call(cs=ODD) == -4
    assert call(d=dims(N=1 << 28, B=16)) == -2
    assert call(o=append_opts(ks=None)) == -1
    assert call(o=append_opts(vs=None)) == -1
    assert call(o=append_opts(ks=FAKE_P + 2)) == -4
    assert call(o=append_opts(qw=FAKE_P + 4)) == -4
    assert call(o=append_opts(kw=FAKE_P + 8)) == -4
    for eps in (-1e-6, float("inf"), float("nan")):
        assert call(o=append_opts(eps=eps)) == -2
    # nothing to rotate and no q: these are not asked for, the rest is
    assert call(q=None, q_out=None, Hq=0, pos=None, cs=None, rot=0, maxp=0, slots=None) == -1
    assert call(q=None, q_out=None, Hq=0, pos=None, cs=None, rot=0, maxp=0, T=0) == 0


def test_gather_rejects(lib):
    def call(d=None, ko=FAKE, vo=FAKE, kc=FAKE, ks=FAKE, slots=FAKE, T=4, no_dims=False):
        d = d or dims()
        return lib.pa_gather_cache_q8(ko, vo, kc, FAKE, ks, FAKE, slots, T, None if no_dims else ctypes.byref(d), None)
    assert call(no_dims=True) == -1
    assert call(d=dims(D=80)) == -3
    assert call(d=dims(B=4)) == -3
    assert call(d=dims(dtype=2)) == -3
    assert call(d=dims(H=0)) == -2
    assert call(d=dims(N=1 << 28)) == -2
    assert call(T=-1) == -2
    assert call(T=0, ko=None) == 0
    for name in ("ko", "vo", "kc", "ks", "slots"):
        assert call(**{name: None}) == -1
    for name in ("ko", "vo", "kc"):
        assert call(**{name: ODD}) == -4
    assert call(ks=ctypes.c_void_p(0x100002)) == -4


def test_copy_blocks_of_8bit_pools(lib):
    def call(d):
        return lib.pa_copy_blocks(FAKE, FAKE, 32, FAKE, FAKE, 32, FAKE, 0, ctypes.byref(d), None)
    assert call(dims(dtype=2)) == 0
    assert call(dims(dtype=2, D=32)) == -3
    assert call(dims(dtype=3)) == -3
    with pytest.raises(ValueError):
        pa.copy_blocks(*[torch.zeros(2, 1, 8, 64).to(E4M3)] * 4, torch.zeros(1, 2, dtype=torch.int32))


def _opts(cap=0.0, window=0):
    return ctypes.byref(AttnOpts(cap, window, None, None))


def test_decode_rejects(lib):
    def call(d=None, out=FAKE, q=FAKE, ks=FAKE, vs=FAKE, tables=FAKE, scale=0.1, mb=8, Hq=8, opts=None, ws=FAKE,
             ws_n=BIG, ctr=FAKE, ctr_n=BIG, no_dims=False):
        d = d or dims()
        return lib.pa_decode_grouped_q8(out, q, FAKE, FAKE, ks, vs, tables, FAKE, scale, mb,
                                        None if no_dims else ctypes.byref(d), Hq, opts, ws, ws_n, ctr, ctr_n, None)
    assert call(no_dims=True) == -1
    assert call(d=dims(D=80)) == -3
    assert call(d=dims(B=64)) == -3
    assert call(d=dims(dtype=2)) == -3
    assert call(Hq=6) == -2
    assert call(Hq=0) == -2
    assert call(mb=0) == -2
    assert call(scale=float("nan")) == -2
    assert call(opts=_opts(cap=-1.0)) == -2
    assert call(opts=_opts(window=-1)) == -2
    assert call(d=dims(S=-1)) == -2
    assert call(d=dims(S=0), out=None) == 0
    assert call(d=dims(N=1 << 27, H=4, B=32)) == -2
    for name in ("out", "q", "ks", "vs", "tables"):
        assert call(**{name: None}) == -1
    assert call(q=ODD) == -4
    assert call(ks=ctypes.c_void_p(0x100001)) == -4
    assert call(ctr=None) == -5
    assert call(ctr_n=0) == -5
    assert call(ws=None) == -5
    assert call(ws_n=16) == -5


def test_prefill_rejects(lib):
    def call(d=None, out=FAKE, ks=FAKE, vs=FAKE, qs=FAKE, total=40, maxq=20, scale=0.1, mb=8, Hq=8, opts=None, ws=FAKE,
             ws_n=BIG, ctr=FAKE, ctr_n=BIG):
        d = d or dims()
        return lib.pa_prefill_grouped_q8(out, FAKE, FAKE, FAKE, ks, vs, FAKE, FAKE, qs, total, maxq, scale, mb,
                                         ctypes.byref(d), Hq, opts, ws, ws_n, ctr, ctr_n, None)
    assert call(d=dims(D=256)) == -3
    assert call(d=dims(H=1), Hq=129) == -3
    assert call(Hq=6) == -2
    assert call(total=-1) == -2
    assert call(maxq=-1) == -2
    assert call(mb=0) == -2
    assert call(scale=float("inf")) == -2
    assert call(opts=_opts(window=-3)) == -2
    assert call(total=0) == 0
    assert call(maxq=0) == 0
    assert call(d=dims(S=0)) == 0
    for name in ("out", "ks", "vs", "qs"):
        assert call(**{name: None}) == -1
    assert call(out=ODD) == -4
    assert call(vs=ctypes.c_void_p(0x100002)) == -4
    assert call(ctr=None) == -5
    assert call(ctr_n=4) == -5


def test_python_refuses_cpu_tensors():
    half = torch.zeros(4, 8, 64, dtype=torch.float16)
    cache = torch.zeros(6, 8, 16, 64, dtype=torch.float16).to(E4M3)
    s, slots = torch.ones(8), torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        pa.gather_cache_q8(half, half.clone(), cache, cache, s, s, slots)
    with pytest.raises(ValueError):
        pa.reshape_and_cache_q8(half, half, cache, cache, s, s, slots)
    with pytest.raises(TypeError):
        pa.reshape_and_cache_q8(half, half, cache, cache, None, s, slots)
    with pytest.raises(TypeError):
        pa.gather_cache_q8(half.float(), half, cache, cache, s, s, slots)
    with pytest.raises(TypeError):
        pa.gather_cache_q8(half, half, half[None], half[None], s, s, slots)
    with pytest.raises(TypeError):
        pa.decode_grouped_q8(half, half, half[None], half[None], s, s, slots[None], slots, 1.0)
