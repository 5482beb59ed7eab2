"""Refusals of the rotary and grouped-query calls, on the host: no CUDA call is
reached, so this runs without a GPU.  Also the fp64 test reference itself,
against torch's own attention on small inputs."""
import ctypes

import pytest
import torch

import paged_kv_cache_269_gb300 as pa
from grouped_ref import make_case, reference, rotate
from paged_kv_cache_269_gb300.grouped import AttnOpts

FAKE = ctypes.c_void_p(0x100000)     # never dereferenced: checks fail first
ODD = ctypes.c_void_p(0x100008)
BIG = 1 << 30


@pytest.fixture(scope="module")
def lib():
    return pa.lib()


def dims(S=2, H=4, D=128, B=16, N=32, dtype=0):
    return pa.Dims(S, H, D, B, N, dtype)


def test_rope_rejects(lib):
    def call(d=None, q_out=FAKE, q=FAKE, k=FAKE, pos=FAKE, cs=FAKE, slots=FAKE, T=4, Hq=8, qs=1024,
             ks=512, vs=512, os_=1024, rot=128, maxp=100, no_dims=False):
        d = d or dims()
        return lib.pa_rope_and_cache(q_out, q, k, FAKE, FAKE, FAKE, pos, cs, slots, T, Hq, qs, ks,
                                     vs, os_, rot, maxp, 0, None if no_dims else ctypes.byref(d), None)
    assert call(no_dims=True) == -1
    assert call(d=dims(D=96)) == -3
    assert call(d=dims(B=12)) == -3
    assert call(d=dims(dtype=2)) == -3
    assert call(d=dims(H=0)) == -2
    assert call(Hq=0) == -2
    assert call(T=-1) == -2
    assert call(T=0, q=None) == 0
    assert call(maxp=0) == -2
    assert call(rot=0) == -2
    assert call(rot=144) == -2
    assert call(rot=24) == -3
    assert call(qs=-8) == -2
    assert call(qs=1025) == -4
    assert call(ks=513) == -4
    assert call(os_=512) == -2            # rows of q_out would overlap
    assert call(os_=1028) == -4
    assert call(q_out=None) == -1
    assert call(q=None) == -1
    assert call(pos=None) == -1
    assert call(cs=None) == -1
    assert call(slots=None) == -1
    assert call(k=ODD) == -4
    assert call(q_out=ODD) == -4
    assert call(cs=ODD) == -4
    assert call(d=dims(N=1 << 28, B=16)) == -2


def _opts(cap=0.0, window=0):
    return ctypes.byref(AttnOpts(cap, window, None, None))


def test_decode_grouped_rejects(lib):
    def call(d=None, out=FAKE, q=FAKE, tables=FAKE, scale=0.1, mb=8, Hq=8, opts=None, ws=FAKE,
             ws_n=BIG, ctr=FAKE, ctr_n=BIG, no_dims=False):
        d = d or dims()
        return lib.pa_decode_grouped(out, q, FAKE, FAKE, tables, FAKE, scale, mb,
                                     None if no_dims else ctypes.byref(d), Hq, opts, ws, ws_n, ctr,
                                     ctr_n, None)
    assert call(no_dims=True) == -1
    assert call(d=dims(D=80)) == -3
    assert call(d=dims(B=64)) == -3
    assert call(Hq=6) == -2               # not a multiple of the K/V heads
    assert call(Hq=0) == -2
    assert call(Hq=-4) == -2
    assert call(mb=0) == -2
    assert call(scale=float("nan")) == -2
    assert call(opts=_opts(cap=-1.0)) == -2
    assert call(opts=_opts(cap=float("inf"))) == -2
    assert call(opts=_opts(cap=float("nan"))) == -2
    assert call(opts=_opts(window=-1)) == -2
    assert call(d=dims(S=-1)) == -2
    assert call(d=dims(S=0), out=None) == 0
    assert call(d=dims(N=1 << 27, H=4, B=32)) == -2
    assert call(d=dims(S=1 << 30)) == -2
    assert call(out=None) == -1
    assert call(tables=None) == -1
    assert call(q=ODD) == -4
    assert call(ctr=None) == -5
    assert call(ctr_n=0) == -5
    assert call(ws=None) == -5
    assert call(ws_n=16) == -5
    assert call(ws=ODD) == -5


def test_prefill_grouped_rejects(lib):
    def call(d=None, out=FAKE, qs=FAKE, total=40, maxq=20, scale=0.1, mb=8, Hq=8, opts=None, ws=FAKE,
             ws_n=BIG, ctr=FAKE, ctr_n=BIG):
        d = d or dims()
        return lib.pa_prefill_grouped(out, FAKE, FAKE, FAKE, FAKE, FAKE, qs, total, maxq, scale, mb,
                                      ctypes.byref(d), Hq, opts, ws, ws_n, ctr, ctr_n, None)
    assert call(d=dims(D=256)) == -3      # the tensor-core kernel: 64 and 128
    assert call(d=dims(D=80)) == -3
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
    assert call(out=None) == -1
    assert call(qs=None) == -1
    assert call(out=ODD) == -4
    assert call(ctr=None) == -5
    assert call(ctr_n=4) == -5
    assert call(d=dims(S=65535, H=128), Hq=8192, maxq=1 << 20) == -2


def test_sizes(lib):
    for D in (64, 128, 256):
        one = pa.decode_grouped_workspace_bytes(8, 8, D, 16)
        assert one >= 0 and pa.decode_grouped_workspace_bytes(64, 4, D, 16) >= one
    assert pa.decode_grouped_counters_bytes(64, 32, 8, 128, 16) % 4 == 0
    with pytest.raises(pa.PaError):
        pa.decode_grouped_workspace_bytes(7, 2, 128, 16)
    with pytest.raises(pa.PaError):
        pa.decode_grouped_counters_bytes(-1, 8, 2, 128, 16)
    with pytest.raises(pa.PaError):
        pa.prefill_grouped_workspace_bytes(4, 8, 2, 256, 16, 100)
    assert pa.prefill_grouped_workspace_bytes(4, 8, 2, 128, 16, 100) >= 0
    assert pa.prefill_grouped_counters_bytes(8, 2, 128, 16) > 0


def test_binding_refuses_cpu_tensors():
    c = make_case(1, [5], [1], 4, 2, 64, 16, torch.float16)
    out = torch.empty_like(c.q)
    with pytest.raises(ValueError):
        pa.decode_grouped(out, c.q, c.k_cache, c.v_cache, c.tables, c.lens, 0.1)
    with pytest.raises(ValueError):
        pa.prefill_grouped(out, c.q, c.k_cache, c.v_cache, c.tables, c.lens, c.starts, 0.1)
    k = torch.zeros(1, 2, 64, dtype=torch.float16)
    with pytest.raises(ValueError):
        pa.rope_and_cache(out, c.q, k, k, c.k_cache, c.v_cache, c.lens, pa.rope_table(8, 64), c.lens)


def test_rope_table():
    t = pa.rope_table(5000, 32, base=500.0)
    assert t.shape == (5000, 32) and t.dtype == torch.float32
    ang = 4999 * 500.0 ** (-2 * 3 / 32)
    assert abs(t[4999, 3].item() - torch.tensor(ang, dtype=torch.float64).cos().item()) < 1e-7
    assert abs(t[4999, 19].item() - torch.tensor(ang, dtype=torch.float64).sin().item()) < 1e-7
    f = torch.rand(16, dtype=torch.float64)
    assert torch.equal(pa.rope_table(9, 32, inv_freq=f)[1, :16], f.cos().float())
    with pytest.raises(ValueError):
        pa.rope_table(4, 7)
    with pytest.raises(ValueError):
        pa.rope_table(4, 8, inv_freq=f)


def test_reference_agrees_with_torch_attention():
    c = make_case(3, [37, 5], [37, 2], 4, 2, 64, 16, torch.float16)
    out, bound = reference(c, True)
    for s in range(2):
        n, r = c.ctx[s], slice(c.starts_list[s], c.starts_list[s + 1])
        blk, off = c.tables[s, torch.arange(n) // 16].long(), torch.arange(n) % 16
        k = c.k_cache[blk, :, off].double().transpose(0, 1).repeat_interleave(2, 0)
        v = c.v_cache[blk, :, off].double().transpose(0, 1).repeat_interleave(2, 0)
        mask = torch.ones(c.new[s], n, dtype=torch.bool).tril(n - c.new[s])
        want = torch.nn.functional.scaled_dot_product_attention(
            c.q[r].double().transpose(0, 1), k, v, attn_mask=mask)
        assert torch.allclose(out[r].transpose(0, 1), want, atol=1e-12)
    assert (bound > 0).all()
    x = torch.randn(3, 2, 8, dtype=torch.float64)
    ang = torch.rand(3, 2, dtype=torch.float64)
    y, _ = rotate(x, ang.cos(), ang.sin(), True)
    z = torch.view_as_complex(x[..., :4].reshape(3, 2, 2, 2).contiguous()) * torch.polar(torch.ones_like(ang), ang)[:, None]
    assert torch.allclose(torch.view_as_real(z).reshape(3, 2, 4), y[..., :4])
    assert torch.equal(x[..., 4:], y[..., 4:])
