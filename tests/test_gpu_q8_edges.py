"""GPU tests of the 8-bit cache's calls at the ends of their ranges and where their
kernels change form.  References and bounds as in q8_ref and grouped_ref."""
import pytest
import torch

import paged_kv_cache_269_gb300 as pa
from q8_ref import E4M3, make_q8_case, refresh, scales_for
from test_gpu_q8 import decode, prefill

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
