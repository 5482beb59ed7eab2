"""GPU tests of the 8-bit cache's calls at the ends of their ranges.  References and
bounds as in q8_ref and grouped_ref."""
import pytest
import torch

import paged_kv_cache_269_gb300 as pa
from q8_ref import make_q8_case, refresh
from test_gpu_q8 import decode, prefill

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
