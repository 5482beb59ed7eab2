"""Edges of the rotary and grouped-query calls that need no GPU: sizes,
refusals, and the state of the binding."""
import pytest

import paged_kv_cache_269_gb300 as pa


@pytest.mark.parametrize("D", [64, 128, 256])
def test_decode_counters_hold_a_word_for_every_unit(D):
    """Each (sequence, K/V head, chunk of query heads) has a ticket of its own."""
    for S in list(range(0, 301)) + [4095, 4096]:
        for H, group in ((1, 1), (1, 9), (3, 8), (7, 4), (8, 17), (1, 71)):
            per = 16 if group > 8 and D != 256 else 8
            units = S * H * -(-group // per)
            n = pa.decode_grouped_counters_bytes(S, H * group, H, D, 16)
            assert n % 256 == 0 and n >= max(4 * units, 256)
            assert n < 4 * units + 512
