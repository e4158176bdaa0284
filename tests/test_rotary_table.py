"""The tables of rotary positions for stretched contexts, pair by pair; no GPU."""
import math

import pytest
import torch


@pytest.mark.parametrize("dim,base,trained", [(64, 10000.0, 1024), (128, 500000.0, 8192), (64, 10000.0, 100), (16, 10.0, 5000), (32, 10000.0, 4)])
def test_by_parts_follows_the_turns_of_each_pair(dim, base, trained):
    from speculative_decoding_rejection_decode_gb300 import rotary_table
    fast, slow, factor, gain = 32.0, 1.0, 4.0, 1 + 0.1 * math.log(4.0)
    t = rotary_table(2, dim, base=base, scaling="by_parts", factor=factor, trained_positions=trained, device="cpu")
    angle = torch.atan2(t[1, 1].double(), t[1, 0].double())     # at position 1: the pair's frequency
    index = lambda turns: dim * math.log(trained / (turns * 2 * math.pi)) / (2 * math.log(base))
    lo, hi = math.floor(index(fast)), math.ceil(index(slow))
    for i in range(dim // 2):
        f = base ** (-2 * i / dim)
        kept = 1.0 - min(max((i - lo) / (hi - lo), 0.0), 1.0)
        want = f * kept + f / factor * (1 - kept)
        assert abs(float(angle[i]) - want) <= 2.0 ** -21 * want + 1e-12
        if trained * f / (2 * math.pi) <= slow:                 # turns too seldom: all of the factor
            assert abs(float(angle[i]) - f / factor) <= 2.0 ** -21 * f
        if math.floor(index(fast)) >= i:                        # turns often: none of it
            assert abs(float(angle[i]) - f) <= 2.0 ** -21 * f
        assert abs(float(t[1, 0, i].double() ** 2 + t[1, 1, i].double() ** 2) - gain ** 2) < 1e-6
