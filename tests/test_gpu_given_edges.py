"""Verification from given numbers on the GPU at rows far longer than vocabularies."""
from fractions import Fraction

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def V():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_rejection_decode_gb300 import Verifier
    v = Verifier(0)
    yield v
    v.close()


@pytest.mark.parametrize("n", [1 << 20, (1 << 27) + 3, 1 << 28])
@pytest.mark.parametrize("s", [0.1, 0.4, 0.7, 0.95])
def test_sums_hold_at_any_length(V, n, s):
    # a first half of weights whose sums are exact, a second of 0.1, whose sums round
    # the same way every time: the borders are known as fractions
    h = n // 2
    p = torch.full((1, n), 0.1, device="cuda")
    p[0, :h] = 0.125
    a, b, s = Fraction(1, 8), Fraction(float(np.float32(0.1))), np.float32(s)
    t = Fraction(float(s)) * (h * a + (n - h) * b)
    at = t / a if t < h * a else h + (t - h * a) / b
    want = int(at)
    # sums good to 2^-36 of the total move the crossing by 2^-36 n / 0.8 entries at the most
    off = 2.0 ** -36 * n / 0.8
    assert off < 0.02 and off < float(at - want) < 1 - off
    e = torch.zeros(0, dtype=torch.int32, device="cuda")
    cu = torch.zeros(2, dtype=torch.int32, device="cuda")
    out = V.sample_given(p, p[:0], e, cu, torch.zeros(0, device="cuda"), torch.tensor([s], device="cuda"))
    assert out.tokens.tolist() == [want] and V.get_error() == 0
