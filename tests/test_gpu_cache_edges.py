"""The paged cache on the GPU where calls are unusual: malformed trees, slots that
are not there, hidden rows of any size, batches of unequal requests."""
import math

import pytest
import torch

from cache_reference import HALF_STEP, Step, ancestors, attend_tolerance

pytestmark = pytest.mark.gpu

BF, HF, E4 = torch.bfloat16, torch.float16, torch.float8_e4m3fn
BAD_CU, BAD_TREE, BAD_CACHE = 2, 16, 32


@pytest.fixture(scope="module")
def V():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_rejection_decode_gb300 import Verifier
    v = Verifier(0)
    yield v
    v.close()


def args(s):
    return s.table, s.lengths, s.cu, s.parent


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ---- malformed trees ---------------------------------------------------------------

@pytest.mark.parametrize("cache", [BF, E4])
@pytest.mark.parametrize("nodes,ctx", [(4, 9), (4, 3000), (40, 9), (40, 3000), (300, 200)])   # both kernels, whole and split
@pytest.mark.parametrize("up", ["self", "later", "far", "minus"])
def test_rows_of_malformed_trees_are_zeros(V, cache, nodes, ctx, up):
    s = Step(ctx=[ctx, 70], nodes=[nodes, nodes], tree="random", cache=cache, seed=nodes)
    x = 1                                                    # the bad node, and one below it
    s.parents[0][x], s.parents[0][x + 1] = 0, x
    s.parent[:nodes] = i32(s.parents[0])
    c = s.cache(V)
    good = c.attend(s.q, *args(s))
    assert V.get_error() == 0 and not (good == 0).all(2).any()
    s.parent[x] = {"self": x, "later": x + 1, "far": 1 << 30, "minus": -7}[up]
    out = c.attend(s.q, *args(s), out=torch.full_like(good, 7.0))
    assert V.get_error() == BAD_TREE and V.get_error() == 0
    for j in range(nodes):
        if x in ancestors(s.parents[0], j):
            assert (out[j] == 0).all(), j
        else:
            assert torch.equal(out[j], good[j]), j
    assert torch.equal(out[nodes:], good[nodes:])
