"""The paged cache on the GPU where calls are unusual: malformed trees, slots that
are not there, hidden rows of any size, batches of unequal requests."""
import math

import pytest
import torch

from cache_reference import Step, ancestors, attend_tolerance

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


# ---- commits over slots that are not there -------------------------------------------

@pytest.mark.parametrize("path", [False, True])
@pytest.mark.parametrize("what", ["table", "page", "last page", "root page", "length"])
def test_commit_keeps_the_length_where_slots_are_missing(V, path, what):
    # request 1's accepted rows stood (partly) in slots that no page holds: append
    # left them out, and the length must not take them in
    s = Step(ctx=[5, 14, 3], nodes=[4, 6, 5], cache=E4, page=4, seed=8, poison=False)
    table, lengths = s.table.clone(), s.lengths.clone()
    if what == "table":
        lengths[1] = table.shape[1] * 4 - 4                 # slots 16 .. 19 of the table's 20, of 5 to take in
    elif what == "length":
        lengths[1] = 2 ** 31 - 3
    else:
        table[1, {"page": 4, "last page": 4, "root page": 3}[what]] = {"page": s.num_pages, "last page": -1, "root page": 1 << 30}[what]
    c = s.cache(V)
    c.append(s.new_k, s.new_v, table, lengths, s.cu)
    assert V.get_error() == BAD_CACHE
    before = [t.clone() for t in (s.k.view(torch.uint8), s.v.view(torch.uint8), s.ks, s.vs)]
    got = c.commit(table, lengths, s.cu, i32([2, 4, 0]), i32([1, 2, -1, -1] + [1, 2, 3, 4, -1, -1] + [-1] * 5) if path else None)
    assert V.get_error() == BAD_CACHE and V.get_error() == 0
    assert got.tolist() == [8, int(lengths[1]), 4]
    for now, was in zip((s.k.view(torch.uint8), s.v.view(torch.uint8), s.ks, s.vs), before):
        assert torch.equal(now, was)                         # rows 1, 2, ... stand where they belong
    # the last slot of the last page is a slot like any other
    lengths[1] = s.table.shape[1] * 4 - 5
    assert c.commit(s.table, lengths, s.cu, i32([2, 4, 0])).tolist() == [8, s.table.shape[1] * 4, 4]
    assert V.get_error() == 0


# ---- hidden rows of any size -----------------------------------------------------------

@pytest.mark.parametrize("dtype,head_dim", [(BF, 128), (HF, 128), (BF, 64), (HF, 64)])
@pytest.mark.parametrize("nodes,ctx", [(4, 50), (40, 50), (40, 900), (200, 0)])
@pytest.mark.parametrize("scale", [1e30, 1e4, 1e-30, math.inf, math.nan])
def test_scales_of_hidden_nodes_reach_no_row(V, dtype, head_dim, nodes, ctx, scale):
    # one node's values are larger (or smaller) than all others' by far: its siblings
    # do not see it, and keep every bit of theirs
    s = Step(ctx=[ctx, 11], nodes=[nodes, 40], tree="star", dtype=dtype, cache=E4, head_dim=head_dim, seed=9)
    page, off = s.row(0, ctx + 2)
    s.vs[page, :, off] = scale
    page, off = s.row(0, ctx + 1)
    s.vs[page, 0, off] = 0.0                                # a row of zeros among them
    out = s.cache(V).attend(s.q, *args(s))
    want, big = s.attend()
    assert V.get_error() == 0
    if not math.isfinite(scale):                            # (0 x inf is NaN: no value of that row is finite)
        assert not out[2].isfinite().any()
        out[2], want[2], big[2] = 0, 0, 0
    ok = (out.double() - want).abs() <= attend_tolerance(s, want, big)
    # its own row may lie beyond f16, whose values from 65520 on round to infinity
    ok |= out.isinf() & (want.abs() >= 65504) if dtype == HF else False
    assert ok.all(), [r for r in range(s.N) if not ok[r].all()]


# ---- outputs over inputs, at the C entries ---------------------------------------------------

def test_outputs_over_inputs_are_refused_by_the_library(V):
    import ctypes
    from speculative_decoding_rejection_decode_gb300 import _lib
    s = Step(ctx=[9, 2], nodes=[3, 4], kv_heads=2, group=2, seed=8, poison=False)
    c, N, D = s.cache(V), s.N, 128
    before = s.k.clone()
    buf = torch.zeros(4, N * 8 * D, dtype=BF, device="cuda")
    at, st = buf.data_ptr(), torch.cuda.current_stream().cuda_stream
    i = torch.zeros(64, dtype=torch.int32, device="cuda")
    i[32:34] = s.lengths
    nodes = lambda **kw: ctypes.byref(_lib.specdec_nodes_t(**{**dict(
        page_table=s.table.data_ptr(), table_stride=s.table.shape[1], max_pages=s.table.shape[1], lengths=s.lengths.data_ptr(),
        cu=s.cu.data_ptr(), parent=None, B=2, N=N), **kw}))
    wide = 8 * D     # rows of q, k and v side by side

    def append(q=at, q_row=wide, out=at + 2 * N * wide, heads=4):
        return _lib.specdec_cache_append(V.handle, c._ref, nodes(), _lib.SPECDEC_BF16, at + 8 * D, wide, D, at + 12 * D, wide, D,
                                         q, q_row, D, heads, out, None, 0, 0, 0, st)

    def attend(q, out, q_row=4 * D):
        return _lib.specdec_tree_attention(V.handle, c._ref, nodes(), _lib.SPECDEC_BF16, q, q_row, D, 4, 1.0, out, None, 0, st)

    invalid = _lib.SPECDEC_ERR_INVALID_ARG
    for bad in (dict(out=at), dict(out=at + 16), dict(out=at + 2 * N * wide - 16), dict(q=at + 2 * N * wide, q_row=4 * D, out=at + 2 * N * wide + 16),
                dict(q=at + 4 * N * wide, q_row=4 * D, out=at + 8 * D)):
        assert append(**bad) == invalid, bad
    for q, out in ((at, at), (at, at + 2 * (N - 1) * 4 * D), (at + 16, at)):
        assert attend(q, out) == invalid
    for out_k, out_v in ((at, at), (at, at + 2 * N * 2 * D - 16)):
        assert _lib.specdec_cache_read(V.handle, c._ref, nodes(), _lib.SPECDEC_BF16, out_k, out_v, st) == invalid
    p = i.data_ptr()
    for acc, path, out, kw in ((p, None, p, {}), (p, p + 32, p + 32 + 4 * (N - 1), {}), (p, None, p + 132, dict(lengths=p + 128)),
                               (p, None, p + 40, dict(cu=p + 32)), (p, None, s.table.data_ptr() + 4, {})):
        assert _lib.specdec_cache_commit(V.handle, c._ref, nodes(**kw), acc, path, out, st) == invalid
    torch.cuda.synchronize()
    assert torch.equal(s.k, before) and V.get_error() == 0
    # side by side, q itself and lengths themselves are fine
    assert append() == 0 and append(q=at + 2 * N * wide, q_row=4 * D, out=at + 2 * N * wide) == 0
    assert attend(at, at + 2 * N * 4 * D) == 0
    assert _lib.specdec_cache_commit(V.handle, c._ref, nodes(lengths=p + 128), p, None, p + 128, st) == 0
    assert i[32:34].tolist() == [10, 3] and V.get_error() == 0
