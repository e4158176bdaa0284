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


# ---- scores of any size ------------------------------------------------------------------

def score_tolerance(s, want, big):
    """attend_tolerance with the scores' errors taken from the scores.  A key's score
    (base e) is off by at most D_s = head_dim 2^-24 scale sum |q k| (a float32 sum of
    products) + 2^-22 |z| (the scale, to base 2, and the last addition, each rounded
    to 32 bits) + 2^-20 (the exponential), and over 8-bit caches 2^-17 max |q|
    scale sum |k| (the tile kernel's queries).  With weights w' ~ w e^d, |d_s| <= D_s,
    the result moves by sum w (e^d - 1)(v - o) / sum w e^d, at most
    sum w (e^D - 1) |v - o| / sum w e^-D."""
    scale = s.head_dim ** -0.5
    K, W = s.values("k"), s.values("v")
    tol = attend_tolerance(s, want, big)
    for b in range(s.B):
        for i in range(s.nodes[b]):
            r = s.firsts[b] + i
            at = list(range(s.ctx[b])) + sorted(s.ctx[b] + j for j in ancestors(s.parents[b], i))
            at = torch.tensor(at, device=K.device)
            pages = torch.tensor(s.pages[b], device=K.device)[at // s.page]
            k, v = K[pages, :, at % s.page], W[pages, :, at % s.page]
            q = s.q[r].double().view(s.kv_heads, s.group, -1)
            z = torch.einsum("hgd,shd->hgs", q, k) * scale
            d = s.head_dim * 2.0 ** -24 * scale * torch.einsum("hgd,shd->hgs", q.abs(), k.abs()) + 2.0 ** -22 * z.abs() + 2.0 ** -20
            if s.ks is not None:
                d = d + 2.0 ** -17 * scale * q.abs().amax(-1, keepdim=True) * k.abs().sum(-1).t()[:, None]
            w = torch.softmax(z, -1)
            o = want[r].view(s.kv_heads, s.group, -1)
            off = (v.transpose(0, 1)[:, None] - o[:, :, None]).abs()
            # (weights of 1e-200 and less stay nothing whatever their error)
            up = torch.where(w > 1e-200, w * torch.expm1(d.clamp(max=300.0)), 0.0)
            moved = torch.einsum("hgs,hgsd->hgd", up, off) / (w * (-d).exp()).sum(-1, keepdim=True)
            tol[r] += moved.reshape(s.heads, -1)
    return tol


@pytest.mark.parametrize("dtype,cache", [(BF, BF), (HF, HF), (BF, E4), (HF, E4)])
@pytest.mark.parametrize("nodes", [3, 40])                       # both kernels
def test_every_row_of_extreme_scores(V, dtype, cache, nodes):
    s = Step(ctx=[700], nodes=[nodes], dtype=dtype, cache=cache, seed=10)
    s.q[0] *= 200.0                                             # one key takes all the weight
    s.q[1] = 0.0                                                # all weights equal
    for slot, by in ((3, 300.0), (300, -100.0), (690, 30.0)):    # far above and below the rest, early and late
        page, off = s.row(0, slot)
        if cache == E4:
            s.ks[page, :, off] *= abs(by)
        else:
            s.k[page, :, off] = (s.k[page, :, off].float() * by).to(cache)
    out = s.cache(V).attend(s.q, *args(s))
    want, big = s.attend()
    tol = score_tolerance(s, want, big)
    assert V.get_error() == 0
    err = (out.double() - want).abs()
    assert (err <= tol).all(), [r for r in range(s.N) if not (err[r] <= tol[r]).all()]
    assert float((tol <= 0.1 * big[..., None]).double().mean()) > 0.9   # the bound says something


# ---- batches of unequal requests, long chains ------------------------------------------------

@pytest.mark.parametrize("cache", [BF, E4])
def test_one_large_request_among_many_small_ones(V, cache):
    # 16 rows for the average request: the large one has 75 row tiles in the kernel
    # for few rows, split over the ranges
    s = Step(ctx=[(37 * i) % 301 for i in range(64)] + [3000] + [(53 * i) % 200 for i in range(64)], nodes=[1] * 64 + [300] + [1] * 64,
             kv_heads=2, group=4, page=64, cache=cache, seed=3)
    out = s.cache(V).attend(s.q, *args(s))
    want, big = s.attend()
    assert V.get_error() == 0
    # float32 sums over up to 2^12 keys instead of the bound's 2^11
    tol = attend_tolerance(s, want, big) + 2.0 ** -13 * big[..., None]
    assert ((out.double() - want).abs() <= tol).all()


@pytest.mark.parametrize("cache", [BF, E4])
@pytest.mark.parametrize("ctx", [0, 77, 261])
def test_long_chains(V, cache, ctx):
    # a prompt: contexts that end inside a tile, chains past the largest tree
    s = Step(ctx=[ctx, 5], nodes=[1100, 2], kv_heads=1, group=2, page=48, cache=cache, seed=4)
    out = s.cache(V).attend(s.q, *args(s))
    want, big = s.attend()
    assert V.get_error() == 0
    assert ((out.double() - want).abs() <= attend_tolerance(s, want, big)).all()


# ---- a range that passes the rows --------------------------------------------------------------

@pytest.mark.parametrize("tree", ["chain", "random"])
def test_append_of_a_range_that_passes_the_rows(V, tree):
    s = Step(ctx=[3, 20, 9], nodes=[4, 4, 4], tree=tree, page=8, seed=3, poison=False)
    k0, v0 = s.k.clone(), s.v.clone()
    s.cu[2] = 100                                               # of request 1, and request 2 starts there
    s.cache(V).append(s.new_k, s.new_v, *args(s))
    assert V.get_error() == BAD_CU and V.get_error() == 0
    for now, was, new in ((s.k, k0, s.new_k), (s.v, v0, s.new_v)):
        for j in range(4):
            page, off = s.row(0, 3 + j)
            assert torch.equal(now[page, :, off], new[j])
        assert torch.equal(now[s.pages[1] + s.pages[2]], was[s.pages[1] + s.pages[2]])


@pytest.mark.parametrize("scale,other", [(1e30, 0.01), (1e30, 0.0), (1e18, 2.0 ** -49)])
@pytest.mark.parametrize("ctx", [0, 40])
def test_rows_that_see_a_large_scale_keep_the_others_weights(V, scale, other, ctx):
    # the values of the small ones are nothing beside the large one, their softmax
    # weights are not (a chain: nodes from 2 on see both)
    s = Step(ctx=[ctx], nodes=[30], cache=E4, seed=5)
    s.vs[...] = 0.01
    for slot, by in ((ctx + 1, scale), (ctx, other)):
        page, off = s.row(0, slot)
        s.vs[page, :, off] = by
    out = s.cache(V).attend(s.q, *args(s))
    want, big = s.attend()
    # a scale of 0 counts as 2^-60
    tol = attend_tolerance(s, want, big) + 448 * 2.0 ** -60
    assert ((out.double() - want).abs() <= tol).all()
