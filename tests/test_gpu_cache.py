"""The paged cache on the GPU: append (rotary, quantisation), read, commit and
tree attention, each against plain 64-bit implementations."""
import math

import numpy as np
import pytest
import torch

from cache_reference import HALF_STEP, Step, ancestors, attend_tolerance, rotate64

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


# ---- append ----------------------------------------------------------------------

def plain_quantise(x32):
    """(e4m3, scale) of float32 rows, by the written definition."""
    scale = x32.abs().amax(-1).clamp(min=2.0 ** -40) * (1.0 / 448.0)
    return (x32 / scale[..., None]).to(E4), scale


APPEND = [
    dict(ctx=[0], nodes=[1]),
    dict(ctx=[15, 16, 17, 31], nodes=[2, 1, 0, 5], page=16),
    dict(ctx=[100, 3], nodes=[29, 40], tree="random", page=48, kv_heads=3, group=2),
    dict(ctx=[7] * 40, nodes=[3] * 40, tree="star", page=8, kv_heads=1, group=7, head_dim=64),
    dict(ctx=[0, 1000], nodes=[64, 1], page=64, head_dim=64, dtype=HF),
]


@pytest.mark.parametrize("case", range(len(APPEND)))
@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("rotary", [None, (16, True), (64, False), ("all", False), ("all", True), (48, False)])
def test_append(V, case, eight, rotary):
    kw = dict(APPEND[case])
    dt = kw.get("dtype", BF)
    s = Step(**kw, cache=E4 if eight else dt, seed=case, extra_rows=2)
    from speculative_decoding_rejection_decode_gb300 import rotary_table
    table, freq, inter = None, None, False
    if rotary:
        dim, inter = (s.head_dim if rotary[0] == "all" else rotary[0]), rotary[1]
        table = rotary_table(1100, dim)
        freq = [10000.0 ** (-2.0 * i / dim) for i in range(dim // 2)]
    before = [None if t is None else t.clone() for t in (s.k, s.v, s.ks, s.vs)]
    marker = torch.full_like(s.q, 7.0)
    q = s.cache(V).append(s.new_k, s.new_v, *args(s), q=s.q, rotary=table, interleaved=inter, out_q=marker)
    assert V.get_error() == 0
    assert torch.equal(q[s.n_rows:], torch.full_like(q[s.n_rows:], 7.0))      # rows behind the last request
    touched = torch.zeros(s.num_pages, s.page, dtype=torch.bool, device="cuda")
    for b in range(s.B):
        for j in range(s.nodes[b]):
            page, off = s.row(b, s.ctx[b] + j)
            touched[page, off] = True
            r = s.firsts[b] + j
            pos = s.ctx[b] + len(ancestors(s.parents[b], j)) - 1
            k64, v64, q64 = s.new_k[r].double(), s.new_v[r].double(), s.q[r].double()
            if freq:
                k64 = rotate64(k64, pos, freq, 1.0, inter)
                q64 = rotate64(q64, pos, freq, 1.0, inter)
            # q: 32-bit products of |x| <= 6 with tables good to 2^-24 (two
            # products, one sum: below 2^-19), then one rounding
            assert ((q[r].double() - q64).abs() <= HALF_STEP[dt] * q64.abs() + 2.0 ** -19).all()
            for got, sc, x in ((s.k, s.ks, k64), (s.v, s.vs, v64)):
                g = got[page, :, off].float().double()
                if not eight:
                    assert ((g - x).abs() <= HALF_STEP[dt] * x.abs() + 2.0 ** -19).all()
                    continue
                scale = sc[page, :, off].double()
                amax = x.abs().amax(-1)
                assert ((scale - amax / 448).abs() <= (2.0 ** -19 + 2.0 ** -23 * amax) / 448).all()
                # half a step of e4m3 (2^-4 relative, 2^-10 absolute below its
                # normal numbers), and the 32-bit rotation's error
                bound = torch.maximum(2.0 ** -4 * x.abs(), 2.0 ** -10 * scale[:, None]) * (1 + 2.0 ** -10) + 2.0 ** -18
                assert ((g * scale[:, None] - x).abs() <= bound).all()
                if x is v64:   # no rotation: bytes and scales are exact
                    want, ws = plain_quantise(s.new_v[r].float())
                    assert torch.equal(want.view(torch.uint8), got[page, :, off].view(torch.uint8))
                    assert torch.equal(ws, sc[page, :, off])
    for now, was in zip((s.k, s.v, s.ks, s.vs), before):     # every other slot is as it was
        if now is not None:
            flat = (lambda t: t.view(torch.uint8) if t.dtype == E4 else t.view(torch.int16) if t.element_size() == 2 else t.view(torch.int32))
            same = (flat(now) == flat(was)).transpose(1, 2)
            assert same[~touched].all()


def test_rotated_rows_quantise_exactly_as_written(V):
    # the 32-bit formula with each product and sum rounded is a function of the
    # inputs: the kernel's bytes equal elementary torch operations'
    from speculative_decoding_rejection_decode_gb300 import rotary_table
    for inter in (False, True):
        s = Step(ctx=[9, 70], nodes=[33, 20], cache=E4, seed=5)
        table = rotary_table(128, 128)
        s.cache(V).append(s.new_k, s.new_v, *args(s), rotary=table, interleaved=inter)
        for b in range(2):
            pos = torch.arange(s.nodes[b], device="cuda") + s.ctx[b]
            cos, sin = table[pos, 0][:, None], table[pos, 1][:, None]
            x = s.new_k[s.firsts[b]:s.firsts[b + 1]].float()
            a, c = (x[..., 0::2], x[..., 1::2]) if inter else (x[..., :64], x[..., 64:])
            ra, rc = a * cos - c * sin, c * cos + a * sin
            y = torch.stack([ra, rc], -1).flatten(-2) if inter else torch.cat([ra, rc], -1)
            want, scale = plain_quantise(y)
            for j in range(s.nodes[b]):
                page, off = s.row(b, s.ctx[b] + j)
                assert torch.equal(want[j].view(torch.uint8), s.k[page, :, off].view(torch.uint8))
                assert torch.equal(scale[j], s.ks[page, :, off])


def test_append_strided_rows_and_special_values(V):
    s = Step(ctx=[5, 0], nodes=[4, 3], kv_heads=2, group=2, cache=E4, seed=2)
    row = torch.randn(s.N, 8, 128, device="cuda").to(BF)                     # one projection's row
    q, k, v = row.split([4, 2, 2], 1)
    assert not k.is_contiguous()
    v[0, 0] = 0.0                                                            # zeros: the least scale
    v[1, 0, 3] = math.inf
    v[2, 0, 5] = math.nan
    v[3, 1] = 1e-20
    got = s.cache(V).append(k, v, *args(s), q=q)
    assert torch.equal(got, q)                                               # no table: copied
    for r, (b, j) in enumerate([(0, 0), (0, 1), (0, 2), (0, 3), (1, 0), (1, 1), (1, 2)]):
        page, off = s.row(b, s.ctx[b] + j)
        for x, y, sc in ((k, s.k, s.ks), (v, s.v, s.vs)):
            want, ws = plain_quantise(x[r].float())
            val = want.float() * ws[:, None]
            mine = y[page, :, off].float() * sc[page, :, off][:, None]
            assert torch.equal(val.isnan(), mine.isnan())
            assert torch.equal(val.nan_to_num(), mine.nan_to_num())


def test_append_bad_pages_positions_and_trees(V):
    from speculative_decoding_rejection_decode_gb300 import rotary_table

    def fresh(**kw):
        s = Step(ctx=[3, 20, 9], nodes=[4, 4, 4], tree="random", page=8, seed=3, poison=False, **kw)
        return s, s.k.clone(), s.cache(V)

    s, k0, c = fresh()
    s.table[1, 20 // 8] = s.num_pages                       # one page outside the cache
    c.append(s.new_k, s.new_v, *args(s))
    assert V.get_error() == BAD_CACHE and V.get_error() == 0
    for b, n in ((0, 4), (2, 4)):                           # the others are written
        for j in range(n):
            page, off = s.row(b, s.ctx[b] + j)
            assert torch.equal(s.k[page, :, off], s.new_k[s.firsts[b] + j])
    s, k0, c = fresh()
    s.lengths[2] = 1000                                     # slots outside the table
    s.lengths[0] = -1
    c.append(s.new_k, s.new_v, *args(s))
    assert V.get_error() == BAD_CACHE
    page, off = s.row(1, 20)
    assert torch.equal(s.k[page, :, off], s.new_k[4])
    for b in (0, 2):
        for j in range(4):
            page, off = s.row(b, s.ctx[b] + j)
            assert torch.equal(s.k[page, :, off], k0[page, :, off])
    s, k0, c = fresh()
    table = rotary_table(22, 128)                           # request 1 passes position 21
    q = c.append(s.new_k, s.new_v, *args(s), q=s.q, rotary=table)
    deep = [len(ancestors(s.parents[1], j)) - 1 for j in range(4)]
    assert (V.get_error() == BAD_CACHE) == any(20 + d > 21 for d in deep)
    for j in range(4):
        assert bool((q[4 + j] == 0).all()) == (20 + deep[j] > 21)
    s, k0, c = fresh()
    s.parent[5] = 3                                         # node 1 of request 1: no earlier node
    c.append(s.new_k, s.new_v, *args(s), rotary=rotary_table(64, 128))
    assert V.get_error() == BAD_TREE
    page, off = s.row(1, 21)
    assert torch.equal(s.k[page, :, off], k0[page, :, off])
    s, k0, c = fresh()
    s.cu[2] = 100                                           # passes the rows given
    c.append(s.new_k, s.new_v, *args(s))
    V.get_error()


@pytest.mark.parametrize("parents", [False, True])
def test_append_and_read_of_malformed_ranges(V, parents):
    from speculative_decoding_rejection_decode_gb300 import rotary_table
    table = rotary_table(64, 128)
    for at, value, hit in ((0, -3, 0), (3, 100, 2)):      # starts below 0; passes the rows given
        s = Step(ctx=[3, 20, 9], nodes=[4, 4, 4], tree="random" if parents else "chain", page=8, seed=3, poison=False)
        if parents:
            s.parent[:4] = torch.tensor([-1, 0, 1, 1], dtype=torch.int32, device="cuda")
        k0 = s.k.clone()
        cu = s.cu.clone()
        cu[at] = value
        out_q = torch.full_like(s.q, 7.0)
        s.cache(V).append(s.new_k, s.new_v, s.table, s.lengths, cu, s.parent, q=s.q, rotary=table, out_q=out_q)
        assert V.get_error() == BAD_CU
        out = (torch.full_like(s.new_k, 7.0), torch.full_like(s.new_k, 7.0))
        s.cache(V).read(s.table, s.lengths, cu, out=out)
        assert V.get_error() == BAD_CU
        for b in range(3):
            for j in range(4):
                page, off = s.row(b, s.ctx[b] + j)
                r = s.firsts[b] + j
                assert torch.equal(s.k[page, :, off], k0[page, :, off]) == (b == hit)
                assert bool((out_q[r] == 7.0).all()) == (b == hit)
                assert torch.equal(out[0][r], torch.full_like(out[0][r], 7.0) if b == hit else s.k[page, :, off])


# ---- read --------------------------------------------------------------------------

@pytest.mark.parametrize("cache,dtype,head_dim,page", [(E4, BF, 128, 16), (E4, HF, 64, 48), (BF, BF, 128, 7), (HF, HF, 64, 64)])
def test_read(V, cache, dtype, head_dim, page):
    s = Step(ctx=[0, 1, 33, 100, 0, 257], nodes=[0, 1, 2, 0, 3, 1], cache=cache, dtype=dtype, head_dim=head_dim, page=page, seed=4)
    c = s.cache(V)
    starts = [0, 0, 5, 99, 0, 100]
    counts = [0, 2, 30, 1, 3, 158]
    cu = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    st = torch.tensor(starts, dtype=torch.int32, device="cuda")
    n = sum(counts)
    out = (torch.full((n + 3, 2, head_dim), 7.0, dtype=dtype, device="cuda"), torch.full((n + 3, 2, head_dim), 7.0, dtype=dtype, device="cuda"))
    c.read(s.table, st, cu, out=out)
    assert V.get_error() == 0
    for got, which in zip(out, "kv"):
        val = s.values(which)
        r = 0
        for b in range(s.B):
            for j in range(counts[b]):
                page_, off = s.row(b, starts[b] + j)
                want = val[page_, :, off]
                # a 32-bit product rounded, then the type's rounding (its
                # subnormals: half of the least step)
                tiny = 2.0 ** -25 if dtype == HF else 0.0
                assert ((got[r].double() - want).abs() <= (HALF_STEP[dtype] + 2.0 ** -23) * want.abs() + tiny).all()
                r += 1
        assert (got[n:] == 7.0).all()
    k, v = c.read(s.table, st, cu)
    assert torch.equal(k, out[0][:n].to(k.dtype)) if k.dtype == dtype else k.dtype == BF
    s.table[3, 99 // page] = -5
    s.lengths[0] = 0
    k, v = c.read(s.table, st, cu, dtype=dtype, n_rows=n)
    assert V.get_error() == BAD_CACHE
    assert (k[32] == 0).all() and (v[32] == 0).all()
    assert torch.equal(k[:32], out[0][:32]) and torch.equal(k[33:], out[0][33:n])


# ---- commit ------------------------------------------------------------------------

@pytest.mark.parametrize("cache,head_dim,page", [(BF, 128, 16), (E4, 64, 5), (E4, 128, 64)])
@pytest.mark.parametrize("inplace", [False, True])
def test_commit(V, cache, head_dim, page, inplace):
    rng = np.random.default_rng(7)
    nodes = [1, 0, 29, 12, 40, 2, 30]
    s = Step(ctx=[0, 4, 31, 7, 100, 16, 3], nodes=nodes, tree="random", cache=cache, head_dim=head_dim, page=page, seed=6)
    path = np.full(s.n_rows, -1, np.int32)
    acc = np.zeros(s.B, np.int32)
    for b, n in enumerate(nodes):
        if n:
            p = sorted(ancestors(s.parents[b], int(rng.integers(0, n))))[1:]
            if b == 2:
                p = list(range(2, 20, 3))             # any rising path moves the same way
            acc[b] = len(p)
            path[s.firsts[b]:s.firsts[b] + len(p)] = p
    before = [None if t is None else t.clone() for t in (s.k, s.v, s.ks, s.vs)]
    d = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    lengths = s.lengths.clone()
    got = s.cache(V).commit(s.table, lengths, s.cu, d(acc), d(path), out_lengths=lengths if inplace else None)
    assert V.get_error() == 0
    assert got.tolist() == [c + (1 + int(a) if n else 0) for c, a, n in zip(s.ctx, acc, nodes)]
    assert inplace or lengths.tolist() == s.ctx
    for now, was in zip((s.k, s.v, s.ks, s.vs), before):
        if now is None:
            continue
        want = was.clone()
        w8 = want.view(torch.uint8) if want.dtype == E4 else want
        o8 = was.view(torch.uint8) if was.dtype == E4 else was
        for b in range(s.B):
            for i in range(int(acc[b])):
                sp, so = s.row(b, s.ctx[b] + int(path[s.firsts[b] + i]))
                dp, do = s.row(b, s.ctx[b] + 1 + i)
                w8[dp, :, do] = o8[sp, :, so]
        n8 = now.view(torch.uint8) if now.dtype == E4 else now
        assert torch.equal(n8.view(torch.uint8), w8.view(torch.uint8))
    # chains: only the lengths change
    k0 = s.k.view(torch.uint8).clone()
    got = s.cache(V).commit(s.table, s.lengths, s.cu, d(acc))
    assert got.tolist() == [c + (1 + int(a) if n else 0) for c, a, n in zip(s.ctx, acc, nodes)]
    assert torch.equal(k0, s.k.view(torch.uint8)) and V.get_error() == 0


@pytest.mark.parametrize("acc,path,code", [
    ([1, 5], [1, -1, -1, 1, 2, 3, 4], BAD_TREE),       # more than the request's nodes
    ([-1, 1], [1, -1, -1, 2, -1, -1, -1], BAD_TREE),
    ([2, 1], [2, 2, -1, 2, -1, -1, -1], BAD_TREE),     # the same node twice
    ([2, 1], [2, 1, -1, 2, -1, -1, -1], BAD_TREE),     # does not rise
    ([1, 1], [3, -1, -1, 2, -1, -1, -1], BAD_TREE),    # outside the request
    ([1, 1], [0, -1, -1, 2, -1, -1, -1], BAD_TREE),    # the root
])
def test_commit_refuses_bad_paths(V, acc, path, code):
    s = Step(ctx=[9, 2], nodes=[3, 4], tree="star", seed=8, poison=False)
    k0 = s.k.clone()
    d = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    got = s.cache(V).commit(s.table, s.lengths, s.cu, d(acc), d(path))
    assert V.get_error() == code
    bad = 1 if acc[1] > 3 else 0
    assert got[bad] == s.ctx[bad]
    pages = s.pages[bad]
    assert torch.equal(s.k[pages], k0[pages])
    assert int(got[1 - bad]) == s.ctx[1 - bad] + 1 + acc[1 - bad]


def test_commit_bad_page(V):
    s = Step(ctx=[9, 2], nodes=[3, 4], tree="star", seed=8, poison=False, page=4)
    s.table[0, 2] = 99
    d = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    got = s.cache(V).commit(s.table, s.lengths, s.cu, d([1, 1]), d([2, -1, -1, 2, -1, -1, -1]))
    assert V.get_error() == BAD_CACHE and got.tolist() == [9, 4]


# ---- attention ---------------------------------------------------------------------

ATTEND = [
    dict(ctx=[0], nodes=[1]),
    dict(ctx=[1, 0, 5], nodes=[1, 1, 1], group=1),
    dict(ctx=[126, 127, 128, 129, 255, 256], nodes=[1] * 6, kv_heads=1, group=8),
    dict(ctx=[500], nodes=[1], kv_heads=8, group=4),
    dict(ctx=[0, 63, 64, 300, 17], nodes=[0, 9, 3, 8, 2], page=64),
    dict(ctx=[700, 31, 0], nodes=[29, 16, 40], tree="random", page=48),
    dict(ctx=[33, 1500], nodes=[64, 64], tree="random", kv_heads=2, group=7, page=100),
    dict(ctx=[250] * 20, nodes=[5] * 20, tree="star", kv_heads=1, group=2, page=8),
    dict(ctx=[10, 0], nodes=[300, 130], group=1, kv_heads=1),                  # long chains: many row tiles
    dict(ctx=[3], nodes=[200], tree="random", group=4, kv_heads=1),
    dict(ctx=[2], nodes=[33], group=16, kv_heads=2),
    dict(ctx=[3000, 5, 0, 1], nodes=[2, 1, 1, 3], kv_heads=4, group=4, page=128),
]


@pytest.mark.parametrize("case", range(len(ATTEND)))
@pytest.mark.parametrize("dtype,cache,head_dim", [(BF, BF, 128), (HF, HF, 64), (BF, E4, 128), (HF, E4, 64), (HF, HF, 128), (BF, BF, 64),
                                                  (HF, E4, 128), (BF, E4, 64)])
def test_attend(V, case, dtype, cache, head_dim):
    s = Step(**ATTEND[case], dtype=dtype, cache=cache, head_dim=head_dim, seed=case, extra_rows=1)
    out = torch.full((s.N, s.heads, head_dim), 7.0, dtype=dtype, device="cuda")
    s.cache(V).attend(s.q, *args(s), out=out)
    assert V.get_error() == 0
    assert (out[s.n_rows:] == 7.0).all()
    want, big = s.attend()
    err = (out[:s.n_rows].double() - want).abs()
    assert (err <= attend_tolerance(s, want, big)).all(), float((err - attend_tolerance(s, want, big)).max())


def test_attend_scale_strides_and_repeat(V):
    s = Step(ctx=[77, 400], nodes=[7, 3], tree="random", seed=1, group=4)
    wide = torch.randn(s.N, s.heads + 4, 128, device="cuda").to(BF)
    s.q = wide[:, 2:2 + s.heads]
    table = torch.zeros(2, 60, dtype=torch.int32, device="cuda")
    table[:, :s.table.shape[1]] = s.table
    got = s.cache(V).attend(s.q, table[:, :40], s.lengths, s.cu, s.parent, scale=0.05)
    want, big = s.attend(scale=0.05)
    assert ((got.double() - want).abs() <= attend_tolerance(s, want, big)).all()
    for _ in range(3):      # the same bits every time
        assert torch.equal(got, s.cache(V).attend(s.q, table[:, :40], s.lengths, s.cu, s.parent, scale=0.05))


@pytest.mark.parametrize("cache", [BF, E4])
@pytest.mark.parametrize("nodes", [2, 9])
@pytest.mark.parametrize("scale", [0.0, -0.07, 1e-30])
def test_attend_odd_scales(V, cache, nodes, scale):
    s = Step(ctx=[300, 40], nodes=[nodes, nodes], tree="star", cache=cache, seed=4)
    got = s.cache(V).attend(s.q, *args(s), scale=scale)
    want, big = s.attend(scale=scale)
    assert V.get_error() == 0
    assert ((got.double() - want).abs() <= attend_tolerance(s, want, big)).all()


@pytest.mark.parametrize("nodes", [2, 9])
@pytest.mark.parametrize("power", [-120, 100])
def test_attend_queries_of_any_size(V, nodes, power):
    # 8-bit caches: the kernels scale a query row by a power of two
    s = Step(ctx=[300, 40], nodes=[nodes, nodes], cache=E4, seed=5)
    s.q *= 2.0 ** power
    got = s.cache(V).attend(s.q, *args(s), scale=2.0 ** (-3.5 - power) if power > 0 else None)
    want, big = s.attend(scale=2.0 ** (-3.5 - power) if power > 0 else None)
    assert ((got.double() - want).abs() <= attend_tolerance(s, want, big)).all()


@pytest.mark.parametrize("nodes", [1, 12])
@pytest.mark.parametrize("page", [64, 40])
def test_attend_scales_off_16_bytes(V, nodes, page):
    s = Step(ctx=[700, 90], nodes=[nodes, nodes], cache=E4, page=page, seed=6)
    want = s.cache(V).attend(s.q, *args(s))
    for name in ("ks", "vs"):
        flat = torch.empty(getattr(s, name).numel() + 1, device="cuda")[1:]
        flat.copy_(getattr(s, name).reshape(-1))
        setattr(s, name, flat.view(s.ks.shape) if name == "ks" else flat.view(s.k.shape[:3]))
    assert torch.equal(s.cache(V).attend(s.q, *args(s)), want)


@pytest.mark.parametrize("cache", [BF, E4])
@pytest.mark.parametrize("nodes", [1, 7])
def test_attend_many_requests(V, cache, nodes):
    # more requests than CTAs, some without nodes or context
    rng = np.random.default_rng(2)
    ctx = [int(x) for x in rng.integers(0, 400, 400)]
    ctx[5] = ctx[399] = 0
    n = [0 if i % 17 == 3 else nodes for i in range(400)]
    s = Step(ctx=ctx, nodes=n, kv_heads=2, group=4, head_dim=64, page=32, cache=cache, seed=7)
    got = s.cache(V).attend(s.q, *args(s))
    want, big = s.attend()
    assert V.get_error() == 0
    assert ((got.double() - want).abs() <= attend_tolerance(s, want, big)).all()


def test_attend_far_contexts(V):
    # one request over 70000 keys: every range of the work holds a part of it
    s = Step(ctx=[70000], nodes=[6], kv_heads=1, group=8, page=64, seed=8)
    got = s.cache(V).attend(s.q, *args(s))
    want, big = s.attend()
    # float32 sums over 2^17 keys instead of the bound's 2^11: 2^6 times its 2^-13
    tol = attend_tolerance(s, want, big) + (2.0 ** -7 - 2.0 ** -13) * big[..., None]
    assert ((got.double() - want).abs() <= tol).all()
    # and on average far below: weights rounded at random
    assert float((got.double() - want).norm() / want.norm()) < 2 * 2.0 ** -8


def test_outputs_in_place_and_overlapping(V):
    from speculative_decoding_rejection_decode_gb300 import rotary_table
    table = rotary_table(600, 128)
    for inter in (False, True):
        s = Step(ctx=[500, 3], nodes=[9, 30], tree="random", seed=9)
        want = s.cache(V).append(s.new_k, s.new_v, *args(s), q=s.q, rotary=table, interleaved=inter)
        got = s.cache(V).append(s.new_k, s.new_v, *args(s), q=s.q, rotary=table, interleaved=inter, out_q=s.q)
        assert got is s.q and torch.equal(got, want)
    with pytest.raises(ValueError):
        s.cache(V).attend(s.q, *args(s), out=s.q)
    wide = torch.zeros(2 * s.N, s.heads, 128, dtype=BF, device="cuda")
    with pytest.raises(ValueError):
        s.cache(V).attend(wide[1:s.N + 1], *args(s), out=wide[:s.N])
    s.cache(V).attend(wide[:s.N], *args(s), out=wide[s.N:])      # side by side is fine


@pytest.mark.parametrize("cache", [BF, E4])
@pytest.mark.parametrize("nodes", [4, 40])
def test_values_of_hidden_nodes_reach_no_row(V, cache, nodes):
    # infinities and NaN in a sibling's key and value; the rows that see it get them
    s = Step(ctx=[50, 11], nodes=[nodes, nodes], tree="star", cache=cache, seed=9)
    for b, j, what in ((0, 2, math.inf), (1, 3, math.nan)):
        page, off = s.row(b, s.ctx[b] + j)
        if cache == E4:
            s.v.view(torch.uint8)[page, 0, off, 5] = 0x7F
            s.k.view(torch.uint8)[page, 1, off, 5] = 0x7F
        else:
            s.v[page, 0, off, 5] = what
            s.k[page, 1, off, 5] = what
    out = s.cache(V).attend(s.q, *args(s))
    want, big = s.attend()
    big = big.nan_to_num(0, 0, 0)
    for b, bad in ((0, 2), (1, 3)):
        for j in range(nodes):
            r = s.firsts[b] + j
            if j != bad:
                assert out[r].isfinite().all()
                ok = (out[r].double() - want[r]).abs() <= attend_tolerance(s, want, big)[r]
                assert ok.all()
            else:
                assert not out[r, :s.group, 5].isfinite().any()
                rest = out[r, :s.group].clone()
                rest[:, 5] = 0
                assert rest.isfinite().all()


def test_extreme_scores_and_scales(V):
    s = Step(ctx=[300], nodes=[3], seed=10)
    s.q[0] *= 200.0                       # one key takes all the weight
    s.k[s.pages[0][0], :, 3] = -30000.0   # scores far below and above the rest
    s.q[1] = 0.0                          # all weights equal
    out = s.cache(V).attend(s.q, *args(s))
    want, big = s.attend()
    # row 0's scores are 200 times larger, and so is their rounding error
    tol = attend_tolerance(s, want, big)
    tol[0] += 200 * 2 * 2.3e-4 * big[0][:, None]
    assert ((out.double() - want).abs()[1:2] <= tol[1:2]).all() and out.isfinite().all()
    s = Step(ctx=[300], nodes=[3], cache=E4, seed=10)
    s.q *= 2.0 ** -30                     # queries that f16 alone would lose
    s.ks *= 2.0 ** 30
    s.vs[s.pages[0][0]] = 1e-12           # rows of nearly nothing, with weight
    s.vs[s.pages[0][1], :, 2] = 0.0
    out = s.cache(V).attend(s.q, *args(s))
    want, big = s.attend()
    assert ((out.double() - want).abs() <= attend_tolerance(s, want, big)).all()


def test_attend_bad_pages_lengths_and_trees(V):
    s = Step(ctx=[100, 40, 9], nodes=[3, 4, 5], tree="random", page=16, seed=11)
    c = s.cache(V)
    good = c.attend(s.q, *args(s))
    table = s.table.clone()
    table[0, 2] = s.num_pages + 7                         # 16 keys hidden
    got = c.attend(s.q, table, s.lengths, s.cu, s.parent)
    assert V.get_error() == BAD_CACHE
    assert torch.equal(got[3:], good[3:]) and got.isfinite().all()
    K, W = s.values("k"), s.values("v")
    for i in range(3):
        at = [x for x in range(100) if not 32 <= x < 48] + [100 + j for j in ancestors(s.parents[0], i)]
        rows = [s.row(0, x) for x in at]
        k = torch.stack([K[p, :, o] for p, o in rows])
        v = torch.stack([W[p, :, o] for p, o in rows])
        q = s.q[i].double().view(s.kv_heads, s.group, -1)
        w = torch.softmax(torch.einsum("hgd,shd->hgs", q, k) / math.sqrt(128), -1)
        want = torch.einsum("hgs,shd->hgd", w, v).reshape(s.heads, -1)
        assert ((got[i].double() - want).abs() <= (2.0 ** -8 + 1e-3) * v.abs().max() + 2.0 ** -8 * want.abs()).all()
    table = s.table.clone()
    table[2, :] = -1                                      # a request that sees no key
    got = c.attend(s.q, table, s.lengths, s.cu, s.parent)
    assert V.get_error() == BAD_CACHE and (got[7:] == 0).all() and torch.equal(got[:7], good[:7])
    for name, change, code in (("len", -1, BAD_CACHE), ("len", 1000, BAD_CACHE), ("cu", 90, BAD_CU)):
        lengths, cu = s.lengths.clone(), s.cu.clone()
        if name == "len":
            lengths[2] = change
        else:
            cu[3] = change
        out = torch.full_like(s.q, 7.0)
        c.attend(s.q, s.table, lengths, cu, s.parent, out=out)
        assert V.get_error() == code
        assert (out[7:] == 7.0).all()
        assert torch.equal(out[:7], good[:7])
    parent = s.parent.clone()
    parent[8] = 4                                         # node 1 of request 2: no earlier node
    out = c.attend(s.q, s.table, s.lengths, s.cu, parent)
    assert V.get_error() == BAD_TREE and torch.equal(out[:7], good[:7]) and out.isfinite().all()
    big = Step(ctx=[5], nodes=[1025], tree="star", kv_heads=1, group=1, seed=1)
    out = torch.full_like(big.q, 7.0)
    big.cache(V).attend(big.q, *args(big), out=out)
    assert V.get_error() == BAD_TREE and (out == 7.0).all()


def test_largest_tree(V):
    s = Step(ctx=[40], nodes=[1024], tree="random", kv_heads=1, group=1, seed=12, head_dim=64)
    out = s.cache(V).attend(s.q, *args(s))
    want, big = s.attend()
    assert V.get_error() == 0
    assert ((out.double() - want).abs() <= attend_tolerance(s, want, big)).all()


def test_pages_past_32_bit_offsets(V):
    # rows of the last pages lie past 2^31 elements (and 2^32 bytes)
    from speculative_decoding_rejection_decode_gb300 import KVCache
    pages, kv, page = 70000, 2, 128
    c = KVCache.empty(V, pages, page, kv, 128, BF)
    s = Step(ctx=[200], nodes=[3], kv_heads=kv, page=page, seed=13, poison=False)
    far = [pages - 1, pages - 2, 1][: len(s.pages[0])]
    for here, there in zip(s.pages[0], far):
        c.k[there], c.v[there] = s.k[here], s.v[here]
    table = torch.tensor([far], dtype=torch.int32, device="cuda")
    want = s.cache(V).attend(s.q, *args(s))
    assert torch.equal(c.attend(s.q, table, s.lengths, s.cu), want)
    c.append(s.new_k, s.new_v, table, s.lengths, s.cu)
    k, v = c.read(table, s.lengths, s.cu)
    assert torch.equal(k, s.new_k) and torch.equal(v, s.new_v)
    got = c.commit(table, s.lengths, s.cu, torch.tensor([1], dtype=torch.int32, device="cuda"),
                   torch.tensor([2, -1, -1], dtype=torch.int32, device="cuda"))
    k, _ = c.read(table, s.lengths, s.cu)
    assert got.tolist() == [202] and torch.equal(k[1], s.new_k[2]) and V.get_error() == 0


def test_tiles_of_pages_past_32_bit_offsets(V):
    from speculative_decoding_rejection_decode_gb300 import KVCache
    for page in (128, 24):                       # fetched as boxes of 128 rows, and of 8
        pages, kv = 70000 * 128 // page, 2
        c = KVCache.empty(V, pages, page, kv, 128, BF)
        s = Step(ctx=[200], nodes=[9], kv_heads=kv, page=page, tree="random", seed=13, poison=False)
        far = [pages - 1 - i if i % 2 else i for i in range(1, len(s.pages[0]) + 1)]
        for here, there in zip(s.pages[0], far):
            c.k[there], c.v[there] = s.k[here], s.v[here]
        table = torch.tensor([far], dtype=torch.int32, device="cuda")
        want = s.cache(V).attend(s.q, *args(s))
        assert torch.equal(c.attend(s.q, table, s.lengths, s.cu, s.parent), want)
        del c


@pytest.mark.parametrize("nodes", [3, 40])
def test_values_near_the_largest(V, nodes):
    # scales of 8-bit values far above and below one: what bf16 rows may hold
    for power in (-40, 100, 116):
        s = Step(ctx=[300], nodes=[nodes], cache=E4, seed=15)
        s.vs *= 2.0 ** power
        out = s.cache(V).attend(s.q, *args(s))
        want, big = s.attend()
        assert ((out.double() - want).abs() <= attend_tolerance(s, want, big)).all()


@pytest.mark.parametrize("cache", [BF, E4])
def test_infinite_value_in_a_deep_tree(V, cache):
    s = Step(ctx=[50], nodes=[1000], kv_heads=1, group=1, head_dim=64, tree="random", cache=cache, seed=16)
    s.parent[:] = torch.arange(1000, device="cuda", dtype=torch.int32) - 1   # one branch
    clean = s.cache(V).attend(s.q, *args(s))
    page, off = s.row(0, 52)
    if cache == E4:
        s.v.view(torch.uint8)[page, 0, off, 5] = 0x7F
    else:
        s.v[page, 0, off, 5] = math.inf
    out = s.cache(V).attend(s.q, *args(s))
    assert V.get_error() == 0
    assert torch.equal(out[:2], clean[:2]) and not out[2:, :, 5].isfinite().any()
    out[:, :, 5] = clean[:, :, 5]
    assert torch.equal(out, clean)


# ---- graphs and streams -------------------------------------------------------------

def test_two_graphs_of_one_handle_on_two_streams(V):
    """Captured calls have workspaces of their own: replays may overlap."""
    steps = [Step(ctx=[2000, 700, 30], nodes=[6, 29, 1], tree="random", kv_heads=4, seed=s, cache=E4) for s in (1, 2)]
    eager, graphs = [], []
    for s in steps:
        c = s.cache(V)
        c.append(s.new_k, s.new_v, *args(s), q=s.q)
        eager.append((c.attend(s.q, *args(s)), *c.read(s.table, s.lengths, s.cu, n_rows=s.n_rows)))
    torch.cuda.synchronize()
    for s in steps:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c = s.cache(V)
            c.append(s.new_k, s.new_v, *args(s), q=s.q)
            out = (c.attend(s.q, *args(s)), *c.read(s.table, s.lengths, s.cu, n_rows=s.n_rows))
        graphs.append((g, out))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        for (g, _o), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for (_g, out), want in zip(graphs, eager):
        for a, b in zip(out, want):
            assert torch.equal(a, b)
    # new lengths in the captured tensors: the work follows them
    s, (g, out) = steps[0], graphs[0]
    s.lengths.copy_(torch.tensor([5, 699, 0], dtype=torch.int32))
    g.replay()
    want = s.cache(V).attend(s.q, *args(s))
    torch.cuda.synchronize()
    assert torch.equal(out[0], want) and V.get_error() == 0


def test_calls_on_a_side_stream(V):
    s = Step(ctx=[900, 30], nodes=[6, 9], tree="random", seed=3)
    want = s.cache(V).attend(s.q, *args(s))
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        q = s.q * 1.0
        got = s.cache(V).attend(q, *args(s))
    st.synchronize()
    assert torch.equal(got, want)


def test_no_rows_at_all(V):
    s = Step(ctx=[4, 0], nodes=[0, 0], seed=1)
    c = s.cache(V)
    assert c.attend(s.q, *args(s)).shape == (0, s.heads, 128)
    assert c.append(s.new_k, s.new_v, *args(s), q=s.q).shape == (0, s.heads, 128)
    assert c.read(s.table, s.lengths, s.cu)[0].shape[0] == 0
    z = torch.zeros(2, dtype=torch.int32, device="cuda")
    assert c.commit(s.table, s.lengths, s.cu, z, z[:0]).tolist() == [4, 0]
    assert V.get_error() == 0


# ---- a step as it is used -------------------------------------------------------------

@pytest.mark.parametrize("cache", [BF, E4])
def test_speculative_steps_reproduce_plain_decoding(V, cache):
    """Greedy decoding of a one-layer model, token by token, against steps that
    draft trees, append them, attend, verify (Verifier.tree) and commit: the same
    tokens, and the cache of the accepted tokens holds the same rows."""
    from speculative_decoding_rejection_decode_gb300 import KVCache, rotary_table
    g = torch.Generator(device="cuda")
    g.manual_seed(21)
    H, Hkv, D, vocab, B, steps = 4, 2, 64, 97, 3, 24
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    embed, wq, wk, wv, wo = r(vocab, 64), r(64, H * D), r(64, Hkv * D), r(64, Hkv * D), r(H * D, vocab)
    table = rotary_table(256, D)
    pages = torch.arange(B * 16, dtype=torch.int32, device="cuda").view(B, 16).flip(1).contiguous()

    # projections of every token once: a library product's rounding may depend on
    # how many rows it has, and the caches are compared bit for bit
    made = {h: (embed @ w / 8).view(-1, n, D).to(BF) for h, w, n in (("q", wq, H), ("k", wk, Hkv), ("v", wv, Hkv))}

    def forward(c, tokens, lengths, cu, parent):
        x = embed[tokens.long()]
        row = lambda w, h: made["q" if w is wq else "k" if w is wk else "v"][tokens.long()]
        q = c.append(row(wk, Hkv), row(wv, Hkv), pages, lengths, cu, parent, q=row(wq, H), rotary=table)
        o = c.attend(q, pages, lengths, cu, parent)
        return (o.float().flatten(1) @ wo + 0.3 * x[:, :1]) .to(torch.float32)

    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    # token by token
    c1 = KVCache.empty(V, B * 16, 8, Hkv, D, cache)
    cur, lengths, cu1 = i32([1, 2, 3]), torch.zeros(B, dtype=torch.int32, device="cuda"), i32([0, 1, 2, 3])
    plain = []
    for t in range(steps):
        cur = forward(c1, cur, lengths, cu1, None).argmax(1).to(torch.int32)
        lengths = lengths + 1
        plain.append(cur)
    plain = torch.stack(plain, 1).tolist()
    # trees: the true next tokens hidden among wrong ones, breaking off after a few
    rng = np.random.default_rng(3)
    c2 = KVCache.empty(V, B * 16, 8, Hkv, D, cache)
    lengths = torch.zeros(B, dtype=torch.int32, device="cuda")
    done = [[] for _ in range(B)]
    last = [1, 2, 3]
    while min(len(d) for d in done) < steps - 8:
        toks, pars, cu = [], [], [0]
        for b in range(B):
            tk, par, at = [last[b]], [-1], 0
            for level in range(3):
                n0 = len(tk)
                right = int(rng.integers(0, 3))
                want = plain[b][len(done[b]) + level] if len(done[b]) + level < steps else 0
                for k in range(3):
                    wrong = int(rng.integers(0, vocab))
                    tk.append(want if k == right and rng.random() < 0.8 else wrong)
                    par.append(at)
                at = n0 + right
            toks += tk
            pars += par
            cu.append(len(toks))
        toks, pars, cu = i32(toks), i32(pars), i32(cu)
        logits = forward(c2, toks, lengths, cu, pars)
        out = V.tree(logits, None, toks, pars, cu, 0.0, 0)
        lengths = c2.commit(pages, lengths, cu, out.num_accepted, out.path, out_lengths=lengths)
        for b in range(B):
            n = int(out.num_accepted[b])
            got = out.tokens[int(cu[b]):int(cu[b]) + n + 1].tolist()
            done[b] += got
            last[b] = got[-1]
        assert V.get_error() == 0
    for b in range(B):
        n = min(steps, len(done[b]))
        assert done[b][:n] == plain[b][:n], b
    assert int(lengths.sum()) == sum(len(d) for d in done)
    n = [min(steps, len(d)) for d in done]
    cu = i32(np.concatenate([[0], np.cumsum(n)]).astype(np.int32))
    zero = torch.zeros(B, dtype=torch.int32, device="cuda")
    for a, b in zip(c1.read(pages, zero, cu), c2.read(pages, zero, cu)):
        assert torch.equal(a, b)
