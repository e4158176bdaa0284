"""Rotary positions with several axes on the GPU: on the way into the cache and on
dense rows."""
import math

import pytest
import torch

from cache_reference import HALF_STEP, Step, ancestors, rotate64

pytestmark = pytest.mark.gpu

BF, HF, E4 = torch.bfloat16, torch.float16, torch.float8_e4m3fn
BAD_CACHE, BAD_TREE = 32, 16


@pytest.fixture(scope="module")
def V():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_rejection_decode_gb300 import Verifier
    v = Verifier(0)
    yield v
    v.close()


def args(s):
    return s.table, s.lengths, s.cu


def plain_turn(x, positions, axes, table, inter, way=1.0):
    """x [N, H, D] turned by elementary torch operations in 32 bits, products and sums
    rounded one by one: the kernels' bytes."""
    n = len(axes)
    at = positions.long()[torch.tensor(axes, device=x.device)].T
    pair = torch.arange(n, device=x.device)[None]
    cos, sin = table[at, 0, pair][:, None], way * table[at, 1, pair][:, None]
    x = x.float()
    a, b = (x[..., 0:2 * n:2], x[..., 1:2 * n:2]) if inter else (x[..., :n], x[..., n:2 * n])
    ra, rb = a * cos - b * sin, b * cos + a * sin
    y = torch.stack([ra, rb], -1).flatten(-2) if inter else torch.cat([ra, rb], -1)
    return torch.cat([y, x[..., 2 * n:]], -1)


AXES = [((8,), False), ((16, 24, 24), False), ((24, 20, 20), True), ((3, 5), False), ((1, 2, 3, 10), True), ((11, 1, 20), False)]


@pytest.mark.parametrize("sections,spread", AXES)
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("D,dtype", [(128, BF), (128, HF), (64, BF), (256, BF), (80, HF)])
@pytest.mark.parametrize("N", [1, 33, 5000])
def test_rotate(V, sections, spread, inter, D, dtype, N):
    from speculative_decoding_rejection_decode_gb300 import rotary_axes, rotary_table
    axes = rotary_axes(sections, spread=spread)
    if 2 * len(axes) > D:
        pytest.skip("fewer dimensions than pairs")
    g = torch.Generator(device="cuda")
    g.manual_seed(N + D)
    wide = torch.randn(N, 7, D, generator=g, device="cuda").to(dtype)
    x = wide[:, 1:6]
    table = rotary_table(300, 2 * len(axes))
    pos = torch.randint(0, 300, (len(sections), N), generator=g, device="cuda", dtype=torch.int32)
    got = V.rotate(x, pos, table, axes=axes, interleaved=inter)
    assert V.get_error() == 0 and got.is_contiguous()
    assert torch.equal(got, plain_turn(x, pos, axes, table, inter).to(dtype))
    back = V.rotate(got, pos, table, axes=axes, interleaved=inter, inverse=True)
    assert torch.equal(back, plain_turn(got, pos, axes, table, inter, -1.0).to(dtype))
    # in place, through the strides, and nothing beside the rows moves
    before = wide.clone()
    assert V.rotate(x, pos, table, axes=axes, interleaved=inter, out=x) is x
    assert torch.equal(x, got) and torch.equal(wide[:, 0], before[:, 0]) and torch.equal(wide[:, 6], before[:, 6])
    # against 64 bits: 32-bit products of |x| < 6 with tables good to 2^-24, one rounding
    n = min(N, 20)
    for r in range(n):
        want = before[r, 1:6].double()
        for i, a in enumerate(axes):
            p, q = (2 * i, 2 * i + 1) if inter else (i, i + len(axes))
            t = int(pos[a, r]) * 10000.0 ** (-2.0 * i / (2 * len(axes)))
            u, w = want[:, p].clone(), want[:, q].clone()
            want[:, p], want[:, q] = u * math.cos(t) - w * math.sin(t), w * math.cos(t) + u * math.sin(t)
        assert ((got[r].double() - want).abs() <= HALF_STEP[dtype] * want.abs() + 2.0 ** -19).all()


def test_the_gradient_is_the_turn_back(V):
    # <g, turn(x)> = <back(g), x>, up to the roundings of both sides: half a step of each
    # turned value, 5000 * 640 terms of size 1 with random signs, at most all alike
    from speculative_decoding_rejection_decode_gb300 import rotary_axes, rotary_table
    axes, table = rotary_axes((16, 24, 24), spread=True), rotary_table(300, 128)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x, y = (torch.randn(500, 5, 128, generator=g, device="cuda").to(HF) for _ in range(2))
    pos = torch.randint(0, 300, (3, 500), generator=g, device="cuda", dtype=torch.int32)
    a = (y.double() * V.rotate(x, pos, table, axes=axes).double())
    b = (V.rotate(y, pos, table, axes=axes, inverse=True).double() * x.double())
    assert abs(float(a.sum() - b.sum())) <= HALF_STEP[HF] * float(a.abs().sum() + b.abs().sum()) * 1.01


def test_rotate_refuses_positions_outside_the_table(V):
    from speculative_decoding_rejection_decode_gb300 import rotary_table
    table = rotary_table(50, 64)
    x = torch.randn(6, 3, 64, device="cuda").to(BF)
    good = torch.tensor([[0, 1, 49, 3, 4, 5], [5, 4, 3, 2, 1, 0]], dtype=torch.int32, device="cuda")
    axes = (0, 1) * 16
    want = V.rotate(x, good, table, axes=axes)
    bad = good.clone()
    bad[0, 1], bad[1, 3], bad[1, 4] = 50, -1, 2 ** 31 - 1
    got = V.rotate(x, bad, table, axes=axes)
    assert V.get_error() == BAD_CACHE
    lost = torch.tensor([1, 3, 4], device="cuda")
    assert (got[lost] == 0).all() and torch.equal(got[[0, 2, 5]], want[[0, 2, 5]])
    assert V.rotate(x[:0], good[:, :0], table, axes=axes).numel() == 0


def test_rotate_captured_and_on_another_stream(V):
    from speculative_decoding_rejection_decode_gb300 import rotary_table
    table = rotary_table(50, 64)
    x = torch.randn(600, 3, 64, device="cuda").to(BF)
    pos = torch.randint(0, 50, (600,), device="cuda", dtype=torch.int32)
    want = V.rotate(x, pos, table)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = V.rotate(x, pos, table)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        g.replay()
        other = V.rotate(x, pos, table)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(other, want)


APPEND = [dict(ctx=[0], nodes=[1]), dict(ctx=[15, 16, 17, 31], nodes=[2, 1, 0, 5], page=16),
          dict(ctx=[100, 3], nodes=[29, 400], tree="random", page=48, kv_heads=3, group=2),
          dict(ctx=[7] * 40, nodes=[3] * 40, page=8, kv_heads=1, group=7, head_dim=64),
          dict(ctx=[0, 1000], nodes=[6400, 1], page=64, head_dim=64, dtype=HF)]


@pytest.mark.parametrize("case", range(len(APPEND)))
@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("sections,spread", [((8,), False), ((10, 11, 11), False), ((12, 10, 10), True), ((1, 2, 3, 10), False)])
@pytest.mark.parametrize("inter", [False, True])
def test_append_with_positions(V, case, eight, sections, spread, inter):
    from speculative_decoding_rejection_decode_gb300 import rotary_axes, rotary_table
    kw = dict(APPEND[case])
    dt = kw.get("dtype", BF)
    s = Step(**kw, cache=E4 if eight else dt, seed=case, extra_rows=2)
    axes = rotary_axes(sections, spread=spread)
    table = rotary_table(700, 2 * len(axes))
    pos = torch.randint(0, 700, (len(sections), s.N), device="cuda", dtype=torch.int32)
    marker = torch.full_like(s.q, 7.0)
    q = s.cache(V).append(s.new_k, s.new_v, *args(s), s.parent, q=s.q, rotary=table, interleaved=inter, positions=pos,
                          axes=axes, out_q=marker)
    assert V.get_error() == 0
    n = s.n_rows
    assert torch.equal(q[n:], torch.full_like(q[n:], 7.0))
    assert torch.equal(q[:n], plain_turn(s.q, pos, axes, table, inter)[:n].to(dt))
    k32, v32 = plain_turn(s.new_k, pos, axes, table, inter), s.new_v.float()
    for b in range(s.B):
        slots = torch.arange(s.ctx[b], s.ctx[b] + s.nodes[b], device="cuda")
        pages = torch.tensor(s.pages[b], device="cuda")[slots // s.page] if s.nodes[b] else slots
        at = slice(s.firsts[b], s.firsts[b + 1])
        for got, sc, x in ((s.k, s.ks, k32), (s.v, s.vs, v32)):
            g = got[pages, :, slots % s.page]
            if not eight:
                assert torch.equal(g, x[at].to(dt))
                continue
            scale = x[at].abs().amax(-1).clamp(min=2.0 ** -40) * (1.0 / 448.0)
            assert torch.equal(sc[pages, :, slots % s.page], scale)
            assert torch.equal(g.view(torch.uint8), (x[at] / scale[..., None]).to(E4).view(torch.uint8))


@pytest.mark.parametrize("tree", ["chain", "random"])
@pytest.mark.parametrize("cache", [BF, E4])
def test_positions_and_offsets_that_say_what_slots_say(V, tree, cache):
    """On one axis, positions of length + depth are the plain append; offsets move it."""
    from speculative_decoding_rejection_decode_gb300 import rotary_table
    table = rotary_table(300, 128)

    def run(shift, **kw):
        s = Step(ctx=[9, 70, 0], nodes=[33, 20, 5], tree=tree, cache=cache, seed=5)
        if shift == "plain":
            given = {}
        else:
            depth = [len(ancestors(s.parents[b], j)) - 1 for b in range(s.B) for j in range(s.nodes[b])]
            req = [b for b in range(s.B) for _ in range(s.nodes[b])]
            where = [s.ctx[b] + d + shift[b] for b, d in zip(req, depth)]
            given = {"pos": dict(positions=torch.tensor(where, dtype=torch.int32, device="cuda")),
                     "off": dict(position_offsets=torch.tensor(shift, dtype=torch.int32, device="cuda"))}[kw["how"]]
        q = s.cache(V).append(s.new_k, s.new_v, *args(s), s.parent, q=s.q, rotary=table, **given)
        assert V.get_error() == 0
        return q, *s.cache(V).read(*args(s)[:2], s.cu, n_rows=s.n_rows)

    plain = run("plain")
    for how in ("pos", "off"):
        assert all(torch.equal(a, b) for a, b in zip(run([0, 0, 0], how=how), plain))
    moved = run([-9, 100, 7], how="pos")
    assert all(torch.equal(a, b) for a, b in zip(run([-9, 100, 7], how="off"), moved))
    assert not torch.equal(moved[0], plain[0]) and torch.equal(moved[2], plain[2])


@pytest.mark.parametrize("cache", [BF, E4])
def test_append_in_place_and_captured(V, cache):
    from speculative_decoding_rejection_decode_gb300 import rotary_axes, rotary_table
    table, axes = rotary_table(300, 128), rotary_axes((24, 20, 20))
    steps = [Step(ctx=[9, 70, 0], nodes=[33, 20, 5], cache=cache, seed=40 + i) for i in range(2)]
    pos = [torch.randint(0, 300, (3, s.N), generator=torch.Generator("cuda").manual_seed(i), device="cuda", dtype=torch.int32)
           for i, s in enumerate(steps)]
    run = lambda s, p, q, **kw: s.cache(V).append(s.new_k, s.new_v, *args(s), q=q, rotary=table, positions=p, axes=axes, **kw)
    want = []
    for s, p in zip(steps, pos):
        q = run(s, p, s.q)
        want.append((q, *s.cache(V).read(*args(s)[:2], s.cu, n_rows=s.n_rows)))
        own = s.q.clone()
        assert torch.equal(run(s, p, own, out_q=own), q) and torch.equal(own, q)
        s.k.zero_(), s.v.zero_()
    graphs = []
    for s, p in zip(steps, pos):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            q = run(s, p, s.q)
            out = (q, *s.cache(V).read(*args(s)[:2], s.cu, n_rows=s.n_rows))
        graphs.append((g, out, torch.cuda.Stream()))
    for _ in range(5):
        for g, _out, st in graphs:
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for (_g, out, _st), w in zip(graphs, want):
        assert all(torch.equal(a, b) for a, b in zip(out, w))
    assert V.get_error() == 0


@pytest.mark.parametrize("heads,D,rotary", [(1, 1024, 128), (1, 16, 16), (300, 16, 16), (2, 24, 16), (3, 136, 128)])
@pytest.mark.parametrize("inter", [False, True])
def test_rotate_few_and_many_pieces(V, heads, D, rotary, inter):
    from speculative_decoding_rejection_decode_gb300 import rotary_table
    g = torch.Generator("cuda").manual_seed(heads + D)
    x = torch.randn(700, heads, D, generator=g, device="cuda").to(BF)
    pos = torch.randint(0, 50, (700,), generator=g, device="cuda", dtype=torch.int32)
    table = rotary_table(50, rotary)
    want = plain_turn(x, pos[None], (0,) * (rotary // 2), table, inter).to(BF)
    assert torch.equal(V.rotate(x, pos, table, interleaved=inter), want)
    assert torch.equal(V.rotate(x, pos, table, interleaved=inter, out=x), want) and V.get_error() == 0
    # one row for many: a broadcast input
    wide = x[:1].expand(700, heads, D)
    want = plain_turn(wide, pos[None], (0,) * (rotary // 2), table, inter).to(BF)
    assert torch.equal(V.rotate(wide, pos, table, interleaved=inter), want) and V.get_error() == 0


def test_rows_with_bad_positions_are_left_out(V):
    from speculative_decoding_rejection_decode_gb300 import rotary_table
    table = rotary_table(100, 128)
    s = Step(ctx=[5, 9], nodes=[4, 3], seed=8)
    pos = torch.zeros(2, s.N, dtype=torch.int32, device="cuda")
    pos[0, 1], pos[1, 5] = 100, -5
    before = s.k.clone()
    q = s.cache(V).append(s.new_k, s.new_v, *args(s), q=s.q, rotary=table, positions=pos, axes=(0, 1) * 32)
    assert V.get_error() == BAD_CACHE
    for r, (b, j) in enumerate((b, j) for b in range(2) for j in range(s.nodes[b])):
        page, off = s.row(b, s.ctx[b] + j)
        left = r in (1, 5)
        assert torch.equal(s.k[page, :, off].nan_to_num(), (before[page, :, off] if left else s.new_k[r]).nan_to_num())
        assert (q[r] == 0).all() if left else torch.equal(q[r], s.q[r])
    # offsets that lead out of the table, on either side; the other request is written
    off = torch.tensor([-6, 90], dtype=torch.int32, device="cuda")
    q = s.cache(V).append(s.new_k, s.new_v, *args(s), q=s.q, rotary=table, position_offsets=off)
    assert V.get_error() == BAD_CACHE
    assert (q[0] == 0).all() and (q[1:5] != 0).any(-1).all() and (q[5:] == 0).all()
    # a tree is not read where positions are given
    parent = torch.full((s.N,), 99, dtype=torch.int32, device="cuda")
    s.cache(V).append(s.new_k, s.new_v, *args(s), parent, rotary=table, positions=pos[:1] * 0)
    assert V.get_error() == 0
    s.cache(V).append(s.new_k, s.new_v, *args(s), parent, rotary=table, position_offsets=off * 0)
    assert V.get_error() == BAD_TREE


def test_extreme_rows_quantise_as_a_division_does(V):
    # infinite, NaN, huge and tiny values: the bytes and scales of elementary torch operations
    s = Step(ctx=[0], nodes=[40], cache=E4, seed=31, poison=False)
    x = s.new_v
    x[0, 0, 3], x[1, 0, 3], x[2, 1, 100] = math.inf, -math.inf, math.nan
    x[3] = 3.38e38
    x[4] *= 1e37
    x[5] *= 1e33                          # scales around the largest that a reciprocal serves
    x[6] *= 1e32
    x[7] *= 1e-38
    x[8] = 0
    x[9] *= 1e-30
    x[10, :, 1:] *= 1e-36
    x[11, 0, 0], x[11, 0, 1:] = 3e38, -1e-38
    s.cache(V).append(s.new_k, s.new_v, *args(s))
    f = x.float()
    scale = f.abs().amax(-1).clamp(min=2.0 ** -40) * (1.0 / 448.0)
    want = (f / scale[..., None]).to(E4).view(torch.uint8)
    for j in range(40):
        page, off = s.row(0, j)
        got = s.v.view(torch.uint8)[page, :, off]
        nan = (want[j] & 0x7F) == 0x7F
        assert torch.equal(got[~nan], want[j][~nan]) and ((got[nan] & 0x7F) == 0x7F).all(), j
        a, b = s.vs[page, :, off], scale[j]
        assert torch.equal(a.nan_to_num(-1.0), b.nan_to_num(-1.0))
    assert V.get_error() == 0


def test_quotients_beside_the_borders(V):
    # rows whose largest value is any 16-bit one, and beside it values next to every border
    # between two bytes: what is stored is what the division gives
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    mids = torch.cat([(1 + (2 * torch.arange(8) + 1) / 16) * 2.0 ** e for e in (-6, -3, 0, 5, 8)] + [(2 * torch.arange(8) + 1) * 2.0 ** -10]).cuda()
    for dtype in (BF, HF):
        top = torch.arange(1 << 10, device="cuda") / (1 << 10) + 1          # every mantissa of either type
        s = Step(ctx=[0], nodes=[1 << 10], kv_heads=1, cache=E4, dtype=dtype, seed=32, poison=False)
        scale = top.to(dtype).float() * (1.0 / 448.0)
        x = (mids[None, :48] * scale[:, None] * (1 + (torch.rand(1 << 10, 48, generator=g, device="cuda") - 0.5) * 2.0 ** -7)).to(dtype)
        x = torch.cat([top.to(dtype)[:, None], x, -x, torch.zeros(1 << 10, 31, dtype=dtype, device="cuda")], 1)[:, None]
        x = torch.minimum(torch.maximum(x, -top.to(dtype)[:, None, None]), top.to(dtype)[:, None, None])
        s.cache(V).append(x, x, *args(s))
        f = x.float()
        sc = f.abs().amax(-1).clamp(min=2.0 ** -40) * (1.0 / 448.0)
        want = (f / sc[..., None]).to(E4).view(torch.uint8)
        slots = torch.arange(1 << 10, device="cuda")
        pages = torch.tensor(s.pages[0], device="cuda")[slots // s.page]
        assert torch.equal(s.k.view(torch.uint8)[pages, :, slots % s.page], want)
