"""Cross attention to an encoder's states on the GPU, against plain 64-bit attention."""
import math

import pytest
import torch

from cache_reference import Step, attend_tolerance

pytestmark = pytest.mark.gpu

BF, HF, E4 = torch.bfloat16, torch.float16, torch.float8_e4m3fn
BAD_CU, BAD_CACHE = 2, 32


@pytest.fixture(scope="module")
def V():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_rejection_decode_gb300 import Verifier
    v = Verifier(0)
    yield v
    v.close()


def hide_the_rest(s):
    """NaN behind every request's states."""
    full, s.nodes = s.nodes, [0] * s.B
    s.poison_unused()
    s.nodes = full


def make(ctx, rows, mask=None, **kw):
    s = Step(ctx=ctx, nodes=rows, poison=False, **kw)
    hide_the_rest(s)
    s.mask = None
    if mask is not None:
        g = torch.Generator(device="cuda")
        g.manual_seed(7)
        s.mask = torch.rand(s.B, max(max(ctx), 1), generator=g, device="cuda") >= mask
        # what a masked slot holds reaches no row
        for b in range(s.B):
            for slot in (~s.mask[b]).nonzero()[:, 0].tolist()[:8]:
                if slot < ctx[b]:
                    page, off = s.row(b, slot)
                    if s.ks is None:
                        s.k[page, :, off], s.v[page, :, off] = math.nan, math.inf
                    else:
                        s.k.view(torch.uint8)[page, :, off] = 0x7F
                        s.vs[page, :, off] = math.inf
    return s


def reference(s, scale=None):
    """float64 [n_rows, heads, head_dim] and, per row, the largest |v| seen."""
    scale = s.head_dim ** -0.5 if scale is None else scale
    K, W = s.values("k"), s.values("v")
    out = torch.zeros(s.n_rows, s.heads, s.head_dim, dtype=torch.float64, device=K.device)
    big = torch.zeros(s.n_rows, s.heads, dtype=torch.float64, device=K.device)
    for b in range(s.B):
        slots = torch.arange(s.ctx[b], device=K.device)
        if s.mask is not None:
            slots = slots[s.mask[b, :s.ctx[b]].bool()]
        if not slots.numel() or not s.nodes[b]:
            continue
        pages = torch.tensor(s.pages[b], device=K.device)[slots // s.page]
        k, v = K[pages, :, slots % s.page], W[pages, :, slots % s.page]
        at = slice(s.firsts[b], s.firsts[b + 1])
        q = s.q[at].double().view(-1, s.kv_heads, s.group, s.head_dim)
        w = (torch.einsum("nhgd,shd->nhgs", q, k) * scale).softmax(-1)
        out[at] = torch.einsum("nhgs,shd->nhgd", w, v).reshape(-1, s.heads, s.head_dim)
        big[at] = v.abs().amax((0, 2)).repeat_interleave(s.group)
    return out, big


def check(V, s, scale=None):
    out = torch.full((s.N, s.heads, s.head_dim), 7.0, dtype=s.dtype, device="cuda")
    s.cache(V).cross_attend(s.q, s.table, s.lengths, s.cu, mask=s.mask, scale=scale, out=out)
    assert V.get_error() == 0
    assert (out[s.n_rows:] == 7.0).all()                # rows behind the last request
    want, big = reference(s, scale)
    got = out[:s.n_rows].double()
    tol = attend_tolerance(s, want, big)
    assert ((got - want).abs() <= tol).all(), float(((got - want).abs() - tol).max())
    for b in range(s.B):                                # nothing to see: zeros
        if s.ctx[b] == 0 or (s.mask is not None and not s.mask[b, :s.ctx[b]].any()):
            assert (out[s.firsts[b]:s.firsts[b + 1]] == 0).all()
    return out


CASES = [
    dict(ctx=[1], rows=[1]),
    dict(ctx=[500], rows=[1], kv_heads=16, group=1, head_dim=64),
    dict(ctx=[0, 1, 17, 0, 300], rows=[3, 2, 0, 1, 9], page=16),
    dict(ctx=[0], rows=[5]),
    dict(ctx=[129, 128, 127, 4, 0], rows=[40, 1, 64, 129, 130], page=64, group=2),
    dict(ctx=[700, 30, 2000], rows=[29, 29, 29], page=48, kv_heads=3, group=7),
    dict(ctx=[1000, 513], rows=[300, 257], page=128, kv_heads=2, group=1),
    dict(ctx=[65, 1300, 5], rows=[700, 100, 513], page=100, kv_heads=1, group=4),
    dict(ctx=[3, 900], rows=[1, 260], page=8, kv_heads=1, group=1),
    dict(ctx=[2500], rows=[513], page=64, kv_heads=2, group=4),
    dict(ctx=[60, 0, 61] * 50, rows=[1, 2, 1] * 50, page=16, kv_heads=1, group=4),
    # many rows for every SM
    dict(ctx=[1000, 513], rows=[300, 257], page=128, kv_heads=40, group=1),
    dict(ctx=[65, 1300, 5], rows=[700, 100, 513], page=104, kv_heads=8, group=4),
    dict(ctx=[3, 900, 0, 64], rows=[1, 260, 300, 129], page=8, kv_heads=40, group=1),
    dict(ctx=[2500], rows=[513], page=64, kv_heads=10, group=7),
    dict(ctx=[60, 0, 61] * 20, rows=[130, 200, 140] * 20, page=16, kv_heads=2, group=1),
]
MANY = dict(kv_heads=32, group=2)     # heads that give every SM some tiles of rows


@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("dtype,cache", [(BF, BF), (HF, HF), (BF, E4), (HF, E4)])
@pytest.mark.parametrize("head_dim", [64, 128])
@pytest.mark.parametrize("mask", [None, 0.3, 0.97])
def test_cross(V, case, dtype, cache, head_dim, mask):
    kw = {**CASES[case], "head_dim": head_dim}
    s = make(kw.pop("ctx"), kw.pop("rows"), mask, dtype=dtype, cache=cache, seed=case, extra_rows=2, **kw)
    check(V, s)


@pytest.mark.parametrize("rows,heads", [(2, {}), (40, {}), (600, {}), (200, MANY)])
def test_rows_that_see_nothing(V, rows, heads):
    for cache in (BF, E4):
        s = make([300, 200, 300, 100], [rows] * 4, 0.0, cache=cache, seed=3, **heads)
        s.mask[0] = False                  # none at all
        s.mask[1, :128] = False            # whole tiles, in front
        s.mask[2, 128:] = False            # and behind
        check(V, s)
        # slots behind the mask's columns are hidden as well
        s.mask = s.mask[:, :150].contiguous()
        out = s.cache(V).cross_attend(s.q, s.table, s.lengths, s.cu, mask=s.mask)
        s.ctx = [min(c, 150) for c in s.ctx]
        want, big = reference(s)
        assert ((out.double() - want).abs() <= attend_tolerance(s, want, big)).all() and V.get_error() == 0
        none = torch.zeros(4, 0, dtype=torch.bool, device="cuda")
        assert (s.cache(V).cross_attend(s.q, s.table, s.lengths, s.cu, mask=none) == 0).all()


@pytest.mark.parametrize("rows,heads", [(3, {}), (300, {}), (300, MANY)])
def test_masks_of_either_type_and_any_stride(V, rows, heads):
    s = make([300, 77], [rows, rows], 0.4, seed=4, **heads)
    want = check(V, s)[:s.n_rows]
    wide = torch.zeros(2, 500, dtype=torch.uint8, device="cuda")
    wide[:, 3:303] = s.mask * 255
    got = s.cache(V).cross_attend(s.q, s.table, s.lengths, s.cu, mask=wide[:, 3:303])
    assert torch.equal(got, want)


@pytest.mark.parametrize("rows,heads", [(2, {}), (30, {}), (520, {}), (260, MANY)])
@pytest.mark.parametrize("scale", [1.0, 0.05, 0.0, -0.1])
def test_scales_and_strides(V, rows, heads, scale):
    s = make([400, 90], [rows, rows + 1], **{**dict(kv_heads=2, group=4, seed=5), **heads})
    if scale == 1.0:
        s.q = s.q * 0.25
    wide = torch.randn(s.N, s.heads + 3, 128, device="cuda").to(BF)
    wide[:, 2:2 + s.heads] = s.q
    s.q = wide[:, 2:2 + s.heads]
    out = check(V, s, scale)
    for _ in range(3):
        assert torch.equal(out, s.cache(V).cross_attend(s.q, s.table, s.lengths, s.cu, scale=scale))


@pytest.mark.parametrize("rows,H,most", [(2, 4, 333), (600, 4, 333), (600, 32, 336)])
def test_a_padded_batch_of_states_is_a_cache(V, rows, H, most):
    from speculative_decoding_rejection_decode_gb300 import KVCache
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    B, D = 3, 64
    k, v = (torch.randn(B, H, most, D, generator=g, device="cuda").to(BF) for _ in range(2))
    q = torch.randn(B * rows, H, D, generator=g, device="cuda").to(BF)
    lengths = torch.tensor([333, 1, 200], dtype=torch.int32, device="cuda")
    cu = torch.arange(B + 1, dtype=torch.int32, device="cuda") * rows
    table = torch.arange(B, dtype=torch.int32, device="cuda")[:, None]
    out = KVCache(V, k, v).cross_attend(q, table, lengths, cu)
    assert V.get_error() == 0
    for b in range(B):
        n = int(lengths[b])
        qq = q[b * rows:(b + 1) * rows].double()
        w = (torch.einsum("nhd,hsd->nhs", qq, k[b, :, :n].double()) / 8).softmax(-1)
        want = torch.einsum("nhs,hsd->nhd", w, v[b, :, :n].double())
        # weights and the result rounded to bf16, scores and sums in 32 bits
        tol = (2.0 ** -8 + 5e-4) * v[b, :, :n].double().abs().amax() + 2.0 ** -8 * want.abs()
        assert ((out[b * rows:(b + 1) * rows].double() - want).abs() <= tol).all()


@pytest.mark.parametrize("rows,heads", [(3, {}), (40, {}), (700, {}), (250, MANY)])
def test_bad_pages_and_lengths(V, rows, heads):
    s = make([200, 100, 300], [rows] * 3, page=32, seed=6, **heads)
    c = s.cache(V)
    good = c.cross_attend(s.q, s.table, s.lengths, s.cu)
    table = s.table.clone()
    table[1, 1] = s.num_pages              # slots 32 .. 63 of request 1 are not held
    got = c.cross_attend(s.q, table, s.lengths, s.cu)
    assert V.get_error() == BAD_CACHE
    assert torch.equal(got[:rows], good[:rows]) and torch.equal(got[2 * rows:], good[2 * rows:])
    s.mask = torch.ones(3, 300, dtype=torch.bool, device="cuda")
    s.mask[1, 32:64] = False
    want, big = reference(s)
    assert ((got.double() - want).abs() <= attend_tolerance(s, want, big)).all()
    # lengths outside the table, a malformed cu: nothing of those requests is written.  The
    # others' keys may be split in other places then, whose partial sums are added in
    # another order in 32 bits (2^-13 of attend_tolerance): the formula is the measure
    s.mask = None
    want, big = reference(s)
    near = lambda x, at: ((x[at].double() - want[at]).abs() <= attend_tolerance(s, want, big)[at]).all()
    out = torch.full_like(good, 7.0)
    lengths = s.lengths.clone()
    lengths[0], lengths[2] = -1, s.table.shape[1] * 32 + 1
    c.cross_attend(s.q, s.table, lengths, s.cu, out=out)
    assert V.get_error() == BAD_CACHE
    assert (out[:rows] == 7).all() and (out[2 * rows:] == 7).all() and near(out, slice(rows, 2 * rows))
    cu = s.cu.clone()
    cu[3] = s.N + 1
    out.fill_(7.0)
    c.cross_attend(s.q, s.table, s.lengths, cu, out=out)
    assert V.get_error() == BAD_CU
    assert near(out, slice(0, 2 * rows)) and (out[2 * rows:] == 7).all()


@pytest.mark.parametrize("nodes,kv", [(3, 2), (300, 2), (300, 50)])
def test_infinite_values_reach_the_rows_that_see_them(V, nodes, kv):
    s = make([400], [nodes], kv_heads=kv, group=2, seed=9)
    clean = s.cache(V).cross_attend(s.q, s.table, s.lengths, s.cu)
    page, off = s.row(0, 130)
    s.v[page, 1, off, 5] = math.inf
    out = s.cache(V).cross_attend(s.q, s.table, s.lengths, s.cu)
    assert not out[:, 2:4, 5].isfinite().any()
    out[:, 2:4, 5] = clean[:, 2:4, 5]
    assert torch.equal(out, clean)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("rows,heads", [(1, {}), (20, {}), (300, {}), (300, MANY)])
def test_a_row_that_sees_one_state_is_its_values(V, dtype, rows, heads):
    # a weight of one, whatever the score
    s = make([1, 40, 200], [rows] * 3, 0.0, dtype=dtype, cache=dtype, seed=13, **heads)
    for b, slot in enumerate((0, 39, 130)):
        s.mask[b] = False
        s.mask[b, slot] = True
    out = s.cache(V).cross_attend(s.q, s.table, s.lengths, s.cu, mask=s.mask)
    assert V.get_error() == 0
    for b, slot in enumerate((0, 39, 130)):
        page, off = s.row(b, slot)
        want = s.v[page, :, off].repeat_interleave(s.group, 0)
        assert (out[b * rows:(b + 1) * rows] == want).all()


def test_one_large_request_among_small_ones(V):
    s = make([3000, 50, 50, 50, 50], [900, 1, 1, 1, 1], kv_heads=2, group=1, seed=10)
    check(V, s)
    s = make([50] * 40 + [3000], [1] * 40 + [200], kv_heads=2, group=1, seed=11)
    check(V, s)
    s = make([50] * 4 + [3000], [1] * 4 + [900], kv_heads=40, group=1, seed=12)
    check(V, s)


def test_two_graphs_on_two_streams(V):
    steps = [make([2000, 0, 30], [6, 29, 600 * k], 0.2, kv_heads=h, seed=k, cache=c) for k, c, h in ((1, BF, 4), (0, E4, 4), (1, BF, 24))]
    run = lambda s: s.cache(V).cross_attend(s.q, s.table, s.lengths, s.cu, mask=s.mask)
    eager = [run(s) for s in steps]
    torch.cuda.synchronize()
    graphs = []
    for s in steps:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = run(s)
        graphs.append((g, out))
    streams = [torch.cuda.Stream() for _ in steps]
    for _ in range(10):
        for (g, _o), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for (_g, out), want in zip(graphs, eager):
        assert torch.equal(out, want)
    assert V.get_error() == 0


# ---- a step of a target that has an encoder and reads images, whole --------------------

@pytest.mark.parametrize("cache", [BF, E4])
def test_a_step_with_everything(V, cache):
    """Prompt with image positions and its states, then two verified steps of a token
    tree: append, attention, cross attention, logits, verification, log probabilities
    of what was emitted, commit.  Each step equals plain formulas over the same rows."""
    from speculative_decoding_rejection_decode_gb300 import KVCache, rotary_axes, rotary_table, tree_rows
    g = torch.Generator(device="cuda")
    g.manual_seed(20)
    kv, group, D, page, vocab, B = 2, 2, 64, 16, 500, 2
    heads = kv * group
    r = lambda *n: torch.randn(*n, generator=g, device="cuda").to(BF)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    own, states = (KVCache.empty(V, 40, page, kv, D, cache) for _ in range(2))
    table, etable = i32([[5, 9, 1, 30], [2, 8, 7, 6]]), i32([[0, 1, 2, 3, 4], [5, 6, 7, 8, 9]])
    rotary, axes = rotary_table(100, D), rotary_axes((12, 10, 10), spread=True)
    elen, zero = i32([70, 33]), i32([0, 0])
    states.append(r(103, kv, D), r(103, kv, D), etable, zero, i32([0, 70, 103]))
    ek, ev = (x.double() for x in states.read(etable, zero, i32([0, 70, 103]), n_rows=103))
    # prompts: 2 words, an image of 3 x 4, 1 word; 5 words
    image = [(0,) * 3, (1,) * 3] + [(2, 2 + y, 2 + x) for y in range(3) for x in range(4)] + [(6,) * 3]
    pos = i32(image + [(i,) * 3 for i in range(5)]).T.contiguous()
    cu0 = i32([0, 15, 20])
    own.append(r(20, kv, D), r(20, kv, D), table, zero, cu0, rotary=rotary, positions=pos, axes=axes)
    lengths, offsets = i32([15, 5]), i32([7 - 15, 0])
    head = torch.randn(heads * D, vocab, generator=g, device="cuda")
    parent, n = i32([-1, 0, 0, 1, 2, 2] * B), 6
    cu = i32([0, n, 2 * n])
    for step in range(2):
        new_k, new_v, q0 = r(B * n, kv, D), r(B * n, kv, D), r(B * n, heads, D)
        q = own.append(new_k, new_v, table, lengths, cu, parent, q=q0, rotary=rotary, position_offsets=offsets)
        a = own.attend(q, table, lengths, cu, parent)
        c = states.cross_attend(a, etable, elen, cu)
        assert V.get_error() == 0
        for b, (e0, e1) in enumerate(((0, 70), (70, 103))):
            w = torch.einsum("nhgd,shd->nhgs", a[b * n:(b + 1) * n].double().view(n, kv, group, D), ek[e0:e1]) / 8
            want = torch.einsum("nhgs,shd->nhgd", w.softmax(-1), ev[e0:e1]).reshape(n, heads, D)
            big = ev[e0:e1].abs().amax()
            # weights (and 8-bit values' factors) and the result rounded; read() rounds 8-bit rows once
            assert ((c[b * n:(b + 1) * n].double() - want).abs() <= 2.0 ** -6 * big).all()
        logits = (c.float().flatten(1) @ head) * 0.5
        draft = (logits + torch.randn(logits.shape, generator=g, device="cuda")).softmax(1).contiguous()
        up = torch.where(parent < 0, 0, parent) + torch.arange(B, device="cuda").repeat_interleave(n).int() * n
        tokens = torch.multinomial(draft[up.long()], 1, generator=g)[:, 0].to(torch.int32)
        out = V.tree(logits, draft, tokens, parent, cu, T=1.0, seed=step)
        rows = tree_rows(out.path, cu)
        lp = V.logprobs(logits, out.tokens, rows=rows, top=3)
        assert V.get_error() == 0
        acc = out.num_accepted.tolist()
        for b in range(B):
            at = 0
            for d in range(acc[b] + 1):
                want = torch.log_softmax(logits[b * n + at].double(), 0)
                slot = b * n + d
                assert rows[slot] == b * n + at
                assert abs(float(lp.logprob[slot]) - float(want[int(out.tokens[slot])])) <= 1e-5 * (1 + abs(float(want.min())))
                assert lp.top_ids[slot].tolist() == logits[b * n + at].topk(3).indices.tolist()
                at = int(out.path[slot]) if d < acc[b] else at
            assert (rows[b * n + acc[b] + 1:(b + 1) * n] == -1).all()
        before = lengths.tolist()
        lengths = own.commit(table, lengths, cu, out.num_accepted, out.path)
        assert lengths.tolist() == [x + 1 + y for x, y in zip(before, acc)] and V.get_error() == 0
