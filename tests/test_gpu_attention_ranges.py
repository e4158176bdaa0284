"""Attention at the ends of its types on the GPU: weights at the lag of their reference, values
near the largest and smallest that bf16 holds, queries and keys that are no numbers."""
import math

import pytest
import torch

from cache_reference import Step, attend_tolerance

pytestmark = pytest.mark.gpu

BF, HF, E4 = torch.bfloat16, torch.float16, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def V():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_rejection_decode_gb300 import Verifier
    v = Verifier(0)
    yield v
    v.close()


# rows of a request and heads that the three kernels serve: few, more, many for every SM
KERNELS = [(2, {}), (40, {}), (300, {}), (300, dict(kv_heads=32, group=2))]


def attend(V, s, cross, **kw):
    c = s.cache(V)
    if cross:
        return c.cross_attend(s.q, s.table, s.lengths, s.cu, **kw)
    return c.attend(s.q, s.table, s.lengths, s.cu, s.parent, **kw)


def reference(s, cross, scale=None):
    """float64 [n_rows, heads, head_dim] and, per row, the largest |v| seen; chains of nodes."""
    scale = s.head_dim ** -0.5 if scale is None else scale
    K, W = s.values("k"), s.values("v")
    out, big = [], []
    for b in range(s.B):
        n = s.nodes[b]
        slots = torch.arange(s.ctx[b] + (0 if cross else n), device=K.device)
        pages = torch.tensor(s.pages[b], device=K.device)[slots // s.page]
        k, v = K[pages, :, slots % s.page], W[pages, :, slots % s.page]
        q = s.q[s.firsts[b]:s.firsts[b + 1]].double().view(n, s.kv_heads, s.group, s.head_dim)
        z = torch.einsum("nhgd,shd->nhgs", q, k) * scale
        later = slots[None] > s.ctx[b] + torch.arange(n, device=K.device)[:, None]
        w = z.masked_fill(later[:, None, None], -math.inf).softmax(-1)
        out.append(torch.einsum("nhgs,shd->nhgd", w, v).reshape(n, s.heads, s.head_dim))
        most = v.abs().amax(2).cummax(0).values                       # [slots, kv_heads], seen up to a slot
        seen = torch.full((n,), s.ctx[b] - 1, device=K.device) if cross else torch.arange(n, device=K.device) + s.ctx[b]
        big.append(most[seen].repeat_interleave(s.group, 1))
    return torch.cat(out), torch.cat(big)


def one_higher(s, lag, slot):
    """Every score 0 but those of `slot`, which are `lag` (times log 2, in base e) for the scale log 2."""
    s.q.zero_()
    s.q[..., 0] = 1.0
    if s.ks is None:
        s.k.zero_()
    else:
        s.k.view(torch.uint8).zero_()
        s.ks.fill_(1.0)
    for b in range(s.B):
        page, off = s.row(b, slot)
        if s.ks is None:
            s.k[page, :, off, 0] = lag
        else:
            s.k[page, :, off, 0] = torch.tensor(8.0).to(E4)
            s.ks[page, :, off] = lag / 8.0


@pytest.mark.parametrize("cross", [False, True])
@pytest.mark.parametrize("dtype,cache", [(HF, E4), (BF, E4), (HF, HF)])
@pytest.mark.parametrize("rows,heads", KERNELS)
def test_a_maximum_that_rises_by_the_lag(V, cross, dtype, cache, rows, heads):
    # A reference may lag behind the maximum: weights just below, at and behind every lag that a
    # kernel may leave, on a value whose scale has the largest mantissa.
    s = Step(ctx=[200], nodes=[rows], dtype=dtype, cache=cache, seed=1, poison=False, **heads)
    if s.vs is not None:
        s.vs.fill_(2.0 - 2.0 ** -20)
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    v = torch.rand(s.v.shape, generator=g, device="cuda") * 2 - 1      # up to the head room of the sums
    s.v.copy_(v.to(s.v.dtype))
    for lag in (7.9995, 8.0, 8.9995, 8.99999, 9.0, 9.0005, 9.9995, 15.9995):
        one_higher(s, lag, 40)
        out = attend(V, s, cross, scale=math.log(2.0))
        assert V.get_error() == 0 and out.isfinite().all(), lag
        want, big = reference(s, cross, math.log(2.0))
        # scores up to 16 are off by less than 2^-18 (products of 32-bit factors), well within the tolerance
        assert ((out.double() - want).abs() <= attend_tolerance(s, want, big)).all(), lag


def some_hidden(s):
    """A mask with hidden slots among every 32."""
    return (torch.arange(max(s.ctx), device="cuda") % 5 != 2).repeat(s.B, 1)


@pytest.mark.parametrize("cross", [None, False, True])                # context and nodes; states; states with a mask
@pytest.mark.parametrize("dtype,cache", [(BF, BF), (HF, HF), (BF, E4), (HF, E4)])
@pytest.mark.parametrize("ctx", [20, 60, 3000])                       # items whole, and split over ranges
@pytest.mark.parametrize("rows,heads", KERNELS)
def test_a_query_that_is_no_number(V, cross, dtype, cache, ctx, rows, heads):
    s = Step(ctx=[ctx, ctx], nodes=[rows, rows], dtype=dtype, cache=cache, seed=5, poison=False, **heads)
    kw = dict(mask=some_hidden(s)) if cross else {}
    clean = attend(V, s, cross is not None, **kw)
    s.q[1, 1, 3] = math.nan
    out = attend(V, s, cross is not None, **kw)
    assert V.get_error() == 0
    assert out[1, 1].isnan().all()
    out[1, 1] = clean[1, 1]
    assert torch.equal(out, clean)


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("dtype,cache", [(BF, BF), (HF, HF), (BF, E4), (HF, E4)])
@pytest.mark.parametrize("ctx", [20, 60, 3000])
@pytest.mark.parametrize("rows,heads", KERNELS)
def test_keys_that_are_no_numbers(V, masked, dtype, cache, ctx, rows, heads):
    s = Step(ctx=[ctx, ctx], nodes=[rows, rows], dtype=dtype, cache=cache, seed=6, poison=False, **heads)
    kw = dict(mask=some_hidden(s)) if masked else {}
    clean = attend(V, s, True, **kw)
    for slot in range(ctx):                                           # every key of request 1, kv head 0
        page, off = s.row(1, slot)
        if s.ks is None:
            s.k[page, 0, off] = math.nan
        else:
            s.ks[page, 0, off] = math.nan
    out = attend(V, s, True, **kw)
    assert V.get_error() == 0
    assert out[rows:2 * rows, :s.group].isnan().all()
    out[rows:2 * rows, :s.group] = clean[rows:2 * rows, :s.group]
    assert torch.equal(out, clean)


@pytest.mark.parametrize("cross", [False, True])
@pytest.mark.parametrize("rows,heads", KERNELS)
@pytest.mark.parametrize("power", [-118, -100, -60, 60, 100, 119])
def test_values_of_any_size(V, cross, rows, heads, power):
    # 200 to 500 weights of at most 1 (the kernel's largest) and values below 2^119: sums below 2^128
    s = Step(ctx=[200], nodes=[rows], seed=3, poison=False, **heads)
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    s.v.copy_(torch.rand(s.v.shape, generator=g, device="cuda") * 2 - 1)
    unit = s.v.clone()
    for lag in (0.0, 7.96875, 15.9375):                              # what bf16 holds of 8 and 16
        one_higher(s, lag, 40)
        s.v.copy_(unit)
        want, big = reference(s, cross, math.log(2.0))
        s.v.mul_(2.0 ** power)                                        # exact
        out = attend(V, s, cross, scale=math.log(2.0))
        assert V.get_error() == 0 and out.isfinite().all(), lag
        got = out.double() * 2.0 ** -power
        assert ((got - want).abs() <= attend_tolerance(s, want, big)).all(), lag


@pytest.mark.parametrize("rows,heads", KERNELS)
@pytest.mark.parametrize("cache", [BF, E4])
@pytest.mark.parametrize("page", [12, 8, 16, 32, 64])                 # copies of 16 bytes, boxes of 8 to 64 rows
def test_masked_slots_of_pages_that_are_not_held(V, rows, heads, cache, page):
    # what a masked slot holds concerns no row, not even whether there is a page for it
    s = Step(ctx=[200, 330], nodes=[rows, rows], cache=cache, page=page, seed=7, poison=False, **heads)
    mask = torch.ones(2, 330, dtype=torch.bool, device="cuda")
    mask[0, 128:] = False                                             # padding
    mask[1, 2 * page:3 * page] = False                                # a page in the middle
    mask[1, 256:256 + page // 2] = False                              # and half of one
    want = attend(V, s, True, mask=mask)
    assert V.get_error() == 0
    table = s.table.clone()
    table[0, -(-128 // page):] = -1
    table[1, 2] = -2
    s.table = table
    assert torch.equal(attend(V, s, True, mask=mask), want)
    assert V.get_error() == 0
    # one slot of it shown: the page is missed
    mask[1, 3 * page - 1] = True
    assert torch.equal(attend(V, s, True, mask=mask), want)
    assert V.get_error() == 32


@pytest.mark.parametrize("cross", [False, True])
@pytest.mark.parametrize("dtype,cache", [(BF, BF), (HF, HF), (BF, E4)])
@pytest.mark.parametrize("rows", [1, 3, 4, 29])
@pytest.mark.parametrize("head_dim", [64, 128])
def test_one_request_over_many_ranges(V, cross, dtype, cache, rows, head_dim):
    # 2 to 152 partial results of every row
    for kv_heads, ctx in ((8, 600), (8, 1500), (8, 1999), (1, 1999), (3, 5000), (2, 20000)):
        s = Step(ctx=[ctx], nodes=[rows], kv_heads=kv_heads, group=4, head_dim=head_dim, dtype=dtype, cache=cache, page=64, seed=8, poison=False)
        out = attend(V, s, cross)
        assert V.get_error() == 0
        want, big = reference(s, cross)
        # (attend_tolerance: sums of up to 2^11 keys add 2^-13 of the largest value; of 2^15, 2^-9)
        assert ((out.double() - want).abs() <= attend_tolerance(s, want, big) + (2.0 ** -9 * big[..., None] if ctx > 2000 else 0.0)).all()


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("width", [8192, 8193, 20000])                # slots that the table holds
def test_ranges_of_short_and_long_tables(V, dtype, width):
    # ragged requests over e4m3: the ranges of work are cut by the table's width, the result is not
    s = Step(ctx=[0, 700, 2000, 3, 1300, 129] * 6, nodes=[9, 5, 9, 29, 6, 40] * 6, kv_heads=2, dtype=dtype, cache=E4, seed=10, page=64, poison=False)
    pad = torch.full((s.B, -(-width // 64) - s.table.shape[1]), -1, dtype=torch.int32, device="cuda")
    s.table = torch.cat([s.table, pad], 1)
    out = attend(V, s, False)
    assert V.get_error() == 0
    want, big = reference(s, False)
    assert ((out.double() - want).abs() <= attend_tolerance(s, want, big)).all()


@pytest.mark.parametrize("cross", [False, True])
@pytest.mark.parametrize("dtype,cache", [(BF, BF), (HF, HF), (BF, E4), (HF, E4)])
@pytest.mark.parametrize("rows,heads", KERNELS)
@pytest.mark.parametrize("rising", [False, True])
def test_references_that_move_often(V, cross, dtype, cache, rows, heads, rising):
    # scores tens of units of log 2 apart, in no order or rising along the keys: every lag is passed,
    # in every part of a tile, while the next scores are under way
    s = Step(ctx=[700], nodes=[rows], dtype=dtype, cache=cache, seed=11, poison=False, **heads)
    s.q.mul_(8.0)
    if rising:
        s.q[..., :4] = s.q[..., :4].abs() + 4
        for slot in range(s.ctx[0] + rows):
            page, off = s.row(0, slot)
            up = torch.tensor(0.008 * slot).to(dtype).float()
            if s.ks is None:
                s.k[page, :, off, :4] = up
            else:
                s.k[page, :, off, :4] = (up / s.ks[page, :, off])[:, None].clamp(max=448).to(E4)
    out = attend(V, s, cross)
    assert V.get_error() == 0
    want, big = reference(s, cross)
    # attend_tolerance with the scores' error of these inputs: float32 sums of D products, D 2^-24 of
    # the sum of their magnitudes (twice that for a pair of weights), and over e4m3 keys in tiles the
    # queries' parts, 2^-17 of a row's largest value
    K = s.values("k").abs()
    pages = torch.tensor(s.pages[0], device=K.device)[torch.arange(s.ctx[0] + rows, device=K.device) // s.page]
    k = K[pages, :, torch.arange(s.ctx[0] + rows, device=K.device) % s.page]
    q = s.q[:s.n_rows].double().abs().view(-1, s.kv_heads, s.group, s.head_dim)
    size = torch.einsum("nhgd,shd->nhgs", q, k).amax(-1)
    d = s.head_dim * 2.0 ** -24 * size
    if s.ks is not None:
        d = d + 2.0 ** -17 * q.amax(-1) * k.sum(-1).amax(0)[None, :, None]
    d = (d * s.head_dim ** -0.5).view(-1, s.heads, 1)
    assert ((out.double() - want).abs() <= attend_tolerance(s, want, big) + 2 * d * big[..., None]).all()
