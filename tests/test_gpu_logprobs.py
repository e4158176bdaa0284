"""Log probabilities of given tokens, entropy, top alternatives and the gradient of
the logits on the GPU, against 64-bit formulas."""
import math

import pytest
import torch

from cache_reference import HALF_STEP

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
BAD_ID, BAD_CU = 1, 2


@pytest.fixture(scope="module")
def V():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_rejection_decode_gb300 import Verifier
    v = Verifier(0)
    yield v
    v.close()


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Want:
    """The 64-bit values of rows x (any type) at temperature T, and error bounds.

    A term 2^y of the sum S has the exponential's error (2^-22) and that of y, half
    steps of |y| from the difference and the product; y comes with the rounded factor
    log2(e) / T (2^-23 relative, an error of the temperature itself: it moves ln p by at
    most 2^-23 times the distance in x / T from the mean, and so do the half steps).  A thread adds at most
    V / 2048 + 24 terms to one of its sums and the sums are joined in about 20 steps
    (each with an exponential of its own, exact powers or another 2^-22), each
    addition half a step: relative errors of S and of the sum of |2^y y| within
      e = 2^-20 + (V / 2048 + 64) 2^-24.
    ln p takes e, and half steps of its terms; H = ln S - W / S takes e once from the
    logarithm and twice from the quotient times the mean distance."""

    def __init__(self, x, T):
        x = x.double()
        V = x.shape[1]
        self.y = x / T
        self.lp = torch.log_softmax(self.y, 1)
        self.p = self.lp.exp()
        self.H = torch.special.entr(self.p).sum(1)
        self.e = 2.0 ** -20 + (V / 2048 + 64) * 2.0 ** -24
        top = self.y.amax(1, keepdim=True)
        dist = torch.where(self.p > 0, top - self.y, 0.0)
        self.mean = (self.p * dist).sum(1)                       # mean distance from the largest
        self.lnS = math.log(V) + 8 * math.log(2)                 # a reference within 2^8 of the largest
        self.range = self.lp.abs().where(self.lp.isfinite(), 0.0) + self.mean[:, None] + self.lnS

    def lp_bound(self, lp):
        return self.e + 2.0 ** -21 * (lp.abs() + self.mean.view(-1, *[1] * (lp.dim() - 1)) + self.lnS)

    def h_bound(self):
        return self.e * (1 + 3 * (self.mean + self.lnS)) + 2.0 ** -21 * (self.mean + self.lnS)


def check(V, x, ids, T=1.0, top=0, rows=None):
    got = V.logprobs(x, ids, T=T, top=top, rows=rows)
    assert V.get_error() == 0
    M = got.entropy.numel()
    live = torch.arange(M, device="cuda") if ids is None else (ids >= 0).nonzero()[:, 0]
    w = Want((x if rows is None else x[rows.long().clamp(min=0)])[live], T)
    if ids is not None:
        lp = w.lp.gather(1, ids[live].long()[:, None])[:, 0]
        g = got.logprob[live].double()
        inf = lp == -math.inf
        assert torch.equal(g[inf], lp[inf])
        assert ((g - lp).abs() <= w.lp_bound(lp))[~inf].all(), ((g - lp).abs()[~inf]).max()
        dead = torch.ones(M, dtype=torch.bool, device="cuda")
        dead[live] = False
        assert (got.logprob[dead] == 0).all() and (got.entropy[dead] == 0).all() and (got.stats[dead] == 0).all()
        if top:
            assert (got.top_ids[dead] == -1).all() and (got.top_logprobs[dead] == 0).all()
    assert ((got.entropy[live].double() - w.H).abs() <= w.h_bound()).all(), (got.entropy[live].double() - w.H).abs().max()
    if top:
        n = min(top, x.shape[1])
        xs = (x if rows is None else x[rows.long().clamp(min=0)])[live].float()
        order = (xs + 0.0).sort(dim=1, descending=True, stable=True).indices[:, :n]      # equal ones by rising index
        assert torch.equal(got.top_ids[live, :n].long(), order)
        assert (got.top_ids[live, n:] == -1).all() and (got.top_logprobs[live, n:] == -math.inf).all()
        lp = w.lp.gather(1, order)
        g = got.top_logprobs[live, :n].double()
        inf = lp == -math.inf
        assert torch.equal(g[inf], lp[inf])
        assert ((g - lp).abs() <= w.lp_bound(lp))[~inf].all()
    return got, w, live


SIZES = [(1, 1), (3, 2), (5, 7), (2, 33), (70, 1000), (9, 4099), (400, 5003), (3, 32000), (20, 65537), (2, 151936), (310, 128257)]


@pytest.mark.parametrize("M,n", SIZES)
@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("top", [0, 1, 5, 32])
def test_logprobs(V, M, n, dtype, top):
    g = gen(M + n)
    x = (torch.randn(M, n, generator=g, device="cuda") * 3).to(dtype)
    ids = torch.randint(-1 if M > 1 else 0, n, (M,), generator=g, device="cuda", dtype=torch.int32)
    check(V, x, ids, T=[1.0, 0.7, 2.5][(M + top) % 3], top=top)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shift", [0, 1, 3, 5])
def test_rows_at_any_address(V, dtype, shift):
    wide = (torch.randn(6, 3000, generator=gen(shift), device="cuda") * 2).to(dtype)
    x = wide[:, shift:shift + 2911]
    got, _, _ = check(V, x, i32([0, 1, 2910, 7, 100, -1]), top=7)
    same = V.logprobs(x.contiguous(), i32([0, 1, 2910, 7, 100, -1]), top=7)
    assert torch.equal(got.top_ids, same.top_ids)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n", [100, 20000, 130001])
def test_ties_masks_and_orders(V, dtype, n):
    g = gen(n)
    rows = [torch.full((n,), 0.25),                                   # all equal
            torch.arange(n).float().mul_(60.0 / n).sub_(30),          # rising: every entry is a new largest
            torch.arange(n).float().mul_(-60.0 / n),                  # falling
            torch.randint(-3, 4, (n,)).float(),                       # many ties
            torch.where(torch.arange(n) % 997 == 5, 1.0, -math.inf),  # few words allowed
            torch.where(torch.arange(n) == n - 1, -5.0, -math.inf),   # a single one
            torch.where(torch.arange(n) % 2 == 0, 0.0, -0.0),         # zeros of both signs are equal
            torch.randn(n) * 300]                                     # almost one-hot
    x = torch.stack(rows).cuda().to(dtype)
    ids = i32([n // 2, n - 1, 0, 3, 5, n - 1, 1, int(x[7].float().argmax())])
    for top in (1, 20, 32):
        check(V, x, ids, top=top)
    # a given token without weight
    got = V.logprobs(x[4:6], i32([6, 0]))
    assert (got.logprob == -math.inf).all() and got.entropy.isfinite().all()


def test_rows_without_a_distribution(V):
    n = 5000
    x = torch.randn(6, n, device="cuda")
    x[0] = -math.inf
    x[1, 17] = math.nan
    x[2, 4000] = math.inf
    x[3] = math.nan
    x[4, 4999] = -math.nan
    for dtype in (F32, BF, HF):
        got = V.logprobs(x.to(dtype), i32([3] * 6), top=4)
        assert V.get_error() == 0
        for t in (got.logprob, got.entropy, got.top_logprobs, got.stats):
            assert t[:5].isnan().all() and t[5].isfinite().all()
        assert (got.top_ids[:5] == -1).all() and (got.top_ids[5] >= 0).all()


def test_largest_and_smallest_logits(V):
    # far from 0 and far apart: only differences count
    for dtype, big in ((F32, 1e30), (BF, 1e30), (HF, 60000.0)):
        x = torch.randn(4, 3001, generator=gen(3), device="cuda").to(dtype)
        x[1] = x[1] * 0 - big
        x[2] = x[2] * 0 + big
        x[3, 5], x[3, 6] = big, -big
        got = V.logprobs(x, i32([7, 7, 7, 5]), top=2)
        flat = math.log(3001)
        assert (got.logprob[1:3] + flat).abs().max() <= 1e-5 and (got.entropy[1:3] - flat).abs().max() <= 1e-4
        assert got.logprob[3] == 0 and got.entropy[3] == 0 and got.top_ids[3, 0] == 5
        assert got.top_ids[1].tolist() == [0, 1] and V.get_error() == 0


@pytest.mark.parametrize("dtype", [F32, BF])
def test_masks_of_the_lowest_value(V, dtype):
    # beside entries of -inf, in rows with and without others; and references near the end
    # of the type, where distances over T pass 32 bits
    low, n = torch.finfo(dtype).min, 9000
    x = (torch.randn(6, n, generator=gen(11), device="cuda") * 2).to(dtype)
    x[0, ::2], x[0, 1::4] = low, -math.inf
    x[1], x[1, 100:6000] = low, -math.inf
    x[2, :7000], x[2, ::3] = low, -math.inf
    x[3, 17] = -low
    x[4, 4000:], x[4, 9] = -math.inf, -low
    x[5], x[5, 5000], x[5, 5001] = low, -low, -low
    for T in (1.0, 0.01, 1e-10, 100.0):
        got = V.logprobs(x, i32([3, 50, 8999, 17, 9, 5001]), T=T, top=2)
        grad = V.logprobs_grad(x, i32([3, 50, 8999, 17, 9, 5001]), got, grad_logprob=torch.ones(6, device="cuda"),
                               grad_entropy=torch.ones(6, device="cuda"), T=T)
        assert V.get_error() == 0 and grad.isfinite().all()
        flat = math.log(n - 5900)
        want = torch.tensor([-flat, 0, 0, -math.log(2)], device="cuda")
        ent = torch.tensor([flat, 0, 0, math.log(2)], device="cuda")
        rows = torch.tensor([1, 3, 4, 5], device="cuda")
        assert ((got.logprob[rows] - want).abs() <= 1e-5).all() and ((got.entropy[rows] - ent).abs() <= 1e-4).all()
        assert got.top_ids[5].tolist() == [5000, 5001] and got.top_ids[3, 0] == 17
    check(V, x[[0, 2]], i32([3, 8999]), T=1.0, top=5)
    check(V, x[[0, 2]], i32([3, 8999]), T=0.5, top=0)


def test_rows_shared_missing_and_out_of_range(V):
    x = torch.randn(10, 4000, generator=gen(4), device="cuda").to(BF)
    rows, ids = i32([3, 3, 9, 0, 3]), i32([5, 6, 3999, 0, 5])
    got, _, _ = check(V, x, ids, rows=rows, top=3)
    assert got.logprob[0] == got.logprob[4] and torch.equal(got.top_ids[0], got.top_ids[1])
    bad = V.logprobs(x, ids, rows=i32([3, 10, -1, 0, 3]), top=3)
    assert V.get_error() == BAD_CU
    assert bad.logprob[[1, 2]].tolist() == [0, 0] and (bad.top_ids[[1, 2]] == -1).all()
    assert torch.equal(bad.logprob[[0, 3, 4]], got.logprob[[0, 3, 4]])
    V.logprobs(x, i32([4000, 1, 2, 3, 4, 5, 6, 7, 8, 9]))
    assert V.get_error() == BAD_ID
    got = V.logprobs(x, None, top=2)
    assert got.logprob is None
    check(V, x, None, top=2)
    assert V.logprobs(x, i32([])).entropy.numel() == 0 and V.get_error() == 0


def test_repeats_itself(V):
    x = (torch.randn(300, 50001, generator=gen(6), device="cuda") * 3).to(BF)
    ids = torch.randint(0, 50001, (300,), generator=gen(7), device="cuda", dtype=torch.int32)
    first = V.logprobs(x, ids, top=20)
    for _ in range(5):
        again = V.logprobs(x, ids, top=20)
        assert all(torch.equal(getattr(first, n), getattr(again, n)) for n in ("logprob", "entropy", "top_ids", "top_logprobs", "stats"))


# ---- gradient ------------------------------------------------------------------------

def grad64(w, ids, T, gl, gh, top_ids=None, gt=None):
    """The formula, and the sum of the magnitudes of its terms (whose errors add)."""
    p, lnp = w.p, w.lp.where(w.p > 0, 0.0)
    all_ = gl + (gt.sum(1) if gt is not None else 0)
    d = -p * (all_[:, None] + gh[:, None] * (lnp + w.H[:, None]))
    mag = p * (all_.abs()[:, None] + gh.abs()[:, None] * (lnp.abs() + w.H[:, None]))
    one = torch.zeros_like(p).scatter_(1, ids.long()[:, None], gl[:, None])
    if gt is not None:
        one.scatter_add_(1, top_ids.long(), gt)
    return (d + one) / T, (mag + one.abs()) / T


@pytest.mark.parametrize("M,n", [(1, 1), (4, 9), (7, 1000), (5, 32000), (3, 32003), (2, 151937)])
@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("top", [0, 5])
@pytest.mark.parametrize("inplace", [False, True])
def test_gradient(V, M, n, dtype, top, inplace):
    g = gen(M * n + top)
    T = 0.8
    x = (torch.randn(M, n, generator=g, device="cuda") * 3).to(dtype)
    if n > 8:
        x[0, 3:7] = -math.inf
    ids = torch.randint(0, n, (M,), generator=g, device="cuda", dtype=torch.int32)
    if M > 2:
        ids[1] = x[1].float().argmax()       # also among the alternatives
    top = min(top, n)
    gl, gh = torch.randn(M, generator=g, device="cuda"), torch.randn(M, generator=g, device="cuda") * 0.3
    gt = torch.randn(M, top, generator=g, device="cuda") if top else None
    w = Want(x, T)
    fwd = V.logprobs(x, ids, T=T, top=top)
    got = V.logprobs_grad(x, ids, fwd, grad_logprob=gl, grad_entropy=gh, grad_top=gt, T=T, out=x if inplace else None)
    assert V.get_error() == 0 and got.dtype == dtype
    want, mag = grad64(w, ids, T, gl.double(), gh.double(), fwd.top_ids, None if gt is None else gt.double())
    # p has the error of its logarithm; the entropy's error is one of the bracket
    tol = mag * 2 * (w.e + 2.0 ** -21 * (w.range + 4)) + w.p * gh.abs().double()[:, None] * w.h_bound()[:, None] / T
    tol = tol + HALF_STEP[dtype] * want.abs() + (2.0 ** -25 if dtype == HF else 1e-37)
    assert ((got.double() - want).abs() <= tol).all(), ((got.double() - want).abs() - tol).max()


def test_gradient_is_what_differences_say(V):
    # the loss as the kernels compute it moves along the gradient as the gradient says
    n, T = 5000, 1.3
    g = gen(11)
    x = torch.randn(3, n, generator=g, device="cuda") * 2
    ids = i32([4, 77, 4999])
    a, b = torch.randn(3, generator=g, device="cuda"), torch.randn(3, generator=g, device="cuda")
    c = torch.randn(3, 4, generator=g, device="cuda")
    fwd = V.logprobs(x, ids, T=T, top=4)
    grad = V.logprobs_grad(x, ids, fwd, grad_logprob=a, grad_entropy=b, grad_top=c, T=T).double()
    way = torch.randn(3, n, generator=g, device="cuda", dtype=torch.float64)
    way[:, fwd.top_ids[0].long()] *= 0.01
    h = 2.0 ** -7

    def loss(y):
        o = V.logprobs(y.float(), ids, T=T)
        t = torch.log_softmax(y.float().double() / T, 1).gather(1, fwd.top_ids.long())
        return (a.double() * o.logprob.double() + b.double() * o.entropy.double()).sum() + (c.double() * t).sum()

    there = (loss(x.double() + h * way) - loss(x.double() - h * way)) / (2 * h)
    # float32 results of size 10 (6 of them, half a step each, and the sums' 2^-20) over 2 h,
    # and the third derivative, at most 8 h^2 / T^3 of the sum of the |factors|
    tol = 6 * 10 * 2.0 ** -20 / (2 * h) + 8 * h * h * float(a.abs().sum() + 10 * b.abs().sum() + c.abs().sum())
    assert abs(float(there - (grad * way).sum())) <= tol


def test_gradient_rows_that_have_none(V):
    x = torch.randn(5, 3001, generator=gen(12), device="cuda").to(BF)
    x[3, 5] = math.nan
    ids = i32([5, -1, 3001, 7, 9])
    fwd = V.logprobs(x, ids, top=3)
    assert V.get_error() == BAD_ID
    out = torch.full((5, 3008), 7.0, dtype=BF, device="cuda")
    got = V.logprobs_grad(x, ids, fwd, grad_logprob=torch.ones(5, device="cuda"), grad_top=torch.ones(5, 3, device="cuda"),
                          out=out[:, :3001])
    assert V.get_error() == 0
    assert (got[[1, 2]] == 0).all() and got[3].isnan().all() and got[[0, 4]].isfinite().all()
    assert (out[:, 3001:] == 7).all()
    # no given gradient at all: zeros; the entropy alone, and without ids
    assert (V.logprobs_grad(x[[0, 4]], ids[[0, 4]], V.logprobs(x[[0, 4]], ids[[0, 4]])) == 0).all()
    x = x[[0, 4]].contiguous()
    f = V.logprobs(x)
    got = V.logprobs_grad(x, None, f, grad_entropy=torch.ones(2, device="cuda")).double()
    w = Want(x, 1.0)
    want, mag = grad64(w, i32([0, 0]), 1.0, torch.zeros(2, device="cuda").double(), torch.ones(2, device="cuda").double())
    assert ((got - want).abs() <= HALF_STEP[BF] * want.abs() + mag * 2.0 ** -15 + w.p * w.h_bound()[:, None]).all()


def test_captured_and_overlapping(V):
    cases = []
    for seed in (1, 2):
        x = (torch.randn(40, 30001, generator=gen(seed), device="cuda") * 3).to(BF)
        ids = torch.randint(0, 30001, (40,), generator=gen(seed), device="cuda", dtype=torch.int32)
        cases.append((x, ids, torch.randn(40, generator=gen(seed), device="cuda")))

    def both(x, ids, g):
        f = V.logprobs(x, ids, top=9)
        return f.logprob, f.entropy, f.top_ids, f.top_logprobs, V.logprobs_grad(x, ids, f, grad_logprob=g, grad_entropy=g)

    want = [both(*c) for c in cases]
    torch.cuda.synchronize()
    graphs = []
    for c in cases:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = both(*c)
        graphs.append((g, out))
    sts = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(10):
        for (g, _o), st in zip(graphs, sts):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for (_g, out), ref in zip(graphs, want):
        assert all(torch.equal(a, b) for a, b in zip(out, ref))
