"""Verification from probabilities and given random numbers on the GPU against a
plain 64-bit implementation (exact rationals where the decision is close)."""
from fractions import Fraction

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

BAD_DRAFT_ID, BAD_CU = 1, 2


@pytest.fixture(scope="module")
def V():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_rejection_decode_gb300 import Verifier
    v = Verifier(0)
    yield v
    v.close()


def plain(p, q, ids, cu, u, s):
    """Tokens, counts and, per request, how near the sampled token's borders lie."""
    B = len(cu) - 1
    p, u, s = p.astype(np.float64), u.astype(np.float64), s.astype(np.float64)
    tokens = np.full(cu[-1] + B, -1, np.int64)
    nacc, near = np.zeros(B, np.int64), np.ones(B)
    for b in range(B):
        g = cu[b + 1] - cu[b]
        n = 0
        while n < g:
            d = cu[b] + n
            x = int(ids[d])
            if not 0 <= x < p.shape[1]:
                break
            px, qx = p[cu[b] + b + n, x], 1.0 if q is None else float(q[d, x])
            if not (u[d] < 1 and Fraction(u[d]) * Fraction(qx) < Fraction(px)):
                break
            tokens[cu[b] + b + n] = x
            n += 1
        row = np.where(p[cu[b] + b + n] > 0, p[cu[b] + b + n], 0.0)
        w = row
        if n < g:
            d = cu[b] + n
            if q is None:
                qd = np.zeros(p.shape[1])
                if 0 <= ids[d] < p.shape[1]:
                    qd[ids[d]] = 1.0
            else:
                qd = q[d].astype(np.float64)
            r = p[cu[b] + b + n] - qd
            w = np.where(r > 0, r, 0.0)
            if not w.sum() > 0:
                w = row
        c = np.cumsum(w)
        t = s[b] * c[-1]
        tokens[cu[b] + b + n] = np.argmax(c > t) if c[-1] > 0 else 0
        if c[-1] > 0:
            near[b] = np.abs(c - t).min() / c[-1]
        nacc[b] = n
    return tokens, nacc, near


def make(V_, counts, *, one_hot=False, seed=0, noise=1.0, stride=None):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    cu = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    B, nd = len(counts), int(cu[-1])
    logits = torch.randn(nd + B, V_, generator=g, device="cuda") * 3
    p = logits.softmax(1)
    own = torch.tensor([cu[b] + b + i for b in range(B) for i in range(counts[b])], dtype=torch.long, device="cuda")
    q = (logits[own] + noise * torch.randn(nd, V_, generator=g, device="cuda")).softmax(1)
    ids = torch.multinomial(q, 1, generator=g)[:, 0].to(torch.int32) if nd else torch.zeros(0, dtype=torch.int32, device="cuda")
    if one_hot and nd:
        ids = p[own].argmax(1).to(torch.int32)
    u, s = torch.rand(nd, generator=g, device="cuda"), torch.rand(B, generator=g, device="cuda")
    if stride:
        wide = torch.zeros(nd + B, stride, device="cuda")
        wide[:, :V_] = p
        p = wide[:, :V_]
    return p, None if one_hot else q, ids, torch.tensor(cu, device="cuda"), u, s


def run(V, w):
    out = V.sample_given(*w)
    host = [None if t is None else t.cpu().numpy() for t in w]
    tok, nacc, near = plain(*host)
    return out, tok, nacc, near


CASES = [(1, [0]), (2, [1, 2]), (5, [3, 0, 2, 1]), (8, [1] * 50), (127, [4, 4]), (1000, [7, 0, 40]), (4093, [2, 5]),
         (32000, [5] * 8), (151936, [1, 8, 3]), (256000, [7, 7])]


@pytest.mark.parametrize("V_,counts", CASES)
@pytest.mark.parametrize("one_hot", [False, True])
def test_given_matches_the_definition(V, V_, counts, one_hot):
    for seed in range(4):
        w = make(V_, counts, one_hot=one_hot, seed=seed, stride=V_ + 3 if seed == 3 else None)
        out, tok, nacc, near = run(V, w)
        assert V.get_error() == 0
        assert out.num_accepted.tolist() == nacc.tolist()
        cu = w[3].tolist()
        for b in range(len(counts)):
            r = slice(cu[b] + b, cu[b + 1] + b + 1)
            # sums are held to 2^-40 of the total at the least; a border nearer
            # than that may fall either way
            if near[b] > 2.0 ** -40:
                assert out.tokens[r].tolist() == tok[r].tolist(), (seed, b)


def test_accept_test_is_exact(V):
    # r q against p at equality and one step to each side, where a division
    # rounded to 32 bits cannot tell
    rng = np.random.default_rng(1)
    n = 4000
    q = rng.random(n).astype(np.float32) * np.float32(0.9) + np.float32(1e-3)
    u = rng.random(n).astype(np.float32)
    p = (u.astype(np.float64) * q.astype(np.float64)).astype(np.float32)
    step = rng.integers(-1, 2, n)
    p = np.where(step > 0, np.nextafter(p, np.float32(2)), np.where(step < 0, np.nextafter(p, np.float32(0)), p)).astype(np.float32)
    want = [Fraction(float(a)) * Fraction(float(b)) < Fraction(float(c)) for a, b, c in zip(u, q, p)]
    P = np.zeros((2 * n, 2), np.float32)
    P[0::2, 0] = p
    P[:, 1] = 0.25
    Q = np.stack([q, np.zeros(n, np.float32)], 1)
    d = lambda x: torch.tensor(x, device="cuda")
    out = V.sample_given(d(P), d(Q), d(np.zeros(n, np.int32)), d(np.arange(n + 1, dtype=np.int32)), d(u), d(np.zeros(n, np.float32)))
    assert out.num_accepted.tolist() == [int(x) for x in want]


def test_ratio_conventions_and_fallbacks(V):
    d = lambda x, t=torch.float32: torch.tensor(x, dtype=t, device="cuda")
    # p = q = 0 and p = 0 reject; q = 0 < p accepts; r = 0 accepts any p > 0
    P = d([[0.0, 1.0], [0.5, 0.5]] * 2 + [[0.5, 0.5], [0.25, 0.75]] * 2)
    Q = d([[0.0, 1.0], [1.0, 0.0], [0.0, 1.0], [1.0, 0.0]])
    out = V.sample_given(P, Q, d([0, 0, 0, 0], torch.int32), d([0, 1, 2, 3, 4], torch.int32),
                         d([0.0, 0.0, 0.999, 0.0]), d([0.5] * 4))
    assert out.num_accepted.tolist() == [0, 0, 1, 1]
    # request 0: p - q is 0 everywhere, the token comes from p; request 1: residual at 1 only... of p - q
    assert out.tokens.tolist()[0] == 1 and out.tokens.tolist()[2] == 1
    # s = 0 takes the first entry that weighs anything, the largest s below 1 the last
    P = d([[0.0, 0.25, 0.0, 0.75, 0.0]] * 2)
    e = d([], torch.int32)
    out = V.sample_given(P, P[:0], e, d([0, 0, 0], torch.int32), d([]), d([0.0, 1.0 - 2.0 ** -24]))
    assert out.tokens.tolist() == [1, 3]
    out = V.sample_given(P, P[:0], e, d([0, 0, 0], torch.int32), d([]), d([0.25, 0.24999]))
    assert out.tokens.tolist() == [3, 1]           # C(1) = s is not above s
    # a row without weight, and entries that are no weight
    P = d([[0.0, 0.0, 0.0], [float("nan"), -1.0, 0.5]])
    out = V.sample_given(P, None, e, d([0, 0, 0], torch.int32), d([]), d([0.9, 0.9]))
    assert out.tokens.tolist() == [0, 2] and V.get_error() == 0


def test_many_small_weights_keep_their_borders(V):
    # 2^18 equal weights beside a large one: a float32 running sum would lose them
    n = 1 << 18
    p = torch.full((1, n + 1), 2.0 ** -25, device="cuda")
    p[0, 0] = 1.0
    e = torch.zeros(0, dtype=torch.int32, device="cuda")
    cu = torch.zeros(2, dtype=torch.int32, device="cuda")
    total = 1.0 + n * 2.0 ** -25
    for k in (1, 2, 777, n - 1, n):
        s = min(np.float32((1.0 + (k - 0.5) * 2.0 ** -25) / total), np.float32(1 - 2.0 ** -24))   # s is in [0, 1)
        c = 1.0 + np.arange(n + 1) * 2.0 ** -25
        want = int(np.argmax(c > float(s) * total))
        out = V.sample_given(p, p[:0], e, cu, torch.zeros(0, device="cuda"), torch.tensor([s], device="cuda"))
        assert out.tokens.tolist() == [want]


def test_bad_ids_and_cu(V):
    w = list(make(100, [3, 3, 2], seed=1))
    good = V.sample_given(*w)
    w[2] = w[2].clone()
    w[2][4] = 100
    w[4] = torch.zeros_like(w[4])                    # all others accepted
    out = V.sample_given(*w)
    assert V.get_error() == BAD_DRAFT_ID and V.get_error() == 0
    assert out.num_accepted.tolist() == [3, 1, 2]
    assert int(out.tokens[4 + 1 + 1]) == -1          # behind request 1's extra token
    host = [t.cpu().numpy() for t in w]
    tok, nacc, _ = plain(*host)
    assert out.tokens.tolist() == tok.tolist()
    w = list(make(100, [3, 3, 2], seed=1))
    w[3] = torch.tensor([0, 3, 2, 8], dtype=torch.int32, device="cuda")
    from speculative_decoding_rejection_decode_gb300 import VerifyOutput
    out = VerifyOutput(tokens=torch.full((11,), 7, dtype=torch.int32, device="cuda"),
                       num_accepted=torch.full((3,), 7, dtype=torch.int32, device="cuda"), beta=None)
    V.sample_given(*w, out=out)
    assert V.get_error() == BAD_CU
    assert out.num_accepted[1] == 7 and torch.equal(out.tokens[:4], good.tokens[:4])


def test_agrees_with_the_generator_driven_verifier(V):
    # the accept uniforms of the counter-based generator give its accepted counts
    from speculative_decoding_rejection_decode_gb300 import uniform
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    B, gamma, V_ = 24, 5, 2000
    logits = torch.randn(B * (gamma + 1), V_, generator=g, device="cuda") * 2
    p = logits.softmax(1)
    rows = torch.arange(B * (gamma + 1), device="cuda").view(B, -1)[:, :gamma].reshape(-1)
    q = (logits[rows] + torch.randn(B * gamma, V_, generator=g, device="cuda")).softmax(1)
    ids = torch.multinomial(q, 1, generator=g)[:, 0].to(torch.int32)
    cu = torch.arange(0, B * gamma + 1, gamma, dtype=torch.int32, device="cuda")
    ref = V(logits, q, ids, cu, 1.0, 9)
    u = torch.cat([uniform(9, b, i, 0, 0, 1) for b in range(B) for i in range(gamma)])
    got = V.sample_given(p, q, ids, cu, u, torch.rand(B, device="cuda"))
    ratio = (p[rows].gather(1, ids[:, None].long()) / q.gather(1, ids[:, None].long()))[:, 0]
    clear = ((u - ratio.clamp(max=1.0)).abs() > 1e-5).view(B, gamma).all(1)
    assert clear.sum() >= B - 2
    assert torch.equal(got.num_accepted[clear], ref.num_accepted[clear])


def test_given_statistics(V):
    # slot 0 follows p: 2^15 requests of one distribution, chi-square
    rng = np.random.default_rng(11)
    B, V_ = 1 << 15, 6
    p0 = rng.dirichlet(np.ones(V_)).astype(np.float32)
    q0 = rng.dirichlet(np.ones(V_)).astype(np.float32)
    ids = torch.tensor(rng.choice(V_, B, p=q0.astype(np.float64) / q0.sum(dtype=np.float64)), dtype=torch.int32, device="cuda")
    P = torch.tensor(p0, device="cuda").repeat(2 * B, 1)
    Q = torch.tensor(q0, device="cuda").repeat(B, 1)
    g = torch.Generator(device="cuda")
    g.manual_seed(12)
    out = V.sample_given(P, Q, ids, torch.arange(B + 1, dtype=torch.int32, device="cuda"),
                         torch.rand(B, generator=g, device="cuda"), torch.rand(B, generator=g, device="cuda"))
    got = torch.bincount(out.tokens[0::2].long(), minlength=V_).cpu().numpy()
    want = p0.astype(np.float64) / p0.sum(dtype=np.float64) * B
    chi2 = float(((got - want) ** 2 / want).sum())
    assert chi2 < 20.5      # 5 degrees of freedom, p = 0.001
    alpha = np.minimum(p0, q0).sum()
    assert abs(float(out.num_accepted.float().mean()) - alpha) < 4 * 0.5 / np.sqrt(B)


def test_given_captured_and_overlapping(V):
    ws = [make(50000, [5, 0, 3, 8], seed=s) for s in (1, 2)]
    want = [V.sample_given(*w) for w in ws]
    torch.cuda.synchronize()
    graphs = []
    for w in ws:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = V.sample_given(*w)
        graphs.append((g, out))
    sts = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        for (g, _o), st in zip(graphs, sts):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for (_g, out), ref in zip(graphs, want):
        assert torch.equal(out.tokens, ref.tokens) and torch.equal(out.num_accepted, ref.num_accepted)
