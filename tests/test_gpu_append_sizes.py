"""Appends of many rows: whatever a block takes, the rows are those of smaller appends."""
import pytest
import torch

from cache_reference import Step

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


@pytest.mark.parametrize("dtype,cache", [(BF, BF), (HF, HF), (BF, E4)])
@pytest.mark.parametrize("head_dim", [64, 128])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("N", [759, 761, 12159, 12161, 18241, 24320])
def test_many_rows_at_once(V, dtype, cache, head_dim, inter, N):
    from speculative_decoding_rejection_decode_gb300 import rotary_table
    s = Step(ctx=[0, 5, 0], nodes=[N // 3, N - N // 3 - 1, 1], kv_heads=1, group=2, head_dim=head_dim, dtype=dtype, cache=cache, page=64,
             seed=9, extra_rows=3, poison=False)
    table, c, n = rotary_table(N + 8, head_dim // 2), s.cache(V), s.n_rows
    flat = lambda: [t.view(torch.uint8).clone() if t.dtype == E4 else t.clone() for t in (s.k, s.v, s.ks, s.vs) if t is not None]
    was = flat()
    q = c.append(s.new_k, s.new_v, s.table, s.lengths, s.cu, q=s.q, rotary=table, interleaved=inter, out_q=torch.full_like(s.q, 7.0))
    at_once = flat()
    for t, w in zip((s.k, s.v, s.ks, s.vs), was):
        (t.view(torch.uint8) if t.dtype == E4 else t).copy_(w)
    # the same in pieces of 500 rows of one request
    for b in range(s.B):
        for j in range(0, s.nodes[b], 500):
            m = min(500, s.nodes[b] - j)
            at = slice(s.firsts[b] + j, s.firsts[b] + j + m)
            i = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
            piece = c.append(s.new_k[at], s.new_v[at], s.table[b:b + 1], i([s.ctx[b] + j]), i([0, m]), q=s.q[at], rotary=table, interleaved=inter)
            assert torch.equal(q[at], piece)
    assert V.get_error() == 0 and (q[n:] == 7.0).all()
    for a, t in zip(at_once, flat()):
        assert torch.equal(a, t)
