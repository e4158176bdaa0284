"""Dense rows turned in any order of rows and heads in memory."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def V():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_rejection_decode_gb300 import Verifier
    v = Verifier(0)
    yield v
    v.close()


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("N,heads", [(1, 5), (33, 1), (33, 5), (3000, 8)])
def test_rows_within_heads(V, N, heads, inter):
    from speculative_decoding_rejection_decode_gb300 import rotary_table
    D, table = 128, rotary_table(300, 96)
    g = torch.Generator(device="cuda")
    g.manual_seed(N)
    store = torch.randn(heads + 2, N + 1, D, generator=g, device="cuda").to(torch.bfloat16)
    before = store.clone()
    x = store[1:-1, :N].transpose(0, 1)                  # [N, heads, D], heads far apart
    pos = torch.randint(0, 300, (N,), generator=g, device="cuda", dtype=torch.int32)
    want = V.rotate(x.contiguous(), pos, table, interleaved=inter)
    for out in (torch.empty(heads, N, D, dtype=x.dtype, device="cuda").transpose(0, 1), torch.empty_like(want)):
        assert V.rotate(x, pos, table, interleaved=inter, out=out) is out
        assert torch.equal(out, want)
    assert V.rotate(x, pos, table, interleaved=inter, out=x) is x
    assert torch.equal(x, want) and V.get_error() == 0
    # nothing beside the rows moves
    x.copy_(before[1:-1, :N].transpose(0, 1))
    assert torch.equal(store, before)


def test_rows_that_overlap_are_refused(V):
    from speculative_decoding_rejection_decode_gb300 import SpecdecError, rotary_table
    table, pos = rotary_table(9, 64), torch.zeros(4, dtype=torch.int32, device="cuda")
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    flat = torch.zeros(4096, dtype=torch.bfloat16, device="cuda")
    for row, head in ((64, 64), (64, 128), (128, 32), (32, 256), (64, 192), (0, 64), (64, 0)):
        with pytest.raises(SpecdecError):
            V.rotate(x, pos, table, out=flat.as_strided((4, 2, 64), (row, head, 1)))
    for row, head in ((128, 64), (64, 256), (72, 280), (200, 64), (400, 136)):
        assert (V.rotate(x, pos, table, out=flat.as_strided((4, 2, 64), (row, head, 1))) == 0).all()
