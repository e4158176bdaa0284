"""Outputs over inputs that other blocks still read: refused before anything is launched."""
import pytest
import torch

from test_cache_host import lib, nodes_of, small_cache  # noqa: F401


def test_turned_queries_over_the_offsets_are_refused(lib):  # noqa: F811
    c, n = small_cache(lib), nodes_of()
    k = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    offsets = q.view(torch.int32).flatten()[10:12]
    with pytest.raises(ValueError, match="position_offsets"):
        c.append(k, k, n["page_table"], n["lengths"], n["cu_num_nodes"], q=q, out_q=q, rotary=torch.zeros(9, 2, 32), position_offsets=offsets)


@pytest.mark.gpu
def test_the_library_refuses_them_too():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_rejection_decode_gb300 import KVCache, SPECDEC_BF16, Verifier, specdec_cache_append_positions
    v = Verifier(0)
    cache = KVCache.empty(v, 4, 16, 2, 64)
    i = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    table, lengths, cu, offsets = i([[0, 1], [2, 3]]), i([0, 5]), i([0, 1, 3]), i([3, 4])
    k = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16, device="cuda")
    rotary = torch.zeros(20, 2, 32, device="cuda")
    nodes = cache._nodes(table, lengths, cu, None, 3)

    def call(at):
        return specdec_cache_append_positions(v.handle, cache._ref, nodes, SPECDEC_BF16, k.data_ptr(), 128, 64, k.data_ptr(), 128, 64,
                                              q.data_ptr(), 256, 64, 4, q.data_ptr(), rotary.data_ptr(), 64, 20, 0, None, 0, 1, None,
                                              at, torch.cuda.current_stream().cuda_stream)

    assert call(offsets.data_ptr()) == 0
    for at in (0, 40, 2 * q.numel() - 8):
        assert call(q.data_ptr() + at) == -1
    assert v.get_error() == 0
    v.close()


def test_a_gradient_of_rows_in_another_order_is_refused(lib):  # noqa: F811
    from speculative_decoding_rejection_decode_gb300 import LogprobOutput
    from test_answers_host import fake
    v, f = fake(lib), torch.zeros
    x, i = f(4, 10), lambda n: torch.zeros(n, dtype=torch.int32)
    assert v.logprobs(x[:0], i(0)).own_rows and not v.logprobs(x, i(0), rows=i(0)).own_rows
    out = LogprobOutput(f(0), f(0), None, None, f(0, 2))
    assert not v.logprobs(x, i(0), rows=i(0), out=out).own_rows and v.logprobs(x, i(0), out=out).own_rows
    # as many tokens as rows, but not their own: the gradient would be that of other rows
    with pytest.raises(ValueError, match="order"):
        v.logprobs_grad(x, i(4), LogprobOutput(f(4), f(4), None, None, f(4, 2), own_rows=False), grad_logprob=f(4))


def test_slots_behind_the_last_request_have_no_row(lib):  # noqa: F811
    from speculative_decoding_rejection_decode_gb300 import tree_rows
    i = lambda x: torch.tensor(x, dtype=torch.int32)
    # the verification leaves slots 5 .. 7 as they are: whatever lies there is no node
    path = i([1, -1, -1, 1, -1, 3, 0, 900])
    assert tree_rows(path, i([0, 3, 5])).tolist() == [0, 1, -1, 3, 4, -1, -1, -1]
    assert tree_rows(path, i([0, 0])).tolist() == [-1] * 8
