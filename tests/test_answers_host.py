"""Refusals of the log probabilities, the positions on several axes and cross attention, and
what the host computes for them: nothing here reaches a GPU."""
import ctypes
import math
from types import SimpleNamespace

import pytest
import torch

from test_cache_host import lib, nodes_of, small_cache, structs  # noqa: F401

INVALID, DTYPE, CAPACITY = -1, -2, -6


def test_log_probabilities_are_checked_before_any_device_work(lib):  # noqa: F811
    good = dict(logits=1 << 30, dtype=lib.SPECDEC_BF16, row_stride=100, num_rows=4, V=100, T=1.0, ids=1 << 20, rows=None,
                n_tokens=4, top=3, out_logprob=1 << 21, out_entropy=1 << 22, out_top_ids=1 << 23, out_top_logprobs=1 << 24,
                out_stats=1 << 25)

    def call(**kw):
        return lib.specdec_logprobs(None, *{**good, **kw}.values(), None)

    assert call(dtype=lib.SPECDEC_E4M3) == DTYPE
    for bad in (dict(logits=None), dict(logits=(1 << 30) + 1), dict(row_stride=99), dict(num_rows=3), dict(num_rows=0), dict(V=0),
                dict(V=(1 << 30) + 1), dict(T=0.0), dict(T=-1.0), dict(T=math.inf), dict(T=math.nan), dict(T=1e-30), dict(T=2e18), dict(ids=None),
                dict(n_tokens=-1), dict(n_tokens=1 << 31), dict(top=-1), dict(top=33), dict(out_top_ids=None),
                dict(out_top_logprobs=None), dict(out_stats=(1 << 25) + 4),
                dict(out_logprob=None, out_entropy=None, top=0, out_stats=None),
                dict(out_logprob=(1 << 30) + 796), dict(out_entropy=(1 << 20) + 12), dict(rows=1 << 22),      # over inputs
                dict(out_entropy=(1 << 21) + 12)):                                                            # over each other
        assert call(**bad) == INVALID, bad
    assert call(n_tokens=0) == INVALID          # no handle
    grad = dict(logits=1 << 30, dtype=lib.SPECDEC_F32, row_stride=100, V=100, T=1.0, ids=1 << 20, n_tokens=4, top=3,
                logprob=1 << 21, entropy=1 << 22, top_ids=1 << 23, top_logprobs=1 << 24, stats=1 << 25,
                grad_logprob=1 << 26, grad_entropy=1 << 27, grad_top=1 << 28, out=1 << 31, out_row_stride=100)

    def back(**kw):
        return lib.specdec_logprobs_grad(None, *{**grad, **kw}.values(), None)

    assert back(dtype=7) == DTYPE
    for bad in (dict(logits=None), dict(out=None), dict(stats=None), dict(out=(1 << 31) + 2), dict(out_row_stride=99), dict(ids=None),
                dict(logprob=None), dict(entropy=None), dict(top_ids=None), dict(top_logprobs=None), dict(top=0), dict(T=0.0),
                dict(out=(1 << 30) + 400), dict(out=1 << 30, out_row_stride=104), dict(out=(1 << 26) - 1596), dict(out=1 << 25)):
        assert back(**bad) == INVALID, bad


def test_positions_are_checked_before_any_device_work(lib):  # noqa: F811
    c, n = structs(lib)
    axes = bytes([0, 1, 2, 0] * 16)
    good = dict(dtype=lib.SPECDEC_BF16, k=1 << 20, k_row_stride=256, k_head_stride=128, v=1 << 21, v_row_stride=256,
                v_head_stride=128, q=1 << 22, q_row_stride=1024, q_head_stride=128, q_heads=8, out_q=1 << 23, rotary=1 << 24,
                rotary_dim=128, rotary_positions=9, interleaved=0, positions=1 << 25, position_stride=3, num_axes=3, axes=axes,
                offsets=None)

    def append(**kw):
        return lib.specdec_cache_append_positions(None, c, n, *{**good, **kw}.values(), None)

    for bad in (dict(rotary=None), dict(offsets=1 << 26), dict(num_axes=0), dict(num_axes=5), dict(num_axes=2), dict(position_stride=2),
                dict(positions=None, offsets=1 << 26, rotary=None), dict(positions=(1 << 23) + 8), dict(rotary_dim=24), dict(k=None)):
        assert append(**bad) == INVALID, bad
    turn = dict(dtype=lib.SPECDEC_BF16, x=1 << 20, x_row_stride=1024, x_head_stride=128, N=5, heads=8, head_dim=128, positions=1 << 25,
                position_stride=5, num_axes=3, axes=axes, rotary=1 << 24, rotary_dim=128, rotary_positions=9, interleaved=0, inverse=0,
                out=1 << 22, out_row_stride=1024, out_head_stride=128)

    def rotate(**kw):
        return lib.specdec_rotate(None, *{**turn, **kw}.values(), None)

    assert rotate(dtype=lib.SPECDEC_F32) == DTYPE
    for bad in (dict(x=None), dict(x=(1 << 20) + 8), dict(out=None), dict(positions=None), dict(rotary=None), dict(N=-1), dict(N=1 << 31),
                dict(heads=0), dict(head_dim=100), dict(head_dim=2048), dict(rotary_dim=24), dict(rotary_dim=144), dict(num_axes=2),
                dict(num_axes=5), dict(position_stride=4), dict(rotary_positions=0), dict(x_row_stride=1020), dict(out_head_stride=120),
                dict(out_row_stride=1016), dict(out=(1 << 20) + 16), dict(out=1 << 20, out_row_stride=1032), dict(out=1 << 24),
                dict(out=(1 << 25) + 32)):
        assert rotate(**bad) == INVALID, bad
    # half of a head turns 256 values: more pairs than two bits each are held for
    assert rotate(head_dim=512, rotary_dim=256, x_head_stride=512, x_row_stride=4096, out_head_stride=512, out_row_stride=4096) == INVALID


def test_cross_attention_is_checked_before_any_device_work(lib):  # noqa: F811
    c, n = structs(lib)
    good = dict(dtype=lib.SPECDEC_BF16, q=1 << 20, q_row_stride=1024, q_head_stride=128, q_heads=8, mask=1 << 21, mask_stride=64,
                mask_slots=64, softmax_scale=1.0, out=1 << 22, workspace=1 << 23, workspace_bytes=1 << 30)

    def cross(**kw):
        return lib.specdec_cross_attention(None, c, n, *{**good, **kw}.values(), None)

    assert cross(dtype=lib.SPECDEC_F32) == DTYPE
    for bad in (dict(q_heads=7), dict(softmax_scale=math.nan), dict(q=None), dict(out=None), dict(mask_stride=63), dict(mask_slots=-1),
                dict(mask=(1 << 22) + 100), dict(out=(1 << 20) + 16)):
        assert cross(**bad) == INVALID, bad
    assert lib.specdec_cross_attention_workspace(None, c, 2, 3, 8, 4) == INVALID


def fake(lib):  # noqa: F811
    from speculative_decoding_rejection_decode_gb300.verifier import Verifier
    v = Verifier.__new__(Verifier)
    v.device, v._h, v._at, v._empty = torch.device("cpu"), 0, -1, torch.zeros(4, dtype=torch.int32)
    return v


def test_arguments_of_log_probabilities(lib):  # noqa: F811
    v = fake(lib)
    x = torch.zeros(4, 10)
    i = lambda n: torch.zeros(n, dtype=torch.int32)
    for bad in (dict(logits=x.double()), dict(logits=x[0]), dict(logits=x.T), dict(logits=x[:1].expand(4, 10)), dict(ids=i(4).long()),
                dict(ids=i(5)), dict(ids=i(8)[::2]), dict(rows=i(3)), dict(top=33), dict(top=-1)):
        with pytest.raises(ValueError):
            v.logprobs(**{"logits": x, "ids": i(4), **bad})
    with pytest.raises(ValueError, match="no rows"):
        v.logprobs(x[:0], i(3), rows=i(3))
    assert v.logprobs(x, i(0)).entropy.numel() == 0
    o = v.logprobs(x[:0], None, top=2)
    assert o.logprob is None and o.top_ids.shape == (0, 2)
    from speculative_decoding_rejection_decode_gb300 import LogprobOutput
    f = torch.zeros
    with pytest.raises(ValueError, match="out"):
        v.logprobs(x, i(4), out=LogprobOutput(None, f(4), None, None, f(4, 2)))
    with pytest.raises(ValueError, match="out.stats"):
        v.logprobs(x, i(4), out=LogprobOutput(f(4), f(4), None, None, f(4, 3)))
    fwd = LogprobOutput(f(4), f(4), None, None, f(4, 2))
    for bad in (dict(logits=f(5, 10)), dict(ids=None), dict(grad_logprob=f(3)), dict(grad_entropy=f(4).double()),
                dict(grad_top=f(4, 0)), dict(grad_top=f(4, 2)), dict(out=f(4, 11)), dict(out=f(4, 10).half())):
        with pytest.raises(ValueError):
            v.logprobs_grad(**{"logits": x, "ids": i(4), "forward": fwd, **bad})
    with pytest.raises(ValueError, match="grad_logprob"):
        v.logprobs_grad(x, None, LogprobOutput(None, f(4), None, None, f(4, 2)), grad_logprob=f(4))


def test_arguments_of_positions(lib):  # noqa: F811
    v = fake(lib)
    x = torch.zeros(6, 4, 64, dtype=torch.bfloat16)
    t = torch.zeros(9, 2, 32)
    p = torch.zeros(2, 6, dtype=torch.int32)
    axes = (0, 1) * 16
    for bad in (dict(x=x.float()), dict(x=x[0]), dict(x=x[..., ::2]), dict(x=x[:, :, 1:]), dict(positions=p.long()), dict(positions=p[:, :5]),
                dict(positions=p.T.contiguous().T), dict(positions=torch.zeros(5, 6, dtype=torch.int32)), dict(axes=None),
                dict(axes=axes[:-1]), dict(axes=(0, 2) * 16), dict(axes=(0, -1) * 16), dict(rotary=t.double()), dict(rotary=t[:, :, :4]),
                dict(rotary=torch.zeros(9, 2, 40)), dict(rotary=t[:0]), dict(out=x.float()), dict(out=x[:5])):
        with pytest.raises(ValueError):
            v.rotate(**{"x": x, "positions": p, "rotary": t, "axes": axes, **bad})
    assert v.rotate(x[:0], p[:, :0], t, axes=axes).shape == (0, 4, 64)
    c, n = small_cache(lib), nodes_of()
    k = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    p = torch.zeros(3, dtype=torch.int32)
    off = torch.zeros(2, dtype=torch.int32)
    for bad, what in ((dict(positions=p, rotary=None), "without rotary"), (dict(position_offsets=off, rotary=None), "without rotary"),
                      (dict(positions=p, position_offsets=off), "exclude"), (dict(axes=axes), "axes without"),
                      (dict(positions=p[:2]), "positions"), (dict(position_offsets=off.long()), "position_offsets"),
                      (dict(position_offsets=p), "position_offsets")):
        with pytest.raises(ValueError, match=what):
            c.append(k, k, n["page_table"], n["lengths"], n["cu_num_nodes"], **{"rotary": t, **bad})


def test_arguments_of_masks(lib):  # noqa: F811
    c, n = small_cache(lib), nodes_of()
    c.verifier._empty = torch.zeros(4, dtype=torch.int32)
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    m = torch.ones(2, 20, dtype=torch.bool)
    for bad in (m.int(), m[0], m[:1], m.T.contiguous().T, m[:1].expand(2, 20)):
        with pytest.raises(ValueError, match="mask"):
            c.cross_attend(q, n["page_table"], n["lengths"], n["cu_num_nodes"], mask=bad)
    for bad in (q[:, :3], q.float(), q[..., :32]):
        with pytest.raises((ValueError, TypeError)):
            c.cross_attend(bad, n["page_table"], n["lengths"], n["cu_num_nodes"], mask=m)


def test_rotary_axes(lib):  # noqa: F811
    from speculative_decoding_rejection_decode_gb300 import rotary_axes
    assert rotary_axes((2, 3, 1)) == (0, 0, 1, 1, 1, 2)
    assert rotary_axes((4, 2, 2), spread=True) == (0, 1, 2, 0, 1, 2, 0, 0)
    assert rotary_axes((1, 0, 3), spread=True) == (0, 2, 2, 2)
    got = rotary_axes((24, 20, 20), spread=True)
    assert got[:60] == (0, 1, 2) * 20 and got[60:] == (0,) * 4
    for bad in ((), (0, 0), (3, -1)):
        with pytest.raises(ValueError):
            rotary_axes(bad)


def test_rows_of_a_tree_s_tokens(lib):  # noqa: F811
    from speculative_decoding_rejection_decode_gb300 import tree_rows
    i = lambda x: torch.tensor(x, dtype=torch.int32)
    # three requests: nodes 0 .. 4 with two accepted, a single one, three with none accepted
    path, cu = i([1, 3, -1, -1, -1, -1, -1, -1, -1]), i([0, 5, 6, 9])
    assert tree_rows(path, cu).tolist() == [0, 1, 3, -1, -1, 5, 6, -1, -1]
    # every node accepted: the next request's first token still comes from its node 0
    assert tree_rows(i([1, 2, -1, 1, -1]), i([0, 3, 5])).tolist() == [0, 1, 2, 3, 4]
    assert tree_rows(i([]), i([0, 0])).numel() == 0
    # a request without nodes between two others
    assert tree_rows(i([-1, 1, -1]), i([0, 1, 1, 3])).tolist() == [0, 1, 2]
