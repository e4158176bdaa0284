"""Refusals of the cache's operators and of verification from given numbers, and
the rotary tables: nothing here reaches a GPU."""
import ctypes
import math
from types import SimpleNamespace

import pytest
import torch

from cache_reference import rotate64

INVALID, DTYPE, CAPACITY = -1, -2, -6


@pytest.fixture(scope="module")
def lib():
    from speculative_decoding_rejection_decode_gb300.build import build
    build()
    from speculative_decoding_rejection_decode_gb300 import _lib
    return _lib


def structs(lib, cache=None, nodes=None):
    c = dict(k=16, v=16, k_scale=None, v_scale=None, dtype=lib.SPECDEC_BF16, num_kv_heads=2, head_dim=128,
             page_size=16, num_pages=4)
    n = dict(page_table=16, table_stride=4, max_pages=4, lengths=16, cu=16, parent=None, B=2, N=3)
    c.update(cache or {})
    n.update(nodes or {})
    return ctypes.byref(lib.specdec_cache_t(**c)), ctypes.byref(lib.specdec_nodes_t(**n))


BAD_STRUCTS = [
    (dict(head_dim=96), None, INVALID), (dict(num_kv_heads=0), None, INVALID), (dict(page_size=0), None, INVALID),
    (dict(num_pages=0), None, INVALID), (dict(k=None), None, INVALID), (dict(v=24), None, INVALID),
    (dict(dtype=0), None, DTYPE), (dict(dtype=3), None, INVALID),             # e4m3 without scales
    (dict(dtype=2), None, DTYPE),                                             # f16 cache, bf16 rows
    (dict(num_pages=1 << 26), None, CAPACITY),                                # 2^31 rows
    (None, dict(B=0), INVALID), (None, dict(N=-1), INVALID), (None, dict(N=1 << 31), INVALID),
    (None, dict(max_pages=0), INVALID), (None, dict(table_stride=3), INVALID),
    (None, dict(page_table=None), INVALID), (None, dict(lengths=None), INVALID), (None, dict(cu=None), INVALID),
    (dict(num_kv_heads=4096, num_pages=1), dict(B=1 << 20), CAPACITY),        # more blocks than a grid holds
]


@pytest.mark.parametrize("cache,nodes,status", BAD_STRUCTS)
def test_caches_and_nodes_are_checked_before_any_device_work(lib, cache, nodes, status):
    c, n = structs(lib, cache, nodes)
    b = lib.SPECDEC_BF16
    assert lib.specdec_cache_append(None, c, n, b, 16, 8, 8, 16, 8, 8, None, 0, 0, 0, None, None, 0, 0, 0, None) == status
    assert lib.specdec_cache_read(None, c, n, b, 16, 16, None) == status
    assert lib.specdec_tree_attention(None, c, n, b, 16, 8, 8, 4, 1.0, 16, 16, 1 << 30, None) == status
    if cache is None or "dtype" not in cache or cache["dtype"] != 2:
        assert lib.specdec_cache_commit(None, c, n, 16, 16, 16, None) == status


def test_rows_are_checked_before_any_device_work(lib):
    c, n = structs(lib)
    f32 = lib.SPECDEC_F32
    good = dict(dtype=lib.SPECDEC_BF16, k=16, k_row_stride=256, k_head_stride=128, v=16, v_row_stride=256,
                v_head_stride=128, q=16, q_row_stride=1024, q_head_stride=128, q_heads=8, out_q=16, rotary=16,
                rotary_dim=128, rotary_positions=9, interleaved=0)

    def append(**kw):
        return lib.specdec_cache_append(None, c, n, *{**good, **kw}.values(), None)

    assert append(dtype=f32) == DTYPE
    for bad in (dict(k=None), dict(k=8), dict(v_row_stride=255), dict(q_head_stride=4), dict(out_q=None), dict(q=None),
                dict(q_heads=0), dict(rotary_dim=24), dict(rotary_dim=144), dict(rotary_dim=0), dict(rotary=4),
                dict(rotary_positions=0)):
        assert append(**bad) == INVALID
    attn = dict(dtype=lib.SPECDEC_BF16, q=16, q_row_stride=1024, q_head_stride=128, q_heads=8, softmax_scale=1.0,
                out=16, workspace=16, workspace_bytes=1 << 30)

    def attend(**kw):
        return lib.specdec_tree_attention(None, c, n, *{**attn, **kw}.values(), None)

    assert attend(dtype=f32) == DTYPE
    for bad in (dict(q_heads=7), dict(q_heads=0), dict(softmax_scale=float("nan")), dict(softmax_scale=float("inf")),
                dict(q=None), dict(out=None), dict(out=8), dict(q_row_stride=4)):
        assert attend(**bad) == INVALID
    assert lib.specdec_cache_read(None, c, n, lib.SPECDEC_BF16, None, 16, None) == INVALID
    assert lib.specdec_cache_commit(None, c, n, None, 16, 16, None) == INVALID
    assert lib.specdec_tree_attention_workspace(None, c, 1, 1, 8, 4) == INVALID
    # good arguments and no handle
    assert append() == INVALID and attend() == INVALID


def test_given_arguments_are_checked(lib):
    assert lib.specdec_rejection_sample_given(None, 16, 8, 16, 8, 16, 16, 16, 16, 1, 8, 4, 16, 16, None) == INVALID


def stub():
    return SimpleNamespace(device=torch.device("cpu"), handle=0, _empty=torch.zeros(4, dtype=torch.int32))


def small_cache(lib, dtype=torch.bfloat16):
    from speculative_decoding_rejection_decode_gb300 import KVCache
    return KVCache.empty(stub(), 4, 16, 2, 64, dtype)


def nodes_of(N=3):
    i = lambda x: torch.tensor(x, dtype=torch.int32)
    return dict(page_table=torch.zeros(2, 3, dtype=torch.int32), lengths=i([0, 5]), cu_num_nodes=i([0, 1, N]))


def test_cache_tensors_are_checked(lib):
    from speculative_decoding_rejection_decode_gb300 import KVCache
    z = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt)
    with pytest.raises(TypeError):
        KVCache(stub(), z(4, 2, 16, 64, dt=torch.float32), z(4, 2, 16, 64, dt=torch.float32))
    with pytest.raises(TypeError):
        KVCache(stub(), z(4, 2, 16, 64), z(4, 2, 16, 64, dt=torch.float16))
    with pytest.raises(ValueError):
        KVCache(stub(), z(4, 2, 16, 96), z(4, 2, 16, 96))
    with pytest.raises(ValueError):
        KVCache(stub(), z(4, 2, 16, 64), z(4, 2, 17, 64))
    with pytest.raises(ValueError):
        KVCache(stub(), z(4, 2, 16, 64).transpose(1, 2), z(4, 2, 16, 64).transpose(1, 2))
    e = torch.zeros(4, 2, 16, 64, dtype=torch.uint8).view(torch.float8_e4m3fn)
    with pytest.raises(ValueError):
        KVCache(stub(), e, e)                                        # no scales
    with pytest.raises(ValueError):
        KVCache(stub(), e, e, torch.ones(4, 2, 16), torch.ones(4, 2, 15))
    with pytest.raises(ValueError):
        KVCache(stub(), z(4, 2, 16, 64), z(4, 2, 16, 64), torch.ones(4, 2, 16), torch.ones(4, 2, 16))


def test_calls_refuse_what_does_not_fit(lib):
    c = small_cache(lib)
    k = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    q = torch.zeros(3, 8, 64, dtype=torch.bfloat16)
    n = nodes_of()
    bad_nodes = [dict(n, lengths=n["lengths"].long()), dict(n, lengths=n["lengths"][:1]),
                 dict(n, cu_num_nodes=n["cu_num_nodes"][:1]), dict(n, page_table=n["page_table"][:1]),
                 dict(n, page_table=torch.zeros(3, 2, dtype=torch.int32).t()),
                 dict(n, node_parent=torch.zeros(2, dtype=torch.int32)),
                 dict(n, page_table=torch.zeros(2, 0, dtype=torch.int32))]
    for kw in bad_nodes:
        with pytest.raises(ValueError):
            c.append(k, k, **kw)
        with pytest.raises(ValueError):
            c.attend(q, **kw)
    for bad in (k[:, :1], k[..., :32], torch.zeros(3, 64, 2, dtype=torch.bfloat16).transpose(1, 2),
                torch.zeros(3 * 2 * 64 + 4, dtype=torch.bfloat16)[4:].view(3, 2, 64)[:, :, :],
                torch.zeros(3, 2, 68, dtype=torch.bfloat16)[..., :64], k.to(torch.float16)):
        with pytest.raises((ValueError, TypeError)):
            c.append(k, bad, **n)
    with pytest.raises(TypeError):
        c.append(k.float(), k.float(), **n)
    with pytest.raises(ValueError):
        c.attend(torch.zeros(3, 7, 64, dtype=torch.bfloat16), **n)           # heads not a multiple
    with pytest.raises(TypeError):
        c.attend(q.to(torch.float16), **n)                                   # another 16-bit type
    with pytest.raises(ValueError):
        c.attend(q, **n, out=torch.zeros(3, 8, 128, dtype=torch.bfloat16)[..., :64])
    for bad in (torch.zeros(9, 2, 4), torch.zeros(9, 2, 40), torch.zeros(9, 32), torch.zeros(9, 2, 32).double()):
        with pytest.raises(ValueError):
            c.append(k, k, **n, rotary=bad)
    with pytest.raises(ValueError):
        c.append(k, k, **n, out_q=q)
    i = lambda x: torch.tensor(x, dtype=torch.int32)
    with pytest.raises(ValueError):
        c.commit(n["page_table"], n["lengths"], n["cu_num_nodes"], i([1]), i([1, 2, -1]))
    with pytest.raises(ValueError):
        c.commit(n["page_table"], n["lengths"], n["cu_num_nodes"], i([1, 1]), i([1, 2, -1]).long())
    with pytest.raises(ValueError):
        c.read(n["page_table"], n["lengths"], n["cu_num_nodes"],
               out=(k, torch.zeros(4, 2, 64, dtype=torch.bfloat16)))


def test_table_rows_and_turned_queries_that_overlap_are_refused(lib):
    c = small_cache(lib)
    n = nodes_of()
    k = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    one = torch.zeros(1, 2, dtype=torch.int32).expand(2, 2)              # every request the same row
    with pytest.raises(ValueError, match="page_table"):
        c.append(k, k, **dict(n, page_table=one))
    wide = torch.zeros(4, 8, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="out_q"):
        c.append(k, k, **n, q=wide[1:], out_q=wide[:3])                  # one row further
    rows = torch.zeros(3, 12, 64, dtype=torch.bfloat16)
    flat = rows.view(-1)[:3 * 8 * 64].view(3, 8, 64)                     # over the rows' own values
    for q, x in ((rows[:, :8], k), (torch.zeros(3, 8, 64, dtype=torch.bfloat16), rows[:, 8:10])):
        with pytest.raises(ValueError, match="out_q"):
            c.append(x, x, **n, q=q, out_q=flat)


def test_sample_given_refuses_what_does_not_fit(lib):
    from speculative_decoding_rejection_decode_gb300 import Verifier
    v = Verifier.__new__(Verifier)
    v.device, v._h, v._empty = torch.device("cpu"), 0, torch.zeros(4, dtype=torch.int32)
    i = lambda x: torch.tensor(x, dtype=torch.int32)
    good = dict(target_probs=torch.rand(5, 8), draft_probs=torch.rand(3, 8), draft_ids=i([1, 2, 3]),
                cu_num_draft_tokens=i([0, 1, 3]), accept_uniforms=torch.rand(3), sample_uniforms=torch.rand(2))
    for kw in (dict(target_probs=torch.rand(4, 8)), dict(target_probs=torch.rand(5, 8).bfloat16()),
               dict(target_probs=torch.rand(8, 5).t()), dict(draft_probs=torch.rand(3, 9)),
               dict(draft_probs=torch.rand(5, 8)), dict(draft_ids=i([1, 2])), dict(draft_ids=torch.tensor([1, 2, 3])),
               dict(accept_uniforms=torch.rand(4)), dict(accept_uniforms=torch.rand(3).double()),
               dict(sample_uniforms=torch.rand(3)), dict(cu_num_draft_tokens=i([0]))):
        with pytest.raises(ValueError):
            v.sample_given(**{**good, **kw})


@pytest.mark.parametrize("dim", [16, 64, 128])
def test_rotary_table_is_the_formula(lib, dim):
    from speculative_decoding_rejection_decode_gb300 import rotary_table
    t = rotary_table(1000, dim, device="cpu")
    assert t.shape == (1000, 2, dim // 2) and t.dtype == torch.float32
    for pos in (0, 1, 7, 999):
        for i in (0, 1, dim // 2 - 1):
            a = pos * 10000.0 ** (-2.0 * i / dim)
            # one rounding to float32 of a 64-bit value
            assert abs(float(t[pos, 0, i]) - math.cos(a)) <= 2.0 ** -24
            assert abs(float(t[pos, 1, i]) - math.sin(a)) <= 2.0 ** -24


def test_rotary_scalings(lib):
    from speculative_decoding_rejection_decode_gb300 import rotary_table
    plain, n = rotary_table(4096, 64, device="cpu"), 4096
    lin = rotary_table(n, 64, scaling="linear", factor=4.0, device="cpu")
    assert torch.allclose(lin[::4][:1000], plain[:1000], atol=1e-6)          # position 4p as p before
    base = rotary_table(n, 64, scaling="base", factor=4.0, device="cpu")
    assert torch.allclose(base[:, :, 0], plain[:, :, 0])                     # the fastest pair stays
    slow = torch.arange(n, dtype=torch.float64) * 10000.0 ** (-62 / 64) / 4.0
    assert torch.allclose(base[:, 0, 31].double(), slow.cos(), atol=1e-6)    # the slowest by the factor
    parts = rotary_table(n, 64, scaling="by_parts", factor=4.0, trained_positions=1024, device="cpu")
    gain = 1 + 0.1 * math.log(4.0)
    assert torch.allclose(parts[:, :, 0], plain[:, :, 0] * gain, atol=1e-6)
    assert torch.allclose(parts[:, 0, 31].double(), slow.cos() * gain, atol=1e-6)
    norm = (parts ** 2).sum(1)
    assert torch.allclose(norm, torch.full_like(norm, gain * gain), atol=1e-5)
    for kw in (dict(scaling="other"), dict(scaling="by_parts", factor=2.0), dict(scaling="linear", factor=0.5)):
        with pytest.raises(ValueError):
            rotary_table(8, 64, device="cpu", **kw)
    with pytest.raises(ValueError):
        rotary_table(8, 63, device="cpu")


def test_reference_rotation_keeps_lengths(lib):
    x = torch.randn(3, 64, dtype=torch.float64)
    freq = [10000.0 ** (-2.0 * i / 32) for i in range(16)]
    for inter in (False, True):
        y = rotate64(x, 17, freq, 1.0, inter)
        assert torch.allclose(y.norm(dim=-1), x.norm(dim=-1)) and torch.equal(y[:, 32:], x[:, 32:])
