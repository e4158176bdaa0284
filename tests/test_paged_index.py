"""The index arithmetic that the cache's kernels share (csrc/paged_index.h),
compiled for the host: no GPU needed to see that every access stays in bounds."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "speculative_decoding_rejection_decode_gb300", "csrc")

SHIM = r"""
#include "paged_index.h"
using namespace specdec;
extern "C" {
int t_node_range(const int32_t* cu, int b, int64_t N, int64_t* first, int32_t* count) {
  return node_range(cu, b, N, *first, *count);
}
int t_request_of_row(const int32_t* cu, int B, int64_t r) { return request_of_row(cu, B, r); }
int64_t t_cache_row(int64_t pages, int kv_heads, int page_size, int max_pages, const int32_t* table, int64_t slot) {
  PagedGeo g = {pages, max_pages, kv_heads, page_size, max_pages};
  return cache_row(g, table, slot);
}
int t_node_depth(const int32_t* parent, int j) { return node_depth(parent, j); }
int64_t t_range_begin(int64_t units, int G, int i) { return range_begin(units, G, i); }
int t_range_of(int64_t units, int G, int64_t u) { return range_of(units, G, u); }
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("paged")
    src, so = d / "shim.cpp", d / "shim.so"
    src.write_text(SHIM)
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-I", CSRC, str(src), "-o", str(so)],
                   check=True)
    lib = ctypes.CDLL(str(so))
    for name in ("t_cache_row", "t_range_begin"):
        getattr(lib, name).restype = ctypes.c_int64
    return lib


def ptr(a):
    return a.ctypes.data_as(ctypes.POINTER(ctypes.c_int32))


def i64(x):
    return ctypes.c_int64(int(x))


@pytest.mark.parametrize("counts", [[1], [3, 0, 2], [0, 0, 5], [4, 0], [0], [1] * 33])
def test_request_of_row(lib, counts):
    cu = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    owner = [b for b, n in enumerate(counts) for _ in range(n)]
    for r in range(int(cu[-1]) + 3):
        want = owner[r] if r < len(owner) else -1
        assert lib.t_request_of_row(ptr(cu), len(counts), i64(r)) == want


@pytest.mark.parametrize("cu", [[0, 5, 3, 8], [2, 4], [0, -1, 4], [7, 7, 7], [0, 1 << 30, 4]])
def test_request_of_row_ends_on_a_malformed_cu(lib, cu):
    cu = np.array(cu, np.int32)
    for r in range(12):
        b = lib.t_request_of_row(ptr(cu), len(cu) - 1, i64(r))
        assert b == -1 or (cu[b] <= r < cu[b + 1])


def test_node_range_refuses_what_is_no_range(lib):
    first, count = ctypes.c_int64(), ctypes.c_int32()

    def of(cu, b, N):
        cu = np.array(cu, np.int32)
        ok = lib.t_node_range(ptr(cu), b, i64(N), ctypes.byref(first), ctypes.byref(count))
        return (first.value, count.value) if ok else None

    assert of([0, 3, 5], 1, 5) == (3, 2)
    assert of([0, 3, 3], 1, 3) == (3, 0)
    assert of([0, 3, 5], 1, 4) is None      # passes the rows given
    assert of([0, 3, 2], 1, 9) is None      # decreases
    assert of([-1, 3], 0, 9) is None


def test_cache_row_stays_inside_the_cache(lib):
    kv, page, pages, most = 3, 5, 4, 3
    table = np.array([2, 0, 3], np.int32)
    for slot in range(-3, 40):
        got = lib.t_cache_row(i64(pages), kv, page, most, ptr(table), i64(slot))
        if 0 <= slot < most * page:
            assert got == table[slot // page] * kv * page + slot % page
            assert got + (kv - 1) * page < pages * kv * page
        else:
            assert got == -1
    for bad in (-1, 4, 2 ** 31 - 1, -2 ** 31):
        t = np.array([bad], np.int32)
        assert lib.t_cache_row(i64(pages), kv, page, 1, ptr(t), i64(2)) == -1


def test_cache_row_passes_32_bits(lib):
    t = np.array([2 ** 24], np.int32)
    got = lib.t_cache_row(i64(2 ** 24 + 1), 8, 64, 1, ptr(t), i64(63))
    assert got == 2 ** 24 * 512 + 63


def test_node_depth(lib):
    par = np.array([-1, 0, 0, 1, 3, 2], np.int32)
    assert [lib.t_node_depth(ptr(par), j) for j in range(6)] == [0, 1, 1, 2, 3, 2]
    assert lib.t_node_depth(None, 7) == 7
    for bad in ([-1, 1], [-1, 2, 0], [-1, -1], [-1, 0, -7]):
        par = np.array(bad, np.int32)
        assert lib.t_node_depth(ptr(par), len(bad) - 1) in (-1, 1)
    assert lib.t_node_depth(ptr(np.array([-1, 1], np.int32)), 1) == -1      # its own parent
    assert lib.t_node_depth(ptr(np.array([-1, -1], np.int32)), 1) == -1     # a second root


@pytest.mark.parametrize("G", [1, 3, 152, 304])
def test_ranges_cover_every_unit_once(lib, G):
    for units in [G, G + 1, 5 * G - 1, 1000 * G + 7, 2 ** 45 + 12345]:
        begins = [lib.t_range_begin(i64(units), G, i) for i in range(G + 1)]
        assert begins[0] == 0 and begins[-1] == units
        sizes = np.diff(begins)
        assert sizes.min() >= units // G and sizes.max() <= units // G + 1
        for i in range(0, G, max(1, G // 7)):
            for u in (begins[i], begins[i + 1] - 1):
                assert lib.t_range_of(i64(units), G, i64(u)) == i
