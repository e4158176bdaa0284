"""Outputs that lie over inputs: refused before anything is launched."""
import pytest
import torch

from test_cache_host import lib, nodes_of, small_cache  # noqa: F401


def test_lengths_over_other_inputs_are_refused(lib):  # noqa: F811
    c, n = small_cache(lib), nodes_of()
    both = torch.tensor([0, 5, 0, 0, 0, 0, 0, 0], dtype=torch.int32)
    i = lambda x: torch.tensor(x, dtype=torch.int32)
    acc, path = i([0, 1]), i([-1, 1, -1])
    for kw in (dict(lengths=both[:2], out_lengths=both[1:3]), dict(acc=both[:2], out_lengths=both[:2]),
               dict(cu=both[:3], out_lengths=both[2:4]), dict(path=both[:3], out_lengths=both[2:4]),
               dict(table=both[:6].view(2, 3), out_lengths=both[5:7])):
        with pytest.raises(ValueError, match="out_lengths"):
            c.commit(kw.get("table", n["page_table"]), kw.get("lengths", n["lengths"]), kw.get("cu", n["cu_num_nodes"]),
                     kw.get("acc", acc), kw.get("path", path), out_lengths=kw["out_lengths"])


def test_one_tensor_for_keys_and_values_is_refused(lib):  # noqa: F811
    c, n = small_cache(lib), nodes_of()
    x = torch.zeros(6, 2, 64, dtype=torch.bfloat16)
    for out in ((x[:3], x[:3]), (x[:3], x[2:5])):
        with pytest.raises(ValueError, match="of their own"):
            c.read(n["page_table"], n["lengths"], n["cu_num_nodes"], out=out)
