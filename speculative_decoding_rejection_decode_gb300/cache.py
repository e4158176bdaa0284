"""The paged key/value cache around the verification of drafted nodes, and the
cos / sin tables of rotary positions: argument marshalling only (every step runs
in the library's CUDA kernels)."""
from __future__ import annotations

import ctypes
import math

import torch

from ._lib import (SPECDEC_BF16, SPECDEC_E4M3, SPECDEC_F16, specdec_cache_append,  # noqa: F401
                   specdec_cache_append_positions, specdec_cache_commit, specdec_cache_read,
                   specdec_cache_t, specdec_cross_attention, specdec_cross_attention_workspace,
                   specdec_nodes_t, specdec_tree_attention, specdec_tree_attention_workspace)
from .verifier import Verifier, _check, _ptr, _overlap, _stream_handle, position_args, rotary_axes  # noqa: F401

_DTYPE = {torch.bfloat16: SPECDEC_BF16, torch.float16: SPECDEC_F16,
          torch.float8_e4m3fn: SPECDEC_E4M3}


def rotary_table(positions: int, rotary_dim: int, *, base: float = 10000.0,
                 scaling: str | None = None, factor: float = 1.0, trained_positions: int = 0,
                 fast_turns: float = 32.0, slow_turns: float = 1.0,
                 device="cuda") -> torch.Tensor:
    """cos and sin of position * base^(-2i / rotary_dim), float32 [positions, 2,
    rotary_dim / 2], computed in 64 bits (angles of far positions lose their
    fraction in 32).  ``scaling`` stretches a model trained on
    ``trained_positions`` to ``factor`` times as many:
      "linear"   every angle divided by factor
      "base"     base * factor^(rotary_dim / (rotary_dim - 2)): the slowest pair
                 is stretched by factor, the fastest not at all
      "by_parts" the YaRN method (Peng et al. 2023): pairs that turn at least
                 ``fast_turns`` times over trained_positions keep their angle,
                 pairs that turn at most ``slow_turns`` times are divided by
                 factor, with a linear ramp over the pair index between (its ends
                 on whole pairs, rounded outward); cos and sin are multiplied by
                 1 + 0.1 ln(factor), which sharpens the softmax"""
    if positions < 1 or rotary_dim < 2 or rotary_dim % 2 or not factor >= 1.0 or not base > 1.0:
        raise ValueError("need positions >= 1, an even rotary_dim, factor >= 1 and base > 1")
    i = torch.arange(rotary_dim // 2, dtype=torch.float64, device=device)
    gain = 1.0
    if scaling == "base":
        if rotary_dim < 4:
            raise ValueError("scaling \"base\" needs rotary_dim >= 4")
        base = base * factor ** (rotary_dim / (rotary_dim - 2))
    freq = base ** (-2.0 * i / rotary_dim)
    if scaling == "linear":
        freq = freq / factor
    elif scaling == "by_parts":
        if trained_positions < 1 or not fast_turns > slow_turns > 0:
            raise ValueError("scaling \"by_parts\" needs trained_positions and fast_turns > slow_turns > 0")

        def pair_of(turns):    # pair index whose angle passes `turns` circles
            return rotary_dim * math.log(trained_positions / (turns * 2 * math.pi)) / (2 * math.log(base))

        # more turns lie at a smaller pair index, so lo < hi; either may lie beyond the
        # pairs there are, which then all stand on the ramp or beside it
        lo, hi = math.floor(pair_of(fast_turns)), math.ceil(pair_of(slow_turns))
        kept = 1.0 - ((i - lo) / (hi - lo)).clamp(0.0, 1.0)
        freq = freq * kept + freq / factor * (1.0 - kept)
        gain = 1.0 + 0.1 * math.log(factor)
    elif scaling not in (None, "base"):
        raise ValueError("scaling must be None, \"linear\", \"base\" or \"by_parts\"")
    a = torch.arange(positions, dtype=torch.float64, device=device)[:, None] * freq
    out = torch.empty(positions, 2, rotary_dim // 2, dtype=torch.float32, device=device)
    out[:, 0] = a.cos() * gain
    out[:, 1] = a.sin() * gain
    return out


class KVCache:
    """Keys and values of one layer in pages, over a Verifier's handle.

    ``k``, ``v``: [num_pages, num_kv_heads, page_size, head_dim], bfloat16,
    float16 or float8_e4m3fn (then with ``k_scale``, ``v_scale``: float32
    [num_pages, num_kv_heads, page_size]); head_dim 64 or 128.  The tensors stay
    the caller's; ``KVCache.empty`` allocates them.

    Every call takes the page table (int32 [B, max_pages]), the requests'
    filled slots ``lengths`` (int32 [B]) and the nodes' layout of
    ``Verifier.tree``: ``cu_num_nodes`` (int32 [B + 1]) and ``node_parent``
    (int32 [N], or None for chains).  Work is queued on the current torch stream
    of the cache's device; what only the device can see (a bad page, length or
    tree) sets the verifier's error word (``Verifier.get_error``)."""

    def __init__(self, verifier: Verifier, k: torch.Tensor, v: torch.Tensor,
                 k_scale: torch.Tensor | None = None, v_scale: torch.Tensor | None = None):
        if k.dtype not in _DTYPE or v.dtype != k.dtype:
            raise TypeError("k and v must both be bfloat16, float16 or float8_e4m3fn")
        if k.dim() != 4 or v.shape != k.shape or not k.is_contiguous() or not v.is_contiguous():
            raise ValueError("k and v must be contiguous [num_pages, num_kv_heads, page_size, head_dim]")
        fp8 = k.dtype == torch.float8_e4m3fn
        for t in (k_scale, v_scale):
            if fp8 and (t is None or t.dtype != torch.float32 or t.shape != k.shape[:3]
                        or not t.is_contiguous() or t.device != k.device):
                raise ValueError("an 8-bit cache needs contiguous float32 scales [num_pages, "
                                 "num_kv_heads, page_size] on the device")
            if not fp8 and t is not None:
                raise ValueError("a 16-bit cache has no scales")
        if k.device != verifier.device or v.device != verifier.device:
            raise ValueError("the cache must be on the verifier's device")
        if k.shape[3] not in (64, 128):
            raise ValueError("head_dim must be 64 or 128")
        self.verifier, self.k, self.v, self.k_scale, self.v_scale = verifier, k, v, k_scale, v_scale
        self.device, self.dtype, self._at = k.device, k.dtype, k.get_device()
        self.num_pages, self.num_kv_heads, self.page_size, self.head_dim = k.shape
        self._c = specdec_cache_t(_ptr(k), _ptr(v), _ptr(k_scale) or None, _ptr(v_scale) or None,
                                  _DTYPE[k.dtype], self.num_kv_heads, self.head_dim,
                                  self.page_size, self.num_pages)
        self._ref = ctypes.byref(self._c)

    @classmethod
    def empty(cls, verifier: Verifier, num_pages: int, page_size: int, num_kv_heads: int,
              head_dim: int, dtype: torch.dtype = torch.bfloat16) -> "KVCache":
        """A cache of zeros."""
        shape, dev = (num_pages, num_kv_heads, page_size, head_dim), verifier.device
        if dtype != torch.float8_e4m3fn:
            return cls(verifier, torch.zeros(shape, dtype=dtype, device=dev),
                       torch.zeros(shape, dtype=dtype, device=dev))
        return cls(verifier, *(torch.zeros(shape, dtype=torch.uint8, device=dev).view(dtype)
                               for _ in range(2)),
                   *(torch.ones(shape[:3], dtype=torch.float32, device=dev) for _ in range(2)))

    def _nodes(self, page_table, lengths, cu, parent, N):
        i32, at, B = torch.int32, self._at, cu.numel() - 1
        if B < 1 or lengths.numel() != B:
            raise ValueError("need cu of B + 1 >= 2 entries and B lengths")
        if page_table.dtype is not i32 or lengths.dtype is not i32 or cu.dtype is not i32 \
                or page_table.get_device() != at or lengths.get_device() != at or cu.get_device() != at:
            raise ValueError("page_table, lengths and cu must be int32 tensors on the device")
        if not lengths.is_contiguous() or not cu.is_contiguous():
            raise ValueError("lengths and cu must be contiguous")
        if parent is not None and (parent.dtype is not i32 or parent.get_device() != at
                                   or parent.numel() != N or not parent.is_contiguous()):
            raise ValueError("node_parent must be a contiguous int32 tensor on the device, one entry per row")
        if page_table.dim() != 2 or page_table.shape[0] != B:
            raise ValueError("page_table must be [B, max_pages]")
        most, (row, one) = page_table.shape[1], page_table.stride()
        if most < 1 or (most > 1 and one != 1) or (B > 1 and row < most):
            raise ValueError("page_table must be [B, max_pages] with contiguous rows of their own")
        return ctypes.byref(specdec_nodes_t(page_table.data_ptr(), max(row, most), most, lengths.data_ptr(),
                                            cu.data_ptr(), None if parent is None else parent.data_ptr() or None,
                                            B, N))

    def _rows(self, t, N, heads, dtype, name):
        """Data pointer and strides of rows [N, heads, head_dim]."""
        if t.shape != (N, heads, self.head_dim):
            raise ValueError(f"{name} must be [{N}, {heads}, {self.head_dim}]")
        if t.dtype is not dtype or t.get_device() != self._at:
            raise ValueError(f"{name} must be {dtype} on the device")
        row, head, one = t.stride()
        at = t.data_ptr()
        if one != 1 or row % 8 or head % 8 or at % 16:
            raise ValueError(f"{name} needs contiguous values, 16-byte aligned rows and strides of "
                             "multiples of 8")
        return at, row, head

    def _row_dtype(self, t):
        if t.dtype not in (torch.bfloat16, torch.float16) or (self.dtype != torch.float8_e4m3fn
                                                              and t.dtype != self.dtype):
            raise TypeError("rows must be bfloat16 or float16, and of a 16-bit cache's own type")
        return _DTYPE[t.dtype]

    def append(self, k: torch.Tensor, v: torch.Tensor, page_table: torch.Tensor,
               lengths: torch.Tensor, cu_num_nodes: torch.Tensor,
               node_parent: torch.Tensor | None = None, *, q: torch.Tensor | None = None,
               rotary: torch.Tensor | None = None, interleaved: bool = False,
               positions: torch.Tensor | None = None, axes=None,
               position_offsets: torch.Tensor | None = None,
               out_q: torch.Tensor | None = None) -> torch.Tensor | None:
        """Writes the nodes' keys and values ([N, num_kv_heads, head_dim], any row
        and head strides) behind the context: node j of request b into slot
        lengths[b] + j.  With ``rotary`` (``rotary_table``) k and q are turned to
        position lengths[b] + depth(j) first, in pairs (i, i + rotary_dim / 2) or,
        interleaved, (2i, 2i + 1).  Where positions are not slot numbers (images, videos),
        ``positions`` gives the rows' own (int32 [N], or [axes, N] with ``axes``, the
        axis of each pair: ``rotary_axes``), or ``position_offsets`` (int32 [B]) what
        each request adds to lengths[b] + depth(j).  Returns the turned q (contiguous;
        ``out_q`` may be q itself), or None."""
        N = k.shape[0]
        dt = self._row_dtype(k)
        kp = self._rows(k, N, self.num_kv_heads, k.dtype, "k")
        vp = self._rows(v, N, self.num_kv_heads, k.dtype, "v")
        qp, heads = (None, 0, 0), 0
        if q is not None:
            heads = q.shape[1] if q.dim() == 3 else 0
            qp = self._rows(q, N, heads, k.dtype, "q")
            if out_q is None:
                out_q = torch.empty(N, heads, self.head_dim, dtype=k.dtype, device=self.device)
            elif out_q.shape != q.shape or out_q.dtype != k.dtype or out_q.device != self.device \
                    or not out_q.is_contiguous():
                raise ValueError("out_q must be contiguous and like q")
            elif N and ((_overlap(out_q, q) and not (out_q.data_ptr() == q.data_ptr() and q.is_contiguous()))
                        or _overlap(out_q, k) or _overlap(out_q, v)):
                raise ValueError("out_q must be q itself or overlap none of q, k and v")
        elif out_q is not None:
            raise ValueError("out_q without q")
        dim = positions_held = 0
        if rotary is not None:
            if rotary.dim() != 3 or rotary.shape[1] != 2 or rotary.dtype != torch.float32 \
                    or rotary.device != self.device or not rotary.is_contiguous():
                raise ValueError("rotary must be contiguous float32 [positions, 2, rotary_dim / 2] "
                                 "on the device")
            positions_held, dim = rotary.shape[0], 2 * rotary.shape[2]
            if dim % 16 or not 0 < dim <= self.head_dim:
                raise ValueError("rotary_dim must be a multiple of 16 up to head_dim")
        elif positions is not None or position_offsets is not None:
            raise ValueError("positions without rotary")
        if axes is not None and positions is None:
            raise ValueError("axes without positions")
        nodes = self._nodes(page_table, lengths, cu_num_nodes, node_parent, N)
        if positions is not None or position_offsets is not None:
            if positions is not None and position_offsets is not None:
                raise ValueError("positions and position_offsets exclude each other")
            if positions is not None:
                where = (*position_args(positions, axes, N, dim // 2, self._at), None)
                if N and q is not None and _overlap(out_q, positions):
                    raise ValueError("out_q must not overlap positions")
            else:
                t = position_offsets
                if t.dtype is not torch.int32 or t.get_device() != self._at or t.numel() != lengths.numel() \
                        or not t.is_contiguous():
                    raise ValueError("position_offsets must be a contiguous int32 tensor on the device, one entry per request")
                if N and q is not None and _overlap(out_q, t):
                    raise ValueError("out_q must not overlap position_offsets")
                where = (None, 0, 1, None, t.data_ptr())
            if N:
                _check(specdec_cache_append_positions(
                    self.verifier.handle, self._ref, nodes, dt, *kp, *vp, *qp, heads,
                    None if q is None else out_q.data_ptr(), rotary.data_ptr(), dim, positions_held,
                    int(interleaved), *where, _stream_handle(self.device)), "specdec_cache_append_positions")
            return out_q
        if N:
            _check(specdec_cache_append(self.verifier.handle, self._ref, nodes, dt, *kp, *vp, *qp, heads,
                                        None if q is None else out_q.data_ptr(), _ptr(rotary) or None,
                                        dim, positions_held, int(interleaved), _stream_handle(self.device)),
                   "specdec_cache_append")
        return out_q

    def read(self, page_table: torch.Tensor, starts: torch.Tensor, cu_rows: torch.Tensor, *,
             n_rows: int | None = None, dtype: torch.dtype | None = None,
             out: tuple[torch.Tensor, torch.Tensor] | None = None) -> tuple[torch.Tensor, torch.Tensor]:
        """Rows read back as dense 16-bit tensors (k, v), [n_rows, num_kv_heads,
        head_dim]: request b's rows cu_rows[b] .. cu_rows[b + 1] - 1 are its slots
        starts[b], starts[b] + 1, ...  ``n_rows`` (= cu_rows[B]) avoids a host read;
        ``dtype`` defaults to the cache's own, bfloat16 for 8 bits."""
        if out is None:
            N = int(cu_rows[-1]) if n_rows is None else int(n_rows)
            dtype = dtype or (torch.bfloat16 if self.dtype == torch.float8_e4m3fn else self.dtype)
            shape = (N, self.num_kv_heads, self.head_dim)
            out = (torch.empty(shape, dtype=dtype, device=self.device),
                   torch.empty(shape, dtype=dtype, device=self.device))
        elif out[0].numel() and _overlap(*out):
            raise ValueError("out must be two tensors of their own")
        N = out[0].shape[0]
        for t in out:
            if t.shape != (N, self.num_kv_heads, self.head_dim) or t.dtype != out[0].dtype \
                    or t.device != self.device or not t.is_contiguous():
                raise ValueError("out must be two contiguous [n_rows, num_kv_heads, head_dim] tensors")
        dt = self._row_dtype(out[0])
        nodes = self._nodes(page_table, starts, cu_rows, None, N)
        if N:
            _check(specdec_cache_read(self.verifier.handle, self._ref, nodes, dt, out[0].data_ptr(),
                                      out[1].data_ptr(), _stream_handle(self.device)),
                   "specdec_cache_read")
        return out

    def _attention(self, q, page_table, lengths, cu, parent, mask, scale, out, ask, call, name):
        N, heads = q.shape[0], q.shape[1] if q.dim() == 3 else 0
        dt = self._row_dtype(q)
        qp = self._rows(q, N, heads, q.dtype, "q")
        if heads < 1 or heads % self.num_kv_heads:
            raise ValueError("q_heads must be a multiple of num_kv_heads")
        nodes = self._nodes(page_table, lengths, cu, parent, N)
        if out is None:
            out = torch.empty(N, heads, self.head_dim, dtype=q.dtype, device=self.device)
        elif out.shape != q.shape or out.dtype != q.dtype or out.device != self.device \
                or not out.is_contiguous():
            raise ValueError("out must be contiguous and like q")
        elif N and out.untyped_storage().data_ptr() == q.untyped_storage().data_ptr() \
                and _overlap(out, q):
            raise ValueError("out must not overlap q")
        if N:
            h = self.verifier.handle
            need = ask(h, self._ref, cu.numel() - 1, N, heads, page_table.shape[1])
            if need < 0:
                _check(need, name + "_workspace")
            ws = torch.empty(need, dtype=torch.uint8, device=self.device) if need else None
            _check(call(h, self._ref, nodes, dt, *qp, heads, *mask,
                        self.head_dim ** -0.5 if scale is None else float(scale), out.data_ptr(),
                        _ptr(ws) or None, need, _stream_handle(self.device)), name)
        return out

    def attend(self, q: torch.Tensor, page_table: torch.Tensor, lengths: torch.Tensor,
               cu_num_nodes: torch.Tensor, node_parent: torch.Tensor | None = None, *,
               scale: float | None = None, out: torch.Tensor | None = None) -> torch.Tensor:
        """Attention of the nodes' queries ([N, q_heads, head_dim], q_heads a
        multiple of num_kv_heads) over their request's context and their own
        ancestors, which ``append`` has written: specdec_tree_attention.  ``scale``
        defaults to 1 / sqrt(head_dim).  Returns [N, q_heads, head_dim]."""
        return self._attention(q, page_table, lengths, cu_num_nodes, node_parent, (), scale, out,
                               specdec_tree_attention_workspace, specdec_tree_attention,
                               "specdec_tree_attention")

    def cross_attend(self, q: torch.Tensor, page_table: torch.Tensor, lengths: torch.Tensor,
                     cu_rows: torch.Tensor, *, mask: torch.Tensor | None = None,
                     scale: float | None = None, out: torch.Tensor | None = None) -> torch.Tensor:
        """Cross attention: every row of q ([N, q_heads, head_dim], request b's rows
        cu_rows[b] .. cu_rows[b + 1] - 1) over its request's slots 0 .. lengths[b] - 1,
        an encoder's states that ``append`` has written once, and no others:
        specdec_cross_attention.  States held as [B, num_kv_heads, most, head_dim] are a
        cache of B pages with the page table arange(B)[:, None].  ``mask`` (bool or uint8
        [B, slots]): slots where it is 0, or behind its columns, are hidden.  A row
        that sees no state is zeros."""
        m = (None, 0, 0)
        if mask is not None:
            if mask.dtype not in (torch.bool, torch.uint8) or mask.get_device() != self._at or mask.dim() != 2 \
                    or mask.shape[0] != lengths.numel() or (mask.shape[1] > 1 and mask.stride(1) != 1) \
                    or (mask.shape[0] > 1 and mask.stride(0) < mask.shape[1]):
                raise ValueError("mask must be bool or uint8 [B, slots] on the device with contiguous rows of their own")
            # a mask without columns hides everything; it still needs an address
            m = (mask.data_ptr() or self.verifier._empty.data_ptr(), max(mask.stride(0), mask.shape[1]), mask.shape[1])
            if out is not None and _overlap(out, mask):
                raise ValueError("out must not overlap mask")
        return self._attention(q, page_table, lengths, cu_rows, None, m, scale, out,
                               specdec_cross_attention_workspace, specdec_cross_attention,
                               "specdec_cross_attention")

    def commit(self, page_table: torch.Tensor, lengths: torch.Tensor, cu_num_nodes: torch.Tensor,
               num_accepted: torch.Tensor, path: torch.Tensor | None = None, *,
               out_lengths: torch.Tensor | None = None) -> torch.Tensor:
        """After the verification: moves the accepted nodes' rows behind the root
        (``path`` as ``Verifier.tree`` reports it; None for chains) and returns the
        new lengths, lengths + 1 + num_accepted (``out_lengths`` may be
        ``lengths`` itself)."""
        B, dev = cu_num_nodes.numel() - 1, self.device
        given = out_lengths is not None
        if not given:
            out_lengths = torch.empty(B, dtype=torch.int32, device=dev)
        for t, n, name in ((num_accepted, B, "num_accepted"), (out_lengths, B, "out_lengths"),
                           (path, None, "path")):
            if t is not None and (t.dtype != torch.int32 or t.device != dev or not t.is_contiguous()
                                  or (n is not None and t.numel() != n)):
                raise ValueError(f"{name} must be a contiguous int32 tensor on the device")
        if given and out_lengths.data_ptr() != lengths.data_ptr() and any(
                t is not None and t.numel() and _overlap(out_lengths, t)
                for t in (lengths, num_accepted, cu_num_nodes, path, page_table)):
            raise ValueError("out_lengths must be lengths itself or overlap none of the inputs")
        # without a path nothing but the lengths changes; any N bounds cu then
        N = (1 << 31) - 1 if path is None else path.numel()
        nodes = self._nodes(page_table, lengths, cu_num_nodes, None, N)
        _check(specdec_cache_commit(self.verifier.handle, self._ref, nodes, num_accepted.data_ptr(),
                                    None if path is None else (path.data_ptr() or self.verifier._empty.data_ptr()),
                                    out_lengths.data_ptr(), _stream_handle(dev)), "specdec_cache_commit")
        return out_lengths
