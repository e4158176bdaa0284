"""Torch-facing wrapper of libspecdec.so: argument marshalling only (every
step of the verifier runs in the library's CUDA kernels)."""
from __future__ import annotations

from dataclasses import dataclass

import torch

from . import _lib
from ._lib import (SPECDEC_BF16, SPECDEC_F16, SPECDEC_F32, SPECDEC_MAX_AXES, SPECDEC_MAX_TOP, SPECDEC_PATH_AUTO, SPECDEC_PATH_DUAL,  # noqa: F401
                   SPECDEC_PATH_FUSED, SPECDEC_PATH_GREEDY, SPECDEC_PATH_PAIR, SPECDEC_PATH_STREAM, SPECDEC_PATH_SWEEP,
                   SPECDEC_PATH_TWO_PASS, specdec_create, specdec_destroy,
                   specdec_get_error, specdec_last_path, specdec_logprobs,
                   specdec_logprobs_grad, specdec_neg_log_uniform, specdec_rotate,
                   specdec_selection_mass,
                   specdec_rejection_sample, specdec_rejection_sample_ex,
                   specdec_rejection_sample_given, specdec_rejection_sample_noalloc,
                   specdec_rejection_sample_topk_topp,
                   specdec_reserve, specdec_set_adjust_counters,
                   specdec_set_path, specdec_set_timing_events, specdec_status_string,
                   specdec_tree_verify, specdec_uniform)


class SpecdecError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        super().__init__(f"{what}: {specdec_status_string(status)} ({status})")
        self.status = status


def _check(rc: int, what: str):
    if rc != 0:
        raise SpecdecError(rc, what)


@dataclass
class VerifyOutput:
    tokens: torch.Tensor         # int32 [N_t]
    num_accepted: torch.Tensor   # int32 [B]
    beta: torch.Tensor | None    # float32 [N_d]
    target_prob: torch.Tensor | None = None   # float32 [N_d] p_i(x_i)
    draft_prob: torch.Tensor | None = None    # float32 [N_d] q_i(x_i)
    accept: torch.Tensor | None = None        # int32 [N_d]


@dataclass
class LogprobOutput:
    logprob: torch.Tensor | None        # float32 [M] ln p(id); None without ids
    entropy: torch.Tensor               # float32 [M]
    top_ids: torch.Tensor | None        # int32 [M, top]; None where top is 0
    top_logprobs: torch.Tensor | None   # float32 [M, top]
    stats: torch.Tensor                 # float32 [M, 2] what the gradient needs of the rows
    own_rows: bool = True               # token t's row is t (no `rows` were given): what the gradient takes


_LOGITS = {torch.float32: SPECDEC_F32, torch.bfloat16: SPECDEC_BF16, torch.float16: SPECDEC_F16}


def _overlap(a: torch.Tensor, b: torch.Tensor) -> bool:
    """Whether the spans of memory of two tensors meet."""
    def span(t):
        last = sum((n - 1) * s for n, s in zip(t.shape, t.stride()))
        return t.data_ptr(), t.data_ptr() + (last + 1) * t.element_size()
    if not a.numel() or not b.numel():
        return False
    (a0, a1), (b0, b1) = span(a), span(b)
    return a0 < b1 and b0 < a1


def _ptr(t):
    return 0 if t is None else t.data_ptr()


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)   # a tenth of the call below


def _stream_handle(device) -> int:
    if _raw_stream is not None and device.index is not None:
        return _raw_stream(device.index)
    return torch.cuda.current_stream(device).cuda_stream


class Verifier:
    """One library handle on one CUDA device."""

    def __init__(self, device: int | torch.device = 0):
        dev = torch.device("cuda", device) if isinstance(device, int) else torch.device(device)
        if dev.type != "cuda":
            raise ValueError("the verifier runs on a CUDA device")
        self.device = dev
        idx = dev.index if dev.index is not None else torch.cuda.current_device()
        rc, self._h = specdec_create(idx)
        _check(rc, "specdec_create")
        self._at = idx
        # a valid device address for required arrays that are empty (draft_ids
        # when every request has gamma = 0): the C ABI wants a pointer even then
        self._empty = torch.zeros(4, dtype=torch.int32, device=dev)

    def _ids_ptr(self, draft_ids) -> int:
        if draft_ids is not None and draft_ids.numel() == 0:
            return self._empty.data_ptr()
        return _ptr(draft_ids)

    def close(self):
        if getattr(self, "_h", 0):
            specdec_destroy(self._h)
            self._h = 0

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    @property
    def handle(self) -> int:
        return self._h

    def reserve(self, max_draft_positions: int, max_batch: int):
        _check(specdec_reserve(self._h, max_draft_positions, max_batch), "specdec_reserve")

    def set_timing_events(self, before_rows, after_rows):
        """torch.cuda.Event pair (already recorded once, so that the CUDA event
        exists) recorded around the row kernel of every later call; None, None
        to stop."""
        a = None if before_rows is None else before_rows.cuda_event
        b = None if after_rows is None else after_rows.cuda_event
        _check(specdec_set_timing_events(self._h, a, b), "specdec_set_timing_events")

    def set_adjust_counters(self, counters: torch.Tensor | None):
        """int64 [8] device tensor that later calls add their top-k / top-p
        selection statistics to (see specdec_set_adjust_counters); None stops."""
        if counters is not None and (counters.device != self.device or counters.dtype != torch.int64
                                     or counters.numel() < 8):
            raise ValueError("counters must be an int64 tensor of 8 entries on the device")
        _check(specdec_set_adjust_counters(self._h, _ptr(counters)), "specdec_set_adjust_counters")

    def set_path(self, path: int):
        _check(specdec_set_path(self._h, path), "specdec_set_path")

    def last_path(self) -> tuple[int, int]:
        rc, p, c = specdec_last_path(self._h)
        _check(rc, "specdec_last_path")
        return p, c

    def get_error(self) -> int:
        rc, e = specdec_get_error(self._h, _stream_handle(self.device))
        _check(rc, "specdec_get_error")
        return e

    def tree(self, target_logits: torch.Tensor, draft_probs: torch.Tensor | None,
             node_tokens: torch.Tensor, node_parent: torch.Tensor, cu_num_nodes: torch.Tensor,
             T: float, seed: int, *, request_offset: int = 0, with_path: bool = True,
             out: "TreeOutput | None" = None) -> "TreeOutput":
        """Verifies token trees (several candidates per position) on the current
        torch stream: specdec_tree_verify.  One target and one draft row per
        node; node_parent holds indices within each request (node 0: -1)."""
        return _tree_call(self, target_logits, draft_probs, node_tokens, node_parent,
                          cu_num_nodes, T, seed, request_offset, with_path, out)

    def sample_given(self, target_probs: torch.Tensor, draft_probs: torch.Tensor | None,
                     draft_ids: torch.Tensor, cu_num_draft_tokens: torch.Tensor,
                     accept_uniforms: torch.Tensor, sample_uniforms: torch.Tensor, *,
                     out: VerifyOutput | None = None) -> VerifyOutput:
        """Verifies drafted chains from probabilities (float32 rows, no logits) and
        given random numbers on the current torch stream:
        specdec_rejection_sample_given.  ``accept_uniforms`` [N_d] and
        ``sample_uniforms`` [B] are float32 in [0, 1); probability rows may lie
        further apart than V; ``draft_probs`` None is a one-hot drafter.  beta is
        not computed (None)."""
        dev, i32, f32 = self.device, torch.int32, torch.float32
        B, nd = cu_num_draft_tokens.numel() - 1, draft_ids.numel()
        for t, dt, n, name in ((draft_ids, i32, nd, "draft_ids"),
                               (cu_num_draft_tokens, i32, max(B, 1) + 1, "cu_num_draft_tokens"),
                               (accept_uniforms, f32, nd, "accept_uniforms"),
                               (sample_uniforms, f32, B, "sample_uniforms")):
            if t.dtype is not dt or t.device != dev or t.numel() != n or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous {dt} tensor of {n} entries on the device")
        V = target_probs.shape[-1]
        for t, rows, name in ((target_probs, nd + B, "target_probs"), (draft_probs, nd, "draft_probs")):
            if t is not None and (t.dtype is not f32 or t.device != dev or t.shape != (rows, V)
                                  or (V > 1 and t.stride(1) != 1) or (rows > 1 and t.stride(0) < V)):
                raise ValueError(f"{name} must be float32 rows [{rows}, {V}] on the device")
        if out is None:
            out = VerifyOutput(torch.empty(nd + B, dtype=i32, device=dev),
                               torch.empty(B, dtype=i32, device=dev), None)
        else:
            for t, n in ((out.tokens, nd + B), (out.num_accepted, B)):
                if t.device != dev or t.dtype is not i32 or t.numel() != n or not t.is_contiguous():
                    raise ValueError("out must hold contiguous int32 tokens [N_t] and num_accepted [B]")
        # with no draft rows at all an empty tensor still means "rows given"
        q = None if draft_probs is None else (_ptr(draft_probs) or self._empty.data_ptr())
        rc = specdec_rejection_sample_given(
            self._h, _ptr(target_probs), max(target_probs.stride(0), V), q,
            V if draft_probs is None else max(draft_probs.stride(0), V), self._ids_ptr(draft_ids),
            _ptr(cu_num_draft_tokens), _ptr(accept_uniforms) or None, _ptr(sample_uniforms), B, V,
            nd, _ptr(out.tokens), _ptr(out.num_accepted), _stream_handle(dev))
        _check(rc, "specdec_rejection_sample_given")
        return out

    def _logit_rows(self, t, name):
        """Data pointer, type and row stride of rows of logits [R, V]."""
        if t.dim() != 2 or t.dtype not in _LOGITS or t.get_device() != self._at \
                or (t.shape[1] > 1 and t.stride(1) != 1) or (t.shape[0] > 1 and t.stride(0) < t.shape[1]):
            raise ValueError(f"{name} must be float32, bfloat16 or float16 rows [R, V] on the device")
        return t.data_ptr(), _LOGITS[t.dtype], max(t.stride(0), t.shape[1])

    def _flat(self, t, dtype, shape, name):
        if t.dtype is not dtype or t.get_device() != self._at or t.shape != shape or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous {dtype} tensor {list(shape)} on the device")

    def logprobs(self, logits: torch.Tensor, ids: torch.Tensor | None = None, *,
                 rows: torch.Tensor | None = None, T: float = 1.0, top: int = 0,
                 out: "LogprobOutput | None" = None) -> "LogprobOutput":
        """Log probabilities of given tokens under softmax(row / T), with the entropy of
        their rows and the ``top`` largest entries (equal logits by rising id), on the
        current torch stream: specdec_logprobs.  ``logits``: [R, V] float32, bfloat16 or
        float16, rows of any stride; ``ids`` (int32 [M], None: no given tokens), ids
        below 0 are skipped (zeros, alternatives -1), so the ``tokens`` of a
        verification can be given as they are; ``rows`` (int32 [M]) the row of each
        token (``tree_rows`` for the tokens of ``tree``), None: its own.  The results carry
        no gradient: ``logprobs_grad`` gives that of the logits."""
        f32, i32 = torch.float32, torch.int32
        x, dt, stride = self._logit_rows(logits, "logits")
        R, V = logits.shape
        M = rows.numel() if rows is not None else ids.numel() if ids is not None else R
        for t, name in ((ids, "ids"), (rows, "rows")):
            if t is not None:
                self._flat(t, i32, (M,), name)
        if M > R and rows is None:
            raise ValueError("more ids than rows")
        if not 0 <= top <= SPECDEC_MAX_TOP:
            raise ValueError(f"top must be 0 .. {SPECDEC_MAX_TOP}")
        if out is None:
            e = lambda *s, dtype=f32: torch.empty(s, dtype=dtype, device=self.device)
            out = LogprobOutput(e(M) if ids is not None else None, e(M), e(M, top, dtype=i32) if top else None,
                                e(M, top) if top else None, e(M, 2))
        else:
            want = {"logprob": ((M,), f32) if ids is not None else None, "entropy": ((M,), f32),
                    "top_ids": ((M, top), i32) if top else None, "top_logprobs": ((M, top), f32) if top else None,
                    "stats": ((M, 2), f32)}
            for name, w in want.items():
                t = getattr(out, name)
                if (t is None) != (w is None):
                    raise ValueError(f"out.{name} does not go with ids and top")
                if w:
                    self._flat(t, w[1], w[0], f"out.{name}")
        out.own_rows = rows is None
        if M:
            if R == 0:
                raise ValueError("logits has no rows")
            _check(specdec_logprobs(self._h, x, dt, stride, R, V, float(T), _ptr(ids) or None, _ptr(rows) or None,
                                    M, top, _ptr(out.logprob) or None, out.entropy.data_ptr(),
                                    _ptr(out.top_ids) or None, _ptr(out.top_logprobs) or None,
                                    out.stats.data_ptr(), _stream_handle(self.device)), "specdec_logprobs")
        return out

    def logprobs_grad(self, logits: torch.Tensor, ids: torch.Tensor | None, forward: "LogprobOutput", *,
                      grad_logprob: torch.Tensor | None = None, grad_entropy: torch.Tensor | None = None,
                      grad_top: torch.Tensor | None = None, T: float = 1.0,
                      out: torch.Tensor | None = None) -> torch.Tensor:
        """The gradient of the logits from those of what ``logprobs`` gave (``forward``,
        with the same logits, ids and T and without ``rows``), float32 [M], [M] and [M,
        top]: specdec_logprobs_grad.  Returns [M, V] of the logits' type; ``out`` may be
        the logits themselves."""
        f32 = torch.float32
        x, dt, stride = self._logit_rows(logits, "logits")
        (R, V), M = logits.shape, forward.stats.shape[0]
        if M != R or not forward.own_rows:
            raise ValueError("the gradient needs a token for every row of the logits, in their order (no rows)")
        if ids is not None:
            self._flat(ids, torch.int32, (M,), "ids")
        if (ids is None) != (forward.logprob is None):
            raise ValueError("ids are not those of the forward call")
        top = 0 if forward.top_ids is None else forward.top_ids.shape[1]
        self._flat(forward.stats, f32, (M, 2), "forward.stats")
        self._flat(forward.entropy, f32, (M,), "forward.entropy")
        if ids is not None:
            self._flat(forward.logprob, f32, (M,), "forward.logprob")
        if top:
            self._flat(forward.top_ids, torch.int32, (M, top), "forward.top_ids")
            self._flat(forward.top_logprobs, f32, (M, top), "forward.top_logprobs")
        for t, shape, name in ((grad_logprob, (M,), "grad_logprob"), (grad_entropy, (M,), "grad_entropy"),
                               (grad_top, (M, top), "grad_top")):
            if t is not None:
                self._flat(t, f32, shape, name)
        if grad_logprob is not None and ids is None:
            raise ValueError("grad_logprob without ids")
        if grad_top is not None and not top:
            raise ValueError("grad_top without alternatives")
        if out is None:
            out = torch.empty(M, V, dtype=logits.dtype, device=self.device)
        o, odt, ostride = self._logit_rows(out, "out")
        if out.shape != logits.shape or odt != dt:
            raise ValueError("out must be like the logits")
        if M:
            _check(specdec_logprobs_grad(
                self._h, x, dt, stride, V, float(T), _ptr(ids) or None, M, top, _ptr(forward.logprob) or None,
                forward.entropy.data_ptr(), _ptr(forward.top_ids) or None, _ptr(forward.top_logprobs) or None,
                forward.stats.data_ptr(), _ptr(grad_logprob) or None, _ptr(grad_entropy) or None,
                _ptr(grad_top) or None, o, ostride, _stream_handle(self.device)), "specdec_logprobs_grad")
        return out

    def rotate(self, x: torch.Tensor, positions: torch.Tensor, rotary: torch.Tensor, *, axes=None,
               interleaved: bool = False, inverse: bool = False, out: torch.Tensor | None = None) -> torch.Tensor:
        """Dense rows x [N, heads, head_dim] (bfloat16 or float16, any row and head
        strides) turned by positions (int32 [N], or [axes, N] with ``axes``, the axis of
        each pair: ``rotary_axes``) of the table ``rotary`` (``rotary_table``), pairs as
        in ``KVCache.append``: specdec_rotate.  ``inverse`` turns back (a table with a gain,
        ``scaling="by_parts"``, is applied once more, not taken back), which is also the
        gradient of a turn; the result itself carries none.  Returns contiguous rows, or
        ``out``: x itself or rows of their own."""
        if x.dim() != 3 or x.dtype not in (torch.bfloat16, torch.float16) or x.get_device() != self._at:
            raise ValueError("x must be bfloat16 or float16 [N, heads, head_dim] on the device")
        N, heads, D = x.shape
        if out is None:
            out = torch.empty(N, heads, D, dtype=x.dtype, device=self.device)
        elif out.shape != x.shape or out.dtype != x.dtype or out.get_device() != self._at:
            raise ValueError("out must be like x")
        for t, name in ((x, "x"), (out, "out")):
            row, head, one = t.stride()
            if N and (one != 1 or row % 8 or head % 8 or t.data_ptr() % 16):
                raise ValueError(f"{name} needs contiguous values, 16-byte aligned rows and strides of multiples of 8")
        if D % 8 or not heads:
            raise ValueError("x needs heads, of a multiple of 8 values")
        table, count, dim = rotary_args(rotary, self._at, D)
        pos, stride, n, which = position_args(positions, axes, N, dim // 2, self._at)
        if N:
            _check(specdec_rotate(self._h, _LOGITS[x.dtype], x.data_ptr(), x.stride(0), x.stride(1), N, heads, D,
                                  pos, stride, n, which, table, dim, count, int(interleaved), int(inverse),
                                  out.data_ptr(), out.stride(0), out.stride(1), _stream_handle(self.device)),
                   "specdec_rotate")
        return out

    def __call__(self, target_logits: torch.Tensor, draft_probs: torch.Tensor | None,
                 draft_ids: torch.Tensor, cu_num_draft_tokens: torch.Tensor, T: float, seed: int,
                 *, with_beta: bool = True, extended: bool = False,
                 out: VerifyOutput | None = None, n_draft: int | None = None,
                 request_offset: int = 0, top_k: torch.Tensor | None = None,
                 top_p: torch.Tensor | None = None) -> VerifyOutput:
        """Runs one verify step on the current torch stream.  ``n_draft`` (= cu[B])
        avoids a host read of cu when output tensors must be allocated.
        ``top_k`` (int32 [B]) / ``top_p`` (float32 [B]) restrict the target
        distribution per request (specdec_rejection_sample_topk_topp)."""
        for t in (target_logits, draft_ids, cu_num_draft_tokens):
            if t.device != self.device or not t.is_contiguous():
                raise ValueError("inputs must be contiguous tensors on the verifier's device")
        if draft_probs is not None and (draft_probs.device != self.device
                                        or draft_probs.dtype != torch.float32
                                        or not draft_probs.is_contiguous()):
            raise ValueError("draft_probs must be a contiguous float32 tensor on the device")
        if target_logits.dtype == torch.float32:
            dtype = SPECDEC_F32
        elif target_logits.dtype == torch.bfloat16:
            dtype = SPECDEC_BF16
        else:
            raise TypeError("target_logits must be float32 or bfloat16")
        if draft_ids.dtype != torch.int32 or cu_num_draft_tokens.dtype != torch.int32:
            raise TypeError("draft_ids and cu_num_draft_tokens must be int32")
        B = cu_num_draft_tokens.numel() - 1
        for t, dt, name in ((top_k, torch.int32, "top_k"), (top_p, torch.float32, "top_p")):
            if t is not None and (t.device != self.device or t.dtype != dt or t.numel() != B
                                  or not t.is_contiguous()):
                raise ValueError(f"{name} must be a contiguous {dt} tensor of B entries on the device")
        V = target_logits.shape[-1]
        if out is None:
            nd = int(cu_num_draft_tokens[-1]) if n_draft is None else int(n_draft)
            kw = dict(device=self.device)
            out = VerifyOutput(
                tokens=torch.empty(nd + B, dtype=torch.int32, **kw),
                num_accepted=torch.empty(B, dtype=torch.int32, **kw),
                beta=torch.empty(nd, dtype=torch.float32, **kw) if with_beta else None)
            if extended:
                out.target_prob = torch.empty(nd, dtype=torch.float32, **kw)
                out.draft_prob = torch.empty(nd, dtype=torch.float32, **kw)
                out.accept = torch.empty(nd, dtype=torch.int32, **kw)
        stream = _stream_handle(self.device)
        if top_k is not None or top_p is not None:
            rc = specdec_rejection_sample_topk_topp(
                self._h, _ptr(target_logits), dtype, _ptr(draft_probs), self._ids_ptr(draft_ids),
                _ptr(cu_num_draft_tokens), B, V, float(T), _ptr(top_k), _ptr(top_p), int(seed),
                int(request_offset), _ptr(out.tokens), _ptr(out.num_accepted), _ptr(out.beta),
                _ptr(out.target_prob), _ptr(out.draft_prob), _ptr(out.accept), stream)
        elif (out.target_prob is not None or out.draft_prob is not None or out.accept is not None
                or request_offset):
            rc = specdec_rejection_sample_ex(
                self._h, _ptr(target_logits), dtype, _ptr(draft_probs), self._ids_ptr(draft_ids),
                _ptr(cu_num_draft_tokens), B, V, float(T), int(seed), int(request_offset),
                _ptr(out.tokens),
                _ptr(out.num_accepted), _ptr(out.beta), _ptr(out.target_prob),
                _ptr(out.draft_prob), _ptr(out.accept), stream)
        else:
            rc = specdec_rejection_sample(
                self._h, _ptr(target_logits), dtype, _ptr(draft_probs), self._ids_ptr(draft_ids),
                _ptr(cu_num_draft_tokens), B, V, float(T), int(seed), _ptr(out.tokens),
                _ptr(out.num_accepted), _ptr(out.beta), stream)
        _check(rc, "specdec_rejection_sample")
        return out


def rotary_args(rotary: torch.Tensor, at: int, head_dim: int) -> tuple[int, int, int]:
    """Data pointer, positions and turning dimensions of a table of cos and sin."""
    if rotary.dim() != 3 or rotary.shape[1] != 2 or rotary.dtype is not torch.float32 \
            or rotary.get_device() != at or not rotary.is_contiguous():
        raise ValueError("rotary must be contiguous float32 [positions, 2, rotary_dim / 2] on the device")
    count, dim = rotary.shape[0], 2 * rotary.shape[2]
    if dim % 16 or not 0 < dim <= min(head_dim, 128) or not count:
        raise ValueError("rotary_dim must be a multiple of 16 up to head_dim and 128")
    return rotary.data_ptr(), count, dim


def position_args(positions: torch.Tensor, axes, N: int, pairs: int, at: int):
    """Data pointer and stride of positions, the number of axes and each pair's own."""
    if positions.dtype is not torch.int32 or positions.get_device() != at or positions.dim() not in (1, 2) \
            or positions.shape[-1] != N or (N > 1 and positions.stride(-1) != 1):
        raise ValueError("positions must be int32 [N] or [axes, N] on the device, the rows' neighbours")
    n = 1 if positions.dim() == 1 else positions.shape[0]
    if not 1 <= n <= SPECDEC_MAX_AXES:
        raise ValueError(f"positions must have 1 .. {SPECDEC_MAX_AXES} axes")
    if n > 1 and axes is None:
        raise ValueError("positions on several axes need the axis of each pair")
    stride = positions.stride(0) if n > 1 else N
    if stride < N:
        raise ValueError("positions must have rows of their own")
    if axes is None:
        return positions.data_ptr(), stride, n, None
    which = tuple(axes)
    if len(which) != pairs or min(which) < 0 or max(which) >= n:
        raise ValueError(f"axes must be {pairs} entries, one for each pair, below {n}")
    return positions.data_ptr(), stride, n, bytes(which)


def rotary_axes(sections, *, spread: bool = False) -> tuple[int, ...]:
    """The axis of each rotary pair for ``sections``, the number of pairs of each axis
    (of time, height and width, say): one block of pairs after the other, or with
    ``spread`` dealt in turn, 0, 1, 2, 0, 1, 2, ..., an axis that has its share passed
    over."""
    left = [int(n) for n in sections]
    if not left or min(left) < 0 or not sum(left):
        raise ValueError("sections must be the number of pairs of each axis")
    if not spread:
        return tuple(a for a, n in enumerate(left) for _ in range(n))
    got = []
    while any(left):
        for a in range(len(left)):
            if left[a]:
                left[a] -= 1
                got.append(a)
    return tuple(got)


def tree_rows(path: torch.Tensor, cu_num_nodes: torch.Tensor) -> torch.Tensor:
    """The target row (int32 [N]) that each slot of ``Verifier.tree``'s tokens comes
    from: node 0's for a request's first token, then those of the accepted nodes; -1
    where no token stands, behind the last request too (``tree`` leaves path and tokens
    there as they are)."""
    first = cu_num_nodes[:-1].long()
    slots = torch.arange(path.numel(), device=path.device)
    req = torch.searchsorted(cu_num_nodes[1:].contiguous(), slots.to(torch.int32), right=True).clamp(max=first.numel() - 1)
    before = torch.cat([path.new_zeros(1), path[:-1]])
    node = torch.where(slots == first[req], 0, before)
    return torch.where((node >= 0) & (slots < cu_num_nodes[-1]), first[req] + node, -1).to(torch.int32)


@dataclass
class TreeOutput:
    tokens: torch.Tensor         # int32 [N] request b: slots cu[b] .. cu[b+1]-1
    num_accepted: torch.Tensor   # int32 [B]
    path: torch.Tensor | None    # int32 [N] accepted nodes (indices within the request), -1


def _tree_call(v: "Verifier", target_logits, draft_probs, node_tokens, node_parent, cu_num_nodes,
               T, seed, request_offset=0, with_path=True, out: TreeOutput | None = None):
    for t in (target_logits, node_tokens, node_parent, cu_num_nodes):
        if t.device != v.device or not t.is_contiguous():
            raise ValueError("inputs must be contiguous tensors on the verifier's device")
    if draft_probs is not None and (draft_probs.device != v.device
                                    or draft_probs.dtype != torch.float32
                                    or not draft_probs.is_contiguous()):
        raise ValueError("draft_probs must be a contiguous float32 tensor on the device")
    if target_logits.dtype == torch.float32:
        dtype = SPECDEC_F32
    elif target_logits.dtype == torch.bfloat16:
        dtype = SPECDEC_BF16
    else:
        raise TypeError("target_logits must be float32 or bfloat16")
    for t in (node_tokens, node_parent, cu_num_nodes):
        if t.dtype != torch.int32:
            raise TypeError("node_tokens, node_parent and cu_num_nodes must be int32")
    B = cu_num_nodes.numel() - 1
    N = node_tokens.numel()
    V = target_logits.shape[-1]
    if out is None:
        out = TreeOutput(tokens=torch.empty(N, dtype=torch.int32, device=v.device),
                         num_accepted=torch.empty(B, dtype=torch.int32, device=v.device),
                         path=torch.empty(N, dtype=torch.int32, device=v.device)
                         if with_path else None)
    rc = specdec_tree_verify(v.handle, _ptr(target_logits), dtype, _ptr(draft_probs),
                             _ptr(node_tokens), _ptr(node_parent), _ptr(cu_num_nodes), B, V,
                             float(T), int(seed), int(request_offset), _ptr(out.tokens),
                             _ptr(out.num_accepted), _ptr(out.path), _stream_handle(v.device))
    _check(rc, "specdec_tree_verify")
    return out


def uniform(seed: int, b: int, pos: int, stream_id: int, v0: int, n: int,
            device: int | torch.device = 0) -> torch.Tensor:
    """The generator's uniforms U(seed, b, pos, stream_id, v0 .. v0+n-1) (float32)."""
    dev = torch.device("cuda", device) if isinstance(device, int) else torch.device(device)
    out = torch.empty(n, dtype=torch.float32, device=dev)
    _check(specdec_uniform(seed, b, pos, stream_id, v0, n, out.data_ptr(), _stream_handle(dev)),
           "specdec_uniform")
    return out


def selection_mass(z: torch.Tensor, V: int) -> tuple[torch.Tensor, torch.Tensor]:
    """The top-p selection's integer masses (int64 holding the uint64 values,
    all below 2^63) and 2^-z (float32) for float32 distances z on the device."""
    if z.dtype != torch.float32 or not z.is_cuda:
        raise ValueError("z must be a float32 CUDA tensor")
    z = z.contiguous()
    mass = torch.empty(z.numel(), dtype=torch.int64, device=z.device)
    p2 = torch.empty(z.numel(), dtype=torch.float32, device=z.device)
    _check(specdec_selection_mass(z.data_ptr(), z.numel(), V, mass.data_ptr(), p2.data_ptr(),
                                  _stream_handle(z.device)), "specdec_selection_mass")
    return mass, p2


def neg_log_uniform(k0: int, n: int, device: int | torch.device = 0) -> torch.Tensor:
    dev = torch.device("cuda", device) if isinstance(device, int) else torch.device(device)
    out = torch.empty(n, dtype=torch.float32, device=dev)
    _check(specdec_neg_log_uniform(k0, n, out.data_ptr(), _stream_handle(dev)),
           "specdec_neg_log_uniform")
    return out
