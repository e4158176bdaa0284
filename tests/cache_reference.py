"""Plain 64-bit implementations of the paged cache's operators, request by
request and row by row, and seeded workloads for them (test infrastructure)."""
import math

import numpy as np
import torch

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


def make_parents(kind, n, rng):
    if kind == "chain":
        return [j - 1 for j in range(n)]
    if kind == "random":
        return [-1 if j == 0 else int(rng.integers(0, j)) for j in range(n)]
    if kind == "star":
        return [-1] + [0] * (n - 1) if n else []
    raise ValueError(kind)


def ancestors(parents, i):
    got = []
    while i >= 0:
        got.append(i)
        i = parents[i]
    return got


class Step:
    """A seeded cache with its page table, contexts and nodes."""

    def __init__(self, *, ctx, nodes, tree="chain", kv_heads=2, group=4, head_dim=128, page=16,
                 dtype=torch.bfloat16, cache=None, seed=0, extra_rows=0, spare_pages=3,
                 device="cuda", poison=True):
        rng = np.random.default_rng(seed)
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        self.ctx, self.nodes, self.kv_heads, self.group = list(ctx), list(nodes), kv_heads, group
        self.heads, self.head_dim, self.page, self.dtype = kv_heads * group, head_dim, page, dtype
        self.cache_dtype = cache or dtype
        self.B, self.n_rows = len(ctx), sum(nodes)
        self.N = self.n_rows + extra_rows
        self.parents = [make_parents(tree, n, rng) for n in nodes]
        need = [-(-(c + n) // page) for c, n in zip(ctx, nodes)]
        total = sum(need) + spare_pages
        order = rng.permutation(total)
        most = max(max(need), 1)
        table = np.zeros((self.B, most), np.int32)
        self.pages, at = [], 0
        for b, k in enumerate(need):
            table[b, :k] = order[at:at + k]
            self.pages.append([int(x) for x in order[at:at + k]])
            at += k
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=device)
        self.table, self.lengths = i32(table), i32(self.ctx)
        self.firsts = np.concatenate([[0], np.cumsum(nodes)]).astype(int).tolist()
        self.cu = i32(self.firsts)
        flat = [p for par in self.parents for p in par] + [-1] * extra_rows
        self.parent = None if tree == "chain" else i32(flat if flat else [-1])[:self.N]
        self.num_pages = total
        shape = (total, kv_heads, page, head_dim)
        n = lambda s, std=1.0: torch.randn(s, generator=g, device=device) * std
        self.ks = self.vs = None
        if self.cache_dtype == torch.float8_e4m3fn:
            self.k = n(shape, 110.0).clamp(-448, 448).to(torch.float8_e4m3fn)
            self.v = n(shape, 110.0).clamp(-448, 448).to(torch.float8_e4m3fn)
            # scales over two orders of magnitude: no single one fits all rows
            self.ks = (torch.rand(shape[:3], generator=g, device=device) + 0.1) * 0.02
            self.vs = 10.0 ** (-3 * torch.rand(shape[:3], generator=g, device=device)) * 0.05
        else:
            self.k, self.v = n(shape, 1.5).to(self.cache_dtype), n(shape).to(self.cache_dtype)
        self.q = n((self.N, self.heads, head_dim), 1.5).to(dtype)
        self.new_k = n((self.N, kv_heads, head_dim)).to(dtype)
        self.new_v = n((self.N, kv_heads, head_dim)).to(dtype)
        if poison:
            self.poison_unused()

    def poison_unused(self):
        """NaN in every slot that no request has filled."""
        used = torch.zeros(self.num_pages, self.page, dtype=torch.bool)
        for b in range(self.B):
            for s in range(self.ctx[b] + self.nodes[b]):
                used[self.pages[b][s // self.page], s % self.page] = True
        off = ~used.to(self.k.device)[:, None, :, None].expand(self.k.shape)
        if self.ks is None:
            for t in (self.k, self.v):
                t.masked_fill_(off, math.nan)
        else:
            for t in (self.k, self.v):
                t.view(torch.uint8).masked_fill_(off, 0x7F)
            for t in (self.ks, self.vs):
                t.masked_fill_(off[..., 0], math.nan)

    def row(self, b, slot):
        return self.pages[b][slot // self.page], slot % self.page

    def cache(self, verifier):
        from speculative_decoding_rejection_decode_gb300 import KVCache
        return KVCache(verifier, self.k, self.v, self.ks, self.vs)

    def values(self, which):
        """The cache's values in 64 bits, [pages, kv_heads, page, head_dim]."""
        x, s = (self.k, self.ks) if which == "k" else (self.v, self.vs)
        x = x.float().double()
        return x if s is None else x * s.double()[..., None]

    def attend(self, scale=None):
        """float64 [n_rows, heads, head_dim] and, per row, the largest |v| seen."""
        scale = self.head_dim ** -0.5 if scale is None else scale
        K, V = self.values("k"), self.values("v")
        out = torch.zeros(self.n_rows, self.heads, self.head_dim, dtype=torch.float64, device=K.device)
        big = torch.zeros(self.n_rows, self.heads, dtype=torch.float64, device=K.device)
        for b in range(self.B):
            c, n = self.ctx[b], self.nodes[b]
            if n == 0:
                continue
            slots = torch.arange(c + n, device=K.device)
            pages = torch.tensor(self.pages[b], device=K.device)[slots // self.page]
            k, v = K[pages, :, slots % self.page], V[pages, :, slots % self.page]
            for i in range(n):
                at = list(range(c)) + sorted(c + j for j in ancestors(self.parents[b], i))
                at = torch.tensor(at, device=K.device)
                q = self.q[self.firsts[b] + i].double().view(self.kv_heads, self.group, -1)
                z = torch.einsum("hgd,shd->hgs", q, k[at]) * scale
                w = torch.softmax(z, -1)
                out[self.firsts[b] + i] = torch.einsum("hgs,shd->hgd", w, v[at]).reshape(self.heads, -1)
                big[self.firsts[b] + i] = v[at].abs().amax((0, 2)).repeat_interleave(self.group)
        return out, big


def attend_tolerance(step, want, big):
    """Elementwise bound of the kernel's error.  Weights are convex, so with V =
    max |v| over the keys a row sees: rounding each weight to 16 bits moves the
    result by at most half a step of V; an error d of a score (base e) moves it by
    at most 2 d V.  A score is a float32 sum of head_dim exact products: |d| <=
    head_dim 2^-24 sum |q k| scale <= 128 * 2^-24 * 30 = 2.3e-4 for these inputs
    (|q| < 7, |k| < 7 and sum |q k| / sqrt(head_dim) < 30), with the exponential's
    own error of 2^-21 far below; the sums over up to 2^11 keys in float32 add
    2^-13 V at most.  bf16 rows over 8-bit caches may scale the values in f16, the
    factor and each product rounded: half a step of f16 each.  The result is rounded
    to its type."""
    weight = HALF_STEP[torch.float16 if step.ks is not None else step.dtype]
    if step.ks is not None and step.dtype == torch.bfloat16:
        weight += 2 * HALF_STEP[torch.float16]
    return (weight + 2 * 2.3e-4 + 2.0 ** -13) * big[..., None] + HALF_STEP[step.dtype] * want.abs() + 1e-30


def rotate64(x, pos, freq, gain, interleaved):
    """x [..., head_dim] float64 turned to position pos."""
    x, h = x.clone(), len(freq)
    for i in range(h):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + h)
        c, s = math.cos(pos * freq[i]) * gain, math.sin(pos * freq[i]) * gain
        u, w = x[..., a].clone(), x[..., b].clone()
        x[..., a], x[..., b] = u * c - w * s, w * c + u * s
    return x
