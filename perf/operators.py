"""Cases of the operators around the verifier: the paged key/value cache that the target's pass over drafted nodes
writes and reads (append, read, attend, commit), and verification from probabilities and given random numbers.

Every case is run in a plain form (elementary torch operations) or, where ``own`` is true, by this repository's kernels.
Sizes that a step's plan holds on the host (context lengths, nodes per request) come from the case alone; everything else
comes from the seed."""
import functools
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}


def listed():
    return [
        # one user, one new token, a short context: the latency of a decode step's attention
        dict(name="attend_token", op="attend", B=1, heads=32, kv_heads=8, head_dim=128, page=16, q_dtype="bf16",
             cache="bf16", ctx_lo=500, ctx_hi=500, nodes_lo=1, nodes_hi=1, tree="chain", sizes=1),
        # a ragged serving batch, 1..8 drafts each behind the last token, contexts from nothing to long
        dict(name="attend_chain_ragged", op="attend", B=64, heads=32, kv_heads=8, head_dim=128, page=64, q_dtype="bf16",
             cache="bf16", ctx_lo=0, ctx_hi=8191, nodes_lo=2, nodes_hi=9, tree="chain", sizes=2),
        # full token trees with branching 4, 2, 2 (29 nodes) over an 8-bit cache
        dict(name="attend_tree_e4m3", op="attend", B=32, heads=32, kv_heads=8, head_dim=128, page=64, q_dtype="bf16",
             cache="e4m3", ctx_lo=6001, ctx_hi=16000, nodes_lo=29, nodes_hi=29, tree="4,2,2", sizes=3),
        # two long documents, 7 drafts: the cache's offsets are large and few requests fill the GPU
        dict(name="attend_long", op="attend", B=2, heads=64, kv_heads=8, head_dim=128, page=64, q_dtype="bf16",
             cache="bf16", ctx_lo=100001, ctx_hi=131000, nodes_lo=8, nodes_hi=8, tree="chain", sizes=4),
        # one user's tree of 29 nodes enters the cache: rotary on the leading half of the head, a far position
        dict(name="append_tree", op="append", B=1, heads=32, kv_heads=8, head_dim=128, page=16, q_dtype="bf16",
             cache="bf16", ctx_lo=100000, ctx_hi=100000, nodes_lo=29, nodes_hi=29, tree="4,2,2", sizes=5,
             rotary_dim=64, interleaved=True, read_back=False),
        # a large batch of trees, quantised to 8 bits on the way in and read back (a cache that another worker takes over)
        dict(name="append_batch_e4m3", op="append", B=512, heads=32, kv_heads=8, head_dim=128, page=64, q_dtype="bf16",
             cache="e4m3", ctx_lo=0, ctx_hi=2000, nodes_lo=29, nodes_hi=29, tree="4,2,2", sizes=6,
             rotary_dim=128, interleaved=False, read_back=True),
        # one short prefix read back
        dict(name="read_short", op="read", B=1, heads=8, kv_heads=8, head_dim=128, page=16, q_dtype="bf16",
             cache="e4m3", ctx_lo=77, ctx_hi=77, nodes_lo=1, nodes_hi=1, tree="chain", sizes=7),
        # whole ragged contexts read back from 8 bits, to be moved or re-used
        dict(name="read_ragged", op="read", B=64, heads=8, kv_heads=8, head_dim=128, page=64, q_dtype="bf16",
             cache="e4m3", ctx_lo=0, ctx_hi=8191, nodes_lo=1, nodes_hi=1, tree="chain", sizes=8),
        # one user's tree written, and its accepted branch put in order
        dict(name="commit_tree", op="commit", B=1, heads=8, kv_heads=8, head_dim=128, page=16, q_dtype="bf16",
             cache="bf16", ctx_lo=999, ctx_hi=999, nodes_lo=29, nodes_hi=29, tree="4,2,2", sizes=9),
        # the same for a large batch over an 8-bit cache
        dict(name="commit_batch_e4m3", op="commit", B=512, heads=8, kv_heads=8, head_dim=128, page=64, q_dtype="bf16",
             cache="e4m3", ctx_lo=0, ctx_hi=2000, nodes_lo=2, nodes_hi=40, tree="random", sizes=10),
        # a small batch verified from given numbers
        dict(name="given_small", op="given", B=8, V=32000, drafts_lo=5, drafts_hi=5, one_hot=False, noise=1.0, sizes=11),
        # a ragged serving batch verified from given numbers
        dict(name="given_ragged", op="given", B=256, V=151936, drafts_lo=1, drafts_hi=8, one_hot=False, noise=1.5, sizes=12),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "append", "read", "commit", "given", "given"])
    sizes = rng.randrange(1, 1 << 30)
    if op == "given":
        V = _log_int(rng, 32, 256000)
        B = _log_int(rng, 1, max(1, min(512, 38_000_000 // V)))
        lo = rng.randrange(0, 5)
        return dict(op=op, B=B, V=V, drafts_lo=lo, drafts_hi=lo + rng.randrange(0, 5), one_hot=rng.random() < 0.3,
                    noise=rng.choice([0.5, 1.0, 1.5]), sizes=sizes)
    kv_heads = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 4, 7, 8])
    head_dim = rng.choice([64, 128])
    q_dtype = rng.choice(["bf16", "f16"])
    cache = rng.choice([q_dtype, "e4m3"])
    page = rng.choice([8, 16, 48, 64, 100, 128])
    tree = rng.choice(["chain", "random", "4,2,2", "2,2,2,2"])
    lo = rng.choice([1, 1, 5])
    hi = lo + _log_int(rng, 1, 40) - 1
    if tree == "4,2,2":
        lo = hi = 29
    if tree == "2,2,2,2":
        lo = hi = 31
    c = dict(op=op, heads=kv_heads * group, kv_heads=kv_heads, head_dim=head_dim, page=page, q_dtype=q_dtype, cache=cache,
             nodes_lo=lo, nodes_hi=hi, tree=tree, sizes=sizes)
    if op in ("append", "commit"):
        c["B"] = _log_int(rng, 1, 512)
        c["ctx_lo"], c["ctx_hi"] = 0, _log_int(rng, 1, 2000)
    else:
        c["B"] = _log_int(rng, 1, 64)
        budget = 128_000 if op == "attend" else 260_000    # rows of context in all
        c["ctx_hi"] = _log_int(rng, 1, max(2, min(131072, budget // c["B"])))
        c["ctx_lo"] = rng.randrange(0, c["ctx_hi"] + 1)
    if op == "append":
        c["rotary_dim"] = rng.choice([0, head_dim // 2, head_dim])
        c["interleaved"] = rng.random() < 0.5
        c["read_back"] = cache == "e4m3"
    return c


# ---- sizes of a case (host side: what a serving loop's plan knows) ------------------------------------------------

def _spread(r, n, lo, hi):
    """n whole numbers over [lo, hi], both ends among them where n allows, in random order."""
    v = [r.randint(lo, hi) for _ in range(n)]
    v[0] = hi
    if n > 1:
        v[-1] = lo
    r.shuffle(v)
    return v


@functools.lru_cache(maxsize=64)
def _plan(key):
    case = dict(key)
    r = random.Random(case["sizes"])
    if case["op"] == "given":
        n = _spread(r, case["B"], case["drafts_lo"], case["drafts_hi"])
        return dict(nodes=n, ctx=[0] * case["B"])
    return dict(ctx=_spread(r, case["B"], case["ctx_lo"], case["ctx_hi"]), nodes=_spread(r, case["B"], case["nodes_lo"], case["nodes_hi"]))


def _plan_of(case):
    return _plan(tuple(sorted((k, v) for k, v in case.items() if k != "name")))


# ---- inputs -------------------------------------------------------------------------------------------------------

def _cu(counts, dev):
    cu = torch.zeros(len(counts) + 1, dtype=torch.int32)
    cu[1:] = torch.tensor(counts, dtype=torch.int64).cumsum(0)
    return cu.to(dev)


def _parents(case, nodes, gen, dev):
    """Parents within each request, concatenated (root -1); None for chains."""
    if case["tree"] == "chain":
        return None
    if case["tree"] == "random":
        local = torch.cat([torch.arange(n) for n in nodes]).to(dev)
        u = torch.rand(local.numel(), generator=gen, device=dev, dtype=torch.float64)
        return torch.where(local > 0, (u * local).long(), -1).to(torch.int32)
    par, level = [-1], [0]
    for k in (int(x) for x in case["tree"].split(",")):
        level = [len(par) - 1 for u in level for _ in range(k) if par.append(u) is None]
    return torch.tensor(par * len(nodes), dtype=torch.int32, device=dev)


def _table(case, plan, gen, dev):
    """A page table of shuffled pages: every request owns the pages of its context and its new nodes."""
    page = case["page"]
    need = torch.tensor([(c + n + page - 1) // page for c, n in zip(plan["ctx"], plan["nodes"])])
    most, total = int(need.max()), int(need.sum())
    order = torch.randperm(total, generator=gen, device=dev).to(torch.int32)
    at = (need.cumsum(0) - need)[:, None] + torch.arange(most)[None]
    held = torch.arange(most)[None] < need[:, None]
    return torch.where(held.to(dev), order[at.clamp(max=total - 1).to(dev)], 0).to(torch.int32).contiguous(), total


def _rotary_table(positions, dim, dev, base=10000.0):
    """cos and sin of position * base^(-2i/dim), [positions, 2, dim/2], made in 64 bits."""
    inv = base ** (-torch.arange(0, dim, 2, dtype=torch.float64, device=dev) / dim)
    a = torch.arange(positions, dtype=torch.float64, device=dev)[:, None] * inv
    return torch.stack([a.cos(), a.sin()], 1).float().contiguous()


def _normal(shape, gen, dev, dtype, std=1.0):
    return torch.empty(shape, dtype=dtype, device=dev).normal_(0.0, std, generator=gen)


def _cache(case, pages, gen, dev):
    """Cache contents [pages, kv_heads, page, head_dim] (and scales) as earlier appends would have left them."""
    shape = (pages, case["kv_heads"], case["page"], case["head_dim"])
    if case["cache"] != "e4m3":
        dt = DTYPES[case["cache"]]
        return _normal(shape, gen, dev, dt, 1.5), _normal(shape, gen, dev, dt), None, None
    got = []
    for std in (1.5, 1.0):
        x8, s = _normal(shape, gen, dev, torch.float16, 120.0).clamp_(-448, 448).to(torch.float8_e4m3fn), None
        s = torch.rand(shape[:3], generator=gen, device=dev) * (std / 120.0) + std / 240.0
        got.append((x8, s))
    return got[0][0], got[1][0], got[0][1], got[1][1]


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    plan = _plan_of(case)
    s = {"case": case, "plan": plan}
    if case["op"] == "given":
        return _prepare_given(case, plan, gen, dev, s)
    N, D, Hkv, qdt = sum(plan["nodes"]), case["head_dim"], case["kv_heads"], DTYPES[case["q_dtype"]]
    s["table"], pages = _table(case, plan, gen, dev)
    s["lengths"] = torch.tensor(plan["ctx"], dtype=torch.int32, device=dev)
    s["cu"] = _cu(plan["nodes"], dev)
    s["parent"] = _parents(case, plan["nodes"], gen, dev)
    s["k"], s["v"], s["ks"], s["vs"] = _cache(case, pages, gen, dev)
    if case["op"] == "attend":
        s["q"] = _normal((N, case["heads"], D), gen, dev, qdt, 1.5)
    if case["op"] == "append":
        # q, k and v as one projection leaves them: slices of one row
        qkv = _normal((N, case["heads"] + 2 * Hkv, D), gen, dev, qdt)
        s["q"], s["new_k"], s["new_v"] = qkv.split([case["heads"], Hkv, Hkv], 1)
        if case["rotary_dim"]:
            s["rotary"] = _rotary_table(max(plan["ctx"]) + max(plan["nodes"]), case["rotary_dim"], dev)
    if case["op"] == "commit":
        s["new_k"], s["new_v"] = _normal((2, N, Hkv, D), gen, dev, qdt).unbind(0)
        s["accepted"], s["path"] = _accepted_path(s, plan, gen, dev)
    if case["op"] == "read":
        s["starts"] = torch.zeros_like(s["lengths"])
        s["cu_rows"] = _cu(plan["ctx"], dev)
    if own:
        from speculative_decoding_rejection_decode_gb300 import KVCache, Verifier
        s["cache"] = KVCache(_verifier(Verifier), s["k"], s["v"], s["ks"], s["vs"])
    return s


@functools.lru_cache(maxsize=1)
def _verifier(cls):
    return cls(torch.cuda.current_device())


def _accepted_path(s, plan, gen, dev):
    """The branch from the root to a random node, as the tree verifier reports it."""
    anc = _ancestors(s["parent"], s["cu"], plan["nodes"])
    B, n, _ = anc.shape
    count = s["cu"].diff().long()
    leaf = (torch.rand(B, generator=gen, device=dev, dtype=torch.float64) * count).long()
    row = anc[torch.arange(B, device=dev), leaf].clone()
    row[:, 0] = False                                   # the root is no draft
    order = torch.where(row, torch.arange(n, device=dev), n).sort(1).values
    req, local = _rows(s["cu"], sum(plan["nodes"]))
    order = torch.cat([order, torch.full_like(order[:, :1], n)], 1)
    path = order[req, local]
    return row.sum(1).to(torch.int32), torch.where(path < n, path, -1).to(torch.int32)


def _prepare_given(case, plan, gen, dev, s):
    V, B, nd = case["V"], case["B"], sum(plan["nodes"])
    cu = _cu(plan["nodes"], dev)
    logits = _normal((nd + B, V), gen, dev, torch.float32, 3.0)
    req, local = _rows(cu, nd)
    drafted = logits[cu.long()[req] + req + local] if nd else logits[:0]
    if case["one_hot"]:
        s["draft_probs"] = None
        s["ids"] = drafted.argmax(1).to(torch.int32)
    else:
        s["draft_probs"] = (drafted + _normal(drafted.shape, gen, dev, torch.float32, case["noise"])).softmax(1)
        s["ids"] = torch.multinomial(s["draft_probs"], 1, generator=gen)[:, 0].to(torch.int32) if nd else req.to(torch.int32)
    s["target_probs"] = logits.softmax(1)
    s["cu"] = cu
    s["accept_u"] = torch.rand(nd, generator=gen, device=dev)
    s["sample_u"] = torch.rand(B, generator=gen, device=dev)
    if own:
        from speculative_decoding_rejection_decode_gb300 import Verifier
        s["verifier"] = _verifier(Verifier)
    return s


# ---- the plain forms ----------------------------------------------------------------------------------------------

def _rows(cu, total):
    """Request and place within it of every row of a ragged batch."""
    at = torch.arange(total, device=cu.device)
    req = torch.searchsorted(cu[1:].long().contiguous(), at, right=True)
    return req, at - cu.long()[req]


def _ancestors(parent, cu, nodes):
    """[B, n, n]: whether node j is node i or one of its ancestors."""
    n, B, dev = max(nodes), len(nodes), cu.device
    at = torch.arange(n, device=dev)
    if parent is None:
        return (at[None, :] <= at[:, None])[None].expand(B, n, n)
    req, local = _rows(cu, sum(nodes))
    step = torch.eye(n, device=dev).repeat(B, 1, 1)
    up = parent.long()
    step[req[up >= 0], local[up >= 0], up[up >= 0]] = 1.0
    for _ in range(max(1, (n - 1).bit_length())):       # paths of twice the length each time
        step = (torch.matmul(step, step) > 0).float()
    return step > 0


def _gathered(s, which, slots):
    """Cache rows of `slots` ([B, L]) of every request as float32 [B, L, kv_heads, head_dim]."""
    page = s["case"]["page"]
    pages = s["table"].gather(1, (slots // page).clamp(max=s["table"].shape[1] - 1)).long()
    x = s[which][pages, :, slots % page].float()
    if s[which + "s"] is not None:
        x = x * s[which + "s"][pages, :, slots % page][..., None]
    return x


def _attend_plain(s):
    case, plan = s["case"], s["plan"]
    Hkv, D, n, B = case["kv_heads"], case["head_dim"], max(plan["nodes"]), case["B"]
    g, N, dev = case["heads"] // Hkv, sum(plan["nodes"]), s["q"].device
    L = max(c + m for c, m in zip(plan["ctx"], plan["nodes"]))
    slots = torch.arange(L, device=dev)[None].expand(B, L)
    lengths, count = s["lengths"].long()[:, None], s["cu"].diff().long()[:, None]
    live = slots < lengths + count
    k = _gathered(s, "k", slots).where(live[..., None, None], 0.0).permute(0, 2, 3, 1)
    v = _gathered(s, "v", slots).where(live[..., None, None], 0.0).transpose(1, 2)
    req, local = _rows(s["cu"], N)
    q = torch.zeros(B, n, case["heads"], D, device=dev)
    q[req, local] = s["q"].float()
    q = q.view(B, n, Hkv, g, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, n * g, D)
    node = (slots - lengths).clamp(0, n - 1)
    seen = _ancestors(s["parent"], s["cu"], plan["nodes"]).gather(2, node[:, None].expand(B, n, L))
    seen = ((slots < lengths)[:, None] | seen) & live[:, None]                       # [B, n, L]
    w = torch.matmul(q, k).mul_(1.0 / math.sqrt(D)).view(B, Hkv, n, g, L)
    w.masked_fill_(~seen[:, None, :, None], -math.inf)
    w.sub_(w.amax(-1, keepdim=True)).exp_()
    o = torch.matmul(w.view(B, Hkv, n * g, L), v) / w.sum(-1).view(B, Hkv, n * g, 1)
    o = o.view(B, Hkv, n, g, D).permute(0, 2, 1, 3, 4).reshape(B, n, case["heads"], D)
    return o[req, local].to(s["q"].dtype)


def _rotate(x, cos, sin, interleaved):
    """x [N, H, D] rotated in its leading dimensions, float32."""
    x, h = x.float(), cos.shape[-1]
    cos, sin = cos[:, None], sin[:, None]
    a, b = (x[..., 0:2 * h:2], x[..., 1:2 * h:2]) if interleaved else (x[..., :h], x[..., h:2 * h])
    ra, rb = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([ra, rb], -1).flatten(-2) if interleaved else torch.cat([ra, rb], -1)
    return torch.cat([turned, x[..., 2 * h:]], -1)


def _store_plain(s, which, x, pages, off):
    if s[which + "s"] is None:
        s[which][pages, :, off] = x.to(s[which].dtype)
        return
    scale = x.abs().amax(-1).clamp(min=2.0 ** -40) / 448.0
    s[which + "s"][pages, :, off] = scale
    s[which].view(torch.uint8)[pages, :, off] = (x / scale[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)


def _append_plain(s):
    case, plan = s["case"], s["plan"]
    req, local = _rows(s["cu"], sum(plan["nodes"]))
    slots = s["lengths"].long()[req] + local
    pages, off = s["table"][req, slots // case["page"]].long(), slots % case["page"]
    k, q = s["new_k"].float(), s.get("q")
    if "rotary" in s:
        depth = _ancestors(s["parent"], s["cu"], plan["nodes"]).sum(-1)[req, local] - 1
        cos, sin = s["rotary"][s["lengths"].long()[req] + depth].unbind(1)
        q = _rotate(q, cos, sin, case["interleaved"]).to(q.dtype)
        k = _rotate(k, cos, sin, case["interleaved"])
    _store_plain(s, "k", k, pages, off)
    _store_plain(s, "v", s["new_v"].float(), pages, off)
    return q


def _read_plain(s, starts, cu, total):
    case = s["case"]
    req, local = _rows(cu, total)
    slots = starts.long()[req] + local
    pages, off = s["table"][req, slots // case["page"]].long(), slots % case["page"]
    got = []
    for which in ("k", "v"):
        x = s[which][pages, :, off]
        if s[which + "s"] is not None:
            x = (x.float() * s[which + "s"][pages, :, off][..., None]).to(DTYPES[case["q_dtype"]])
        got.append(x)
    return got


def _commit_plain(s):
    case, plan = s["case"], s["plan"]
    n = max(plan["nodes"])
    req, local = _rows(s["cu"], sum(plan["nodes"]))
    acc = s["accepted"].long()
    moved = local < acc[req]
    req, d = req[moved], local[moved]
    node = d + 1 if s["path"] is None else s["path"].long()[moved]
    base = s["lengths"].long()[req]
    table, page = s["table"].long(), case["page"]
    src, dst = base + node, base + 1 + d
    for which in ("k", "v", "ks", "vs"):
        x = s[which]
        if x is not None:
            x = x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x
            x[table[req, dst // page], :, dst % page] = x[table[req, src // page], :, src % page]
    return (s["lengths"] + 1 + s["accepted"]).to(torch.int32) if n else s["lengths"]


def _given_plain(s):
    case, plan = s["case"], s["plan"]
    B, V, dev = case["B"], case["V"], s["cu"].device
    nd, most = sum(plan["nodes"]), max(plan["nodes"])
    cu = s["cu"].long()
    gamma = cu.diff()
    b = torch.arange(B, device=dev)
    pt, ids = s["target_probs"], s["ids"].long()
    q = s["draft_probs"]
    passed = torch.zeros(B, most + 1, device=dev)
    if nd:
        req, local = _rows(s["cu"], nd)
        px = pt[cu[req] + req + local, ids].double()
        qx = torch.ones_like(px) if q is None else q.gather(1, ids[:, None])[:, 0].double()
        u = s["accept_u"].double()
        passed[req, local] = ((u < 1.0) & (u * qx < px)).float()
    n = passed.cumprod(1).sum(1).long()
    p = pt[cu[:-1] + b + n].double()
    w = p
    if nd:
        at = (cu[:-1] + n).clamp(max=nd - 1)
        d = torch.zeros_like(p).scatter_(1, ids[at][:, None], 1.0) if q is None else q[at].double()
        less = (p - d).clamp(min=0.0)
        use = (n < gamma) & (less.sum(1) > 0)
        w = torch.where(use[:, None], less, p)
    c = w.cumsum(1)
    token = (c <= (s["sample_u"].double() * c[:, -1])[:, None]).sum(1).clamp(max=V - 1)
    out = torch.full((nd + B,), -1, dtype=torch.int32, device=dev)
    if nd:
        kept = local < n[req]
        out[(cu[req] + req + local)[kept]] = ids[kept].to(torch.int32)
    out[cu[:-1] + b + n] = token.to(torch.int32)
    return out, n.to(torch.int32)


# ---- one pass -----------------------------------------------------------------------------------------------------

def run(state):
    s, op = state, state["case"]["op"]
    total = sum(s["plan"]["nodes"])
    if op == "attend":
        if own:
            return s["cache"].attend(s["q"], s["table"], s["lengths"], s["cu"], s["parent"])
        return _attend_plain(s)
    if op == "append":
        back = s["case"]["read_back"]
        if own:
            q = s["cache"].append(s["new_k"], s["new_v"], s["table"], s["lengths"], s["cu"], s["parent"], q=s["q"],
                                  rotary=s.get("rotary"), interleaved=s["case"]["interleaved"])
            return (q, *(s["cache"].read(s["table"], s["lengths"], s["cu"], n_rows=total, dtype=s["q"].dtype)
                         if back else (s["k"], s["v"])))
        q = _append_plain(s)
        return (q, *(_read_plain(s, s["lengths"], s["cu"], total) if back else (s["k"], s["v"])))
    if op == "read":
        rows = sum(s["plan"]["ctx"])
        if own:
            return s["cache"].read(s["table"], s["starts"], s["cu_rows"], n_rows=rows, dtype=DTYPES[s["case"]["q_dtype"]])
        return _read_plain(s, s["starts"], s["cu_rows"], rows)
    if op == "commit":
        if own:
            s["cache"].append(s["new_k"], s["new_v"], s["table"], s["lengths"], s["cu"], s["parent"])
            lengths = s["cache"].commit(s["table"], s["lengths"], s["cu"], s["accepted"], s["path"])
            return (lengths, *s["cache"].read(s["table"], s["lengths"], s["cu"], n_rows=total, dtype=s["new_k"].dtype))
        _append_plain(s)
        lengths = _commit_plain(s)
        return (lengths, *_read_plain(s, s["lengths"], s["cu"], total))
    if own:
        out = s["verifier"].sample_given(s["target_probs"], s["draft_probs"], s["ids"], s["cu"], s["accept_u"], s["sample_u"])
        return out.tokens, out.num_accepted
    return _given_plain(s)


# ---- what a pass cannot do without --------------------------------------------------------------------------------

def work(case):
    plan = _plan_of(case)
    if case["op"] == "given":
        rows = sum(1 + (0 if case["one_hot"] else 1 - 0.75 ** n) for n in plan["nodes"])   # a rejected row has a draft row
        return {"bytes": rows * case["V"] * 4.0, "flops": rows * case["V"] * 2.0}
    D, Hkv, H = case["head_dim"], case["kv_heads"], case["heads"]
    cached = 2 * Hkv * (D + 4 if case["cache"] == "e4m3" else 2 * D)     # a cache row of k and v, with its scales
    dense = 2 * Hkv * D * 2                                              # the same as 16-bit tensors
    nodes, ctx = sum(plan["nodes"]), sum(plan["ctx"])
    if case["op"] == "attend":
        pairs = sum(n * (c + 1) for n, c in zip(plan["nodes"], plan["ctx"]))             # its context and itself at the least
        return {"bytes": (ctx + nodes) * cached + 2 * nodes * H * D * 2, "flops": 4.0 * D * H * pairs}
    if case["op"] == "append":
        b = nodes * (dense + cached + (2 * H * D * 2 if case["rotary_dim"] else 0) + case["rotary_dim"] * 4)
        return {"bytes": b + (nodes * (cached + dense) if case["read_back"] else 0), "flops": 3.0 * nodes * (H + Hkv) * case["rotary_dim"]}
    if case["op"] == "read":
        return {"bytes": max(1, ctx) * (cached + dense), "flops": 0}
    return {"bytes": nodes * 2 * (dense + cached), "flops": 0}


# ---- the definitions, in 64 bits ----------------------------------------------------------------------------------

def _walk(parent, first, i):
    """Node i and its ancestors, up to the root."""
    chain = []
    while i >= 0:
        chain.append(i)
        i = i - 1 if parent is None else parent[first + i]
    return chain


def _exact_slots(s, b, count, start=0):
    at = torch.arange(start, start + count, device=s["table"].device)
    return s["table"][b].long()[at // s["case"]["page"]], at % s["case"]["page"]


def _exact_values(s, which, pages, off):
    x = s[which][pages, :, off].double()
    return x if s[which + "s"] is None else x * s[which + "s"][pages, :, off].double().unsqueeze(-1)


def _exact_new_rows(s, x, b, first, turn):
    """k or v rows of request b in 64 bits, rotated where `turn`, as the cache's type holds them."""
    case, plan = s["case"], s["plan"]
    n = plan["nodes"][b]
    x = x[first:first + n].double()
    if turn:
        x = _exact_turn(s, x, b, first)
    if case["cache"] != "e4m3":
        return x
    scale = x.abs().amax(-1, keepdim=True).clamp(min=2.0 ** -40) / 448.0
    return (x / scale).to(torch.float8_e4m3fn).double() * scale


def _exact_turn(s, x, b, first):
    case, plan = s["case"], s["plan"]
    parent = None if s["parent"] is None else s["host_parent"]
    depth = [len(_walk(parent, first, i)) - 1 for i in range(plan["nodes"][b])]
    pos = torch.tensor([plan["ctx"][b] + d for d in depth], dtype=torch.float64, device=x.device)
    x = x.clone()
    half = case["rotary_dim"] // 2
    for i in range(half):
        a = (pos * 10000.0 ** (-2.0 * i / case["rotary_dim"]))[:, None]
        p, q = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + half)
        u, w = x[..., p].clone(), x[..., q].clone()
        x[..., p], x[..., q] = u * a.cos() - w * a.sin(), w * a.cos() + u * a.sin()
    return x


def exact(case, seed):
    s = prepare(case, seed)
    plan, op = s["plan"], case["op"]
    if op == "given":
        return None             # whole numbers only
    s["host_parent"] = None if s["parent"] is None else s["parent"].tolist()
    firsts = [sum(plan["nodes"][:b]) for b in range(case["B"])]
    if op == "attend":
        return torch.cat([_exact_attend(s, b, firsts[b]) for b in range(case["B"])])
    if op == "read":
        return [torch.cat([_exact_values(s, w, *_exact_slots(s, b, plan["ctx"][b])) for b in range(case["B"])]) for w in ("k", "v")]
    turn = bool(case.get("rotary_dim"))
    if op == "append" and not case["read_back"]:
        k, v = s["k"].double(), s["v"].double()
        for b, f in enumerate(firsts):
            pages, off = _exact_slots(s, b, plan["nodes"][b], plan["ctx"][b])
            k[pages, :, off] = _exact_new_rows(s, s["new_k"], b, f, turn)
            v[pages, :, off] = _exact_new_rows(s, s["new_v"], b, f, False)
    else:
        k = [_exact_new_rows(s, s["new_k"], b, f, turn) for b, f in enumerate(firsts)]
        v = [_exact_new_rows(s, s["new_v"], b, f, False) for b, f in enumerate(firsts)]
        if op == "commit":
            acc = s["accepted"].tolist()
            path = s["path"].tolist()
            for b, f in enumerate(firsts):
                for d in range(acc[b]):
                    k[b][1 + d], v[b][1 + d] = k[b][path[f + d]].clone(), v[b][path[f + d]].clone()
            return (None, torch.cat(k), torch.cat(v))
        k, v = torch.cat(k), torch.cat(v)
    q = s["q"].double()
    if turn:
        q = torch.cat([_exact_turn(s, q[f:f + n], b, f) for b, (f, n) in enumerate(zip(firsts, plan["nodes"]))])
    return (q, k, v)


def _exact_attend(s, b, first):
    case, plan = s["case"], s["plan"]
    c, n, g = plan["ctx"][b], plan["nodes"][b], case["heads"] // case["kv_heads"]
    pages, off = _exact_slots(s, b, c + n)
    k, v = _exact_values(s, "k", pages, off), _exact_values(s, "v", pages, off)      # [L, kv_heads, D]
    hidden = torch.ones(n, c + n, dtype=torch.bool, device=k.device)
    hidden[:, :c] = False
    for i in range(n):
        hidden[i, [c + j for j in _walk(None if s["parent"] is None else s["host_parent"], first, i)]] = False
    q = s["q"][first:first + n].double()
    out = []
    for h in range(case["heads"]):
        z = (q[:, h] @ k[:, h // g].T) / math.sqrt(case["head_dim"])
        z = z.masked_fill(hidden, -math.inf)
        e = (z - z.max(1, keepdim=True).values).exp()
        out.append((e @ v[:, h // g]) / e.sum(1, keepdim=True))
    return torch.stack(out, 1)
