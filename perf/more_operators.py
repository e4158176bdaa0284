"""Cases of the operators that a target with an encoder or with image and video positions needs around the verifier, and
of what a step answers and a drafter learns from: log probabilities of given tokens (with entropy, top alternatives and
the gradient of the logits), rotary positions with several axes (on the way into the paged cache, and on dense rows),
and cross attention of a step's rows to an encoder's states.

Every case is run in a plain form (elementary torch operations) or, where ``own`` is true, by this repository's kernels.
Sizes that a step's plan holds on the host (lengths, rows and emitted tokens of every request, image grids) come from the
case alone; everything else comes from the seed."""
import functools
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}


def listed():
    return [
        # what a small chat server reports of one verified step: 8 requests of 5 drafts, 5 alternatives for every token
        dict(name="logprob_step", op="logprob", B=8, V=32000, dtype="f32", nodes_lo=6, nodes_hi=6, rows="chain", top=5,
             T=1.0, hidden=0.0, sizes=1),
        # a large batch of token trees: the rows of the emitted tokens lie scattered among all nodes' rows
        dict(name="logprob_tree", op="logprob", B=256, V=151936, dtype="bf16", nodes_lo=29, nodes_hi=29, rows="tree", top=20,
             T=0.7, hidden=0.0, sizes=2),
        # one short sequence of a drafter's training step: log probability and entropy, and the gradient of the logits
        dict(name="logprob_grad_short", op="logprob_grad", B=1, V=32000, dtype="f32", nodes_lo=60, nodes_hi=60, rows="all",
             top=0, T=1.0, hidden=0.0, sizes=3),
        # a packed training batch with an odd vocabulary, a part of whose tokens (prompts) have no loss
        dict(name="logprob_grad_batch", op="logprob_grad", B=8, V=128257, dtype="bf16", nodes_lo=200, nodes_hi=300, rows="some",
             top=0, T=1.0, hidden=0.0, sizes=4),
        # one image in a prompt: text, 24 x 36 patches with (time, height, width) positions, text
        dict(name="append_image", op="append", B=1, heads=32, kv_heads=8, head_dim=128, page=16, q_dtype="bf16", cache="bf16",
             ctx_lo=0, ctx_hi=0, text=21, time=1, high=24, wide=36, sections="24,20,20", spread=True, interleaved=False, sizes=5),
        # a batch of videos whose prompts enter an 8-bit cache, and are read back (a cache that another worker takes over)
        dict(name="append_video_e4m3", op="append", B=16, heads=32, kv_heads=8, head_dim=128, page=64, q_dtype="bf16",
             cache="e4m3", ctx_lo=0, ctx_hi=500, text=33, time=12, high=14, wide=18, sections="16,24,24", spread=False,
             interleaved=False, sizes=6),
        # a few image tokens turned as dense rows, queries and keys as one projection leaves them
        dict(name="rotate_short", op="rotate", N=77, heads=40, all_heads=48, head_dim=128, q_dtype="bf16", sections="16,24,24",
             spread=False, interleaved=False, inverse=False, sizes=7),
        # the gradients of a vision encoder's rows turned back, two axes
        dict(name="rotate_back_batch", op="rotate", N=49999, heads=32, all_heads=32, head_dim=64, q_dtype="bf16", sections="16,16",
             spread=False, interleaved=True, inverse=True, sizes=8),
        # one user's next token meets the states of a short source sentence: the latency of a decode step
        dict(name="cross_token", op="cross", B=1, heads=16, kv_heads=16, head_dim=64, page=16, q_dtype="bf16", cache="bf16",
             len_lo=500, len_hi=500, rows_lo=1, rows_hi=1, masked=0.0, scale=1.0, sizes=9),
        # a ragged serving batch, 1..8 drafts each, every query head with keys of its own, some states masked
        dict(name="cross_drafts_ragged", op="cross", B=64, heads=32, kv_heads=32, head_dim=128, page=64, q_dtype="bf16",
             cache="bf16", len_lo=0, len_hi=2047, rows_lo=2, rows_hi=9, masked=0.1, scale=None, sizes=10),
        # token trees of 29 nodes over long states held in 8 bits
        dict(name="cross_tree_e4m3", op="cross", B=32, heads=32, kv_heads=8, head_dim=128, page=64, q_dtype="bf16", cache="e4m3",
             len_lo=1500, len_hi=12000, rows_lo=29, rows_hi=29, masked=0.0, scale=None, sizes=11),
        # whole target prompts against whole sources: bound by the products
        dict(name="cross_prompt", op="cross", B=8, heads=32, kv_heads=8, head_dim=128, page=64, q_dtype="bf16", cache="bf16",
             len_lo=1500, len_hi=4096, rows_lo=1000, rows_hi=2048, masked=0.0, scale=None, sizes=12),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["logprob", "logprob", "logprob_grad", "append", "rotate", "cross", "cross", "cross"])
    sizes = rng.randrange(1, 1 << 30)
    if op in ("logprob", "logprob_grad"):
        V = _log_int(rng, 32, 256000)
        nodes = rng.randrange(1, 40)
        B = _log_int(rng, 1, max(1, min(512, 200_000_000 // (V * nodes))))
        rows = rng.choice(["chain", "tree", "some", "all"]) if op == "logprob" else rng.choice(["some", "all"])
        return dict(op=op, B=B, V=V, dtype=rng.choice(["bf16", "f16", "f32"]), nodes_lo=max(1, nodes - rng.randrange(0, 9)),
                    nodes_hi=nodes, rows=rows, top=rng.choice([0, 1, 5, 20, 32]) if op == "logprob" else 0,
                    T=rng.choice([1.0, 0.6, 1.5]), hidden=rng.choice([0.0, 0.0, 0.3]), sizes=sizes)
    kv_heads = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 4, 7])
    head_dim = rng.choice([64, 128])
    q_dtype = rng.choice(["bf16", "f16"])
    c = dict(op=op, head_dim=head_dim, q_dtype=q_dtype, sizes=sizes)
    if op == "rotate":
        heads = kv_heads * (group + 1)
        c.update(N=_log_int(rng, 1, 49999 * 32 * 64 // (heads * head_dim)), heads=heads, all_heads=heads + rng.choice([0, kv_heads]))
    else:
        c.update(heads=kv_heads * group, kv_heads=kv_heads, page=rng.choice([8, 16, 48, 64, 100, 128]),
                 cache=rng.choice([q_dtype, "e4m3"]))
    if op == "cross":
        c["B"] = _log_int(rng, 1, 64)
        c["rows_lo"] = rng.choice([1, 1, 5])
        c["rows_hi"] = c["rows_lo"] + _log_int(rng, 1, max(2, min(2000, 8000 // c["B"]))) - 1
        c["len_hi"] = _log_int(rng, 1, max(2, min(16384, 180_000 // c["B"], 30_000_000 // (c["B"] * c["rows_hi"]))))
        c["len_lo"] = rng.randrange(0, c["len_hi"] + 1)
        c["masked"] = rng.choice([0.0, 0.0, 0.2])
        c["scale"] = rng.choice([None, 1.0 / head_dim])
        return c
    c["interleaved"] = rng.random() < 0.5
    pairs = rng.choice([head_dim // 4, head_dim // 2])
    axes = rng.choice([1, 2, 3, 4])
    cuts = sorted(rng.sample(range(1, pairs), axes - 1))
    c["sections"] = ",".join(str(b - a) for a, b in zip([0] + cuts, cuts + [pairs]))
    c["spread"] = rng.random() < 0.5
    if op == "rotate":
        c["inverse"] = rng.random() < 0.5
        return c
    c["B"] = _log_int(rng, 1, 64)
    c["ctx_lo"], c["ctx_hi"] = 0, _log_int(rng, 1, 1000)
    c["text"] = rng.randrange(1, 40)
    c["time"], c["high"], c["wide"] = rng.choice([1, 1, 2, 5]), rng.randrange(1, 20), rng.randrange(1, 20)
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


def _positions(r, case):
    """(time, height, width) of a prompt of text, one grid and text again: text moves on along all axes together, a
    grid's cells lie at their own places behind the text before it, and the text behind it goes on after the largest."""
    before, after = r.randint(0, case["text"]), r.randint(1, case["text"])
    t, h, w = case["time"], r.randint(max(1, case["high"] - 3), case["high"]), r.randint(max(1, case["wide"] - 3), case["wide"])
    rows = [(i, i, i) for i in range(before)]
    rows += [(before + i, before + j, before + k) for i in range(t) for j in range(h) for k in range(w)]
    first = before + max(t, h, w)
    return rows + [(first + i,) * 3 for i in range(after)]


@functools.lru_cache(maxsize=64)
def _plan(key):
    case = dict(key)
    r = random.Random(case["sizes"])
    if case["op"] in ("logprob", "logprob_grad"):
        nodes = _spread(r, case["B"], case["nodes_lo"], case["nodes_hi"])
        # the tokens that a request has emitted, its accepted drafts and one more (or the tokens that have a loss)
        most = {"chain": 1.0, "tree": 0.15, "some": 0.8, "all": 1.0}[case["rows"]]
        kept = [n if case["rows"] == "all" else r.randint(1, max(1, int(n * most))) for n in nodes]
        return dict(nodes=nodes, kept=kept)
    if case["op"] == "append":
        pos = [_positions(r, case) for _ in range(case["B"])]
        return dict(ctx=_spread(r, case["B"], case["ctx_lo"], case["ctx_hi"]), nodes=[len(p) for p in pos], positions=pos)
    if case["op"] == "cross":
        return dict(ctx=_spread(r, case["B"], case["len_lo"], case["len_hi"]), nodes=_spread(r, case["B"], case["rows_lo"], case["rows_hi"]))
    return {}


def _plan_of(case):
    return _plan(tuple(sorted((k, v) for k, v in case.items() if k != "name")))


def _axes(case):
    """Axis of each pair, from the sections: one block after the other, or dealt in turn while an axis has pairs left."""
    left = [int(x) for x in case["sections"].split(",")]
    if not case["spread"]:
        return [a for a, n in enumerate(left) for _ in range(n)]
    got = []
    while any(left):
        for a in range(len(left)):
            if left[a]:
                left[a] -= 1
                got.append(a)
    return got


# ---- inputs -------------------------------------------------------------------------------------------------------

def _cu(counts, dev):
    cu = torch.zeros(len(counts) + 1, dtype=torch.int32)
    cu[1:] = torch.tensor(counts, dtype=torch.int64).cumsum(0)
    return cu.to(dev)


def _table(case, slots, gen, dev):
    """A page table of shuffled pages: every request owns the pages of its slots."""
    page = case["page"]
    need = torch.tensor([(n + page - 1) // page for n in slots])
    most, total = max(1, int(need.max())), max(1, int(need.sum()))
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
        x8 = _normal(shape, gen, dev, torch.float16, 120.0).clamp_(-448, 448).to(torch.float8_e4m3fn)
        got.append((x8, torch.rand(shape[:3], generator=gen, device=dev) * (std / 120.0) + std / 240.0))
    return got[0][0], got[1][0], got[0][1], got[1][1]


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    plan = _plan_of(case)
    s = {"case": case, "plan": plan}
    if own:
        from speculative_decoding_rejection_decode_gb300 import KVCache, Verifier
        s["verifier"] = _verifier(Verifier)
    if case["op"] in ("logprob", "logprob_grad"):
        return _prepare_logprob(case, plan, gen, dev, s)
    if case["op"] == "rotate":
        return _prepare_rotate(case, gen, dev, s)
    qdt, Hkv, D, N = DTYPES[case["q_dtype"]], case["kv_heads"], case["head_dim"], sum(plan["nodes"])
    extra = plan["nodes"] if case["op"] == "append" else [0] * case["B"]
    s["table"], pages = _table(case, [c + n for c, n in zip(plan["ctx"], extra)], gen, dev)
    s["lengths"] = torch.tensor(plan["ctx"], dtype=torch.int32, device=dev)
    s["cu"] = _cu(plan["nodes"], dev)
    s["k"], s["v"], s["ks"], s["vs"] = _cache(case, pages, gen, dev)
    if case["op"] == "append":
        qkv = _normal((N, case["heads"] + 2 * Hkv, D), gen, dev, qdt)
        s["q"], s["new_k"], s["new_v"] = qkv.split([case["heads"], Hkv, Hkv], 1)
        axes = len(case["sections"].split(","))
        rows = [p for request in plan["positions"] for p in request]
        s["positions"] = torch.tensor(rows, dtype=torch.int32).T[[a % 3 for a in range(axes)]].contiguous().to(dev)
        s["axes"] = _axes(case)
        s["rotary"] = _rotary_table(max(max(p) for p in rows) + 1, 2 * len(s["axes"]), dev)
    else:
        s["q"] = _normal((N, case["heads"], D), gen, dev, qdt, 1.5 if case["scale"] != 1.0 else 0.2)
        s["mask"] = None
        if case["masked"]:
            s["mask"] = torch.rand(case["B"], max(1, max(plan["ctx"])), generator=gen, device=dev) >= case["masked"]
            s["mask"][0] = False                          # a request none of whose states may be seen
    if own:
        s["cache"] = KVCache(s["verifier"], s["k"], s["v"], s["ks"], s["vs"])
    return s


@functools.lru_cache(maxsize=1)
def _verifier(cls):
    return cls(torch.cuda.current_device())


def _prepare_logprob(case, plan, gen, dev, s):
    V, R = case["V"], sum(plan["nodes"])
    s["logits"] = _normal((R, V), gen, dev, DTYPES[case["dtype"]], 3.0)
    s["ids"] = torch.randint(0, V, (R,), generator=gen, device=dev, dtype=torch.int32)
    # drafted and sampled tokens are likely ones: half of the ids are the best of 32 random places
    if V > 64:
        near = torch.randint(0, V, (R, 32), generator=gen, device=dev)
        best = near.gather(1, s["logits"].gather(1, near).float().argmax(1, keepdim=True))[:, 0]
        s["ids"][::2] = best[::2].to(torch.int32)
    if case["hidden"]:
        # words that a grammar forbids, never the given token
        off = torch.rand(V, generator=gen, device=dev) < case["hidden"]
        kept = s["logits"].gather(1, s["ids"].long()[:, None])
        s["logits"].masked_fill_(off[None], -math.inf).scatter_(1, s["ids"].long()[:, None], kept)
    cu = _cu(plan["nodes"], dev)
    req, local = _rows(cu, R)
    kept = torch.tensor(plan["kept"], device=dev)[req]
    s["rows"] = None
    if case["rows"] == "tree":
        # the token in slot d of a request comes from the row of a node at depth d: rising nodes
        room = (torch.tensor(plan["nodes"], device=dev)[req] - 1) // kept.clamp(min=1)
        s["rows"] = (cu.long()[req] + torch.where(local > 0, (local * room.clamp(min=1)), 0)).clamp(max=R - 1).to(torch.int32)
    if case["rows"] == "some":
        s["ids"] = torch.where(local >= torch.tensor(plan["nodes"], device=dev)[req] - kept, s["ids"], -1).to(torch.int32)
    elif case["rows"] != "all":
        s["ids"] = torch.where(local < kept, s["ids"], -1).to(torch.int32)
    if case["op"] == "logprob_grad":
        s["g_logprob"] = _normal((R,), gen, dev, torch.float32, 1.0 / R)
        s["g_entropy"] = _normal((R,), gen, dev, torch.float32, 0.1 / R)
    return s


def _prepare_rotate(case, gen, dev, s):
    x = _normal((case["N"], case["all_heads"], case["head_dim"]), gen, dev, DTYPES[case["q_dtype"]])
    s["x"] = x[:, :case["heads"]]
    s["axes"] = _axes(case)
    top = 4096
    s["positions"] = torch.randint(0, top, (max(s["axes"]) + 1, case["N"]), generator=gen, device=dev, dtype=torch.int32)
    s["rotary"] = _rotary_table(top, 2 * len(s["axes"]), dev)
    return s


# ---- the plain forms ----------------------------------------------------------------------------------------------

def _rows(cu, total):
    """Request and place within it of every row of a ragged batch."""
    at = torch.arange(total, device=cu.device)
    req = torch.searchsorted(cu[1:].long().contiguous(), at, right=True)
    return req, at - cu.long()[req]


def _logprob_plain(s):
    case = s["case"]
    M, top, dev = s["ids"].numel(), case["top"], s["ids"].device
    live = (s["ids"] >= 0).nonzero()[:, 0]
    rows = live if s["rows"] is None else s["rows"].long()[live]
    x = s["logits"][rows].float()
    y = x / case["T"]
    y = y - y.amax(1, keepdim=True)
    e = y.exp()
    total = e.sum(1, keepdim=True)
    lp = y - total.log()
    out = [torch.zeros(M, device=dev), torch.zeros(M, device=dev)]
    out[0][live] = lp.gather(1, s["ids"].long()[live, None])[:, 0]
    out[1][live] = -(e * lp).where(e > 0, 0.0).sum(1) / total[:, 0]
    if top:
        n = min(top, case["V"])
        bits = (x + 0.0).view(torch.int32)
        order = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long()
        key = (order << 32) + (0x7FFFFFFF - torch.arange(case["V"], device=dev))
        at = 0x7FFFFFFF - (key.topk(n, 1).values & 0x7FFFFFFF)
        ids = torch.full((M, top), -1, dtype=torch.int32, device=dev)
        lps = torch.zeros(M, top, device=dev)
        lps[live] = -math.inf
        ids[live, :n] = at.to(torch.int32)
        lps[live, :n] = lp.gather(1, at)
        out += [ids, lps]
    if case["op"] == "logprob_grad":
        p = e / total
        g, h = s["g_logprob"][live, None], s["g_entropy"][live, None]
        d = -p * (g + h * (lp.where(e > 0, 0.0) + out[1][live, None]))
        d.scatter_add_(1, s["ids"].long()[live, None], g)
        grad = torch.zeros_like(s["logits"])
        grad[rows] = (d / case["T"]).to(grad.dtype)
        out.append(grad)
    return out


def _rotate(x, cos, sin, interleaved):
    """x [N, H, D] rotated in its leading dimensions, float32."""
    x, h = x.float(), cos.shape[-1]
    cos, sin = cos[:, None], sin[:, None]
    a, b = (x[..., 0:2 * h:2], x[..., 1:2 * h:2]) if interleaved else (x[..., :h], x[..., h:2 * h])
    ra, rb = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([ra, rb], -1).flatten(-2) if interleaved else torch.cat([ra, rb], -1)
    return torch.cat([turned, x[..., 2 * h:]], -1)


def _turns(s):
    """cos and sin of every row and pair, each pair by the position on its own axis."""
    axes = torch.tensor(s["axes"], device=s["positions"].device)
    pos = s["positions"].long()[axes].T                                    # [N, pairs]
    pair = torch.arange(len(s["axes"]), device=pos.device)[None]
    return s["rotary"][pos, 0, pair], s["rotary"][pos, 1, pair]


def _rotate_plain(s):
    cos, sin = _turns(s)
    return _rotate(s["x"], cos, -sin if s["case"]["inverse"] else sin, s["case"]["interleaved"]).to(s["x"].dtype)


def _store_plain(s, which, x, pages, off):
    if s[which + "s"] is None:
        s[which][pages, :, off] = x.to(s[which].dtype)
        return
    scale = x.abs().amax(-1).clamp(min=2.0 ** -40) / 448.0
    s[which + "s"][pages, :, off] = scale
    s[which].view(torch.uint8)[pages, :, off] = (x / scale[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)


def _append_plain(s):
    case = s["case"]
    req, local = _rows(s["cu"], sum(s["plan"]["nodes"]))
    slots = s["lengths"].long()[req] + local
    pages, off = s["table"][req, slots // case["page"]].long(), slots % case["page"]
    cos, sin = _turns(s)
    q = _rotate(s["q"], cos, sin, case["interleaved"]).to(s["q"].dtype)
    _store_plain(s, "k", _rotate(s["new_k"], cos, sin, case["interleaved"]), pages, off)
    _store_plain(s, "v", s["new_v"].float(), pages, off)
    got = []
    for which in ("k", "v"):
        x = s[which][pages, :, off]
        if s[which + "s"] is not None:
            x = (x.float() * s[which + "s"][pages, :, off][..., None]).to(DTYPES[case["q_dtype"]])
        got.append(x)
    return (q, *got)


def _states(s, which, b, dtype):
    """A request's states [length, kv_heads, head_dim]."""
    at = torch.arange(s["plan"]["ctx"][b], device=s["table"].device)
    pages, off = s["table"][b].long()[at // s["case"]["page"]], at % s["case"]["page"]
    x = s[which][pages, :, off].to(torch.float32).to(dtype)
    return x if s[which + "s"] is None else x * s[which + "s"][pages, :, off].to(dtype)[..., None]


def _scale(case):
    return 1.0 / math.sqrt(case["head_dim"]) if case["scale"] is None else case["scale"]


def _cross_plain(s):
    case, plan = s["case"], s["plan"]
    Hkv, D, g = case["kv_heads"], case["head_dim"], case["heads"] // case["kv_heads"]
    out, first = torch.zeros_like(s["q"]), 0
    for b, (n, L) in enumerate(zip(plan["nodes"], plan["ctx"])):
        if L:
            q = s["q"][first:first + n].float().view(n, Hkv, g, D).permute(1, 0, 2, 3).reshape(Hkv, n * g, D)
            k, v = _states(s, "k", b, torch.float32).permute(1, 2, 0), _states(s, "v", b, torch.float32).transpose(0, 1)
            w = torch.matmul(q, k).mul_(_scale(case))
            if s["mask"] is not None:
                w.masked_fill_(~s["mask"][b, :L], -math.inf)
            w = w.sub_(w.amax(-1, keepdim=True).clamp(min=-3e38)).exp_()
            o = torch.matmul(w, v) / w.sum(-1, keepdim=True).clamp(min=1e-30)
            out[first:first + n] = o.view(Hkv, n, g, D).permute(1, 0, 2, 3).reshape(n, case["heads"], D).to(out.dtype)
        first += n
    return out


# ---- one pass -----------------------------------------------------------------------------------------------------

def run(state):
    s, case = state, state["case"]
    op = case["op"]
    if op in ("logprob", "logprob_grad"):
        if not own:
            return _logprob_plain(s)
        got = s["verifier"].logprobs(s["logits"], s["ids"], rows=s["rows"], T=case["T"], top=case["top"])
        if op == "logprob_grad":
            return got.logprob, got.entropy, s["verifier"].logprobs_grad(
                s["logits"], s["ids"], got, grad_logprob=s["g_logprob"], grad_entropy=s["g_entropy"], T=case["T"])
        return (got.logprob, got.entropy, got.top_ids, got.top_logprobs) if case["top"] else (got.logprob, got.entropy)
    if op == "rotate":
        if own:
            return s["verifier"].rotate(s["x"], s["positions"], s["rotary"], axes=s["axes"], interleaved=case["interleaved"],
                                        inverse=case["inverse"])
        return _rotate_plain(s)
    if op == "append":
        if own:
            q = s["cache"].append(s["new_k"], s["new_v"], s["table"], s["lengths"], s["cu"], q=s["q"], rotary=s["rotary"],
                                  interleaved=case["interleaved"], positions=s["positions"], axes=s["axes"])
            return (q, *s["cache"].read(s["table"], s["lengths"], s["cu"], n_rows=sum(s["plan"]["nodes"]), dtype=s["q"].dtype))
        return _append_plain(s)
    if own:
        return s["cache"].cross_attend(s["q"], s["table"], s["lengths"], s["cu"], mask=s["mask"], scale=_scale(case))
    return _cross_plain(s)


# ---- what a pass cannot do without --------------------------------------------------------------------------------

def work(case):
    plan = _plan_of(case)
    size = {"bf16": 2, "f16": 2, "f32": 4}
    if case["op"] in ("logprob", "logprob_grad"):
        live, each = sum(plan["kept"]) * case["V"], size[case["dtype"]]
        written = sum(plan["nodes"]) * case["V"] if case["op"] == "logprob_grad" else 0    # rows without a token are zeros
        return {"bytes": float((live + written) * each + 8 * sum(plan["nodes"])), "flops": 5.0 * live}
    D, H = case["head_dim"], case["heads"]
    if case["op"] == "rotate":
        return {"bytes": 4.0 * case["N"] * H * D + 4.0 * case["N"] * len(case["sections"].split(",")),
                "flops": 6.0 * case["N"] * H * len(_axes(case))}
    Hkv = case["kv_heads"]
    cached = 2 * Hkv * (D + 4 if case["cache"] == "e4m3" else 2 * D)     # a cache row of k and v, with its scales
    dense = 2 * Hkv * D * 2                                              # the same as 16-bit tensors
    nodes, ctx = sum(plan["nodes"]), sum(plan["ctx"])
    if case["op"] == "append":
        return {"bytes": float(nodes * (dense + cached + 4 * H * D + cached + dense)), "flops": 6.0 * nodes * (H + Hkv) * len(_axes(case))}
    pairs = sum(n * c for n, c in zip(plan["nodes"], plan["ctx"]))
    return {"bytes": float(max(1, ctx) * cached + 4 * nodes * H * D), "flops": 4.0 * D * H * pairs}


# ---- the definitions, in 64 bits ----------------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("logprob", "logprob_grad"):
        return _exact_logprob(s)
    if case["op"] == "rotate":
        return _exact_turn(s["x"].double(), s, -1.0 if case["inverse"] else 1.0)
    plan = s["plan"]
    if case["op"] == "append":
        k, v = _exact_turn(s["new_k"].double(), s, 1.0), s["new_v"].double()
        if case["cache"] == "e4m3":
            k, v = (_exact_8_bits(x) for x in (k, v))
        return _exact_turn(s["q"].double(), s, 1.0), k, v
    out, first = [], 0
    for b in range(case["B"]):
        n, L = plan["nodes"][b], plan["ctx"][b]
        q = s["q"][first:first + n].double()
        first += n
        see = torch.ones(L, dtype=torch.bool, device=q.device) if s["mask"] is None else s["mask"][b, :L]
        if not bool(see.any()):
            out.append(torch.zeros_like(q))
            continue
        k, v = _states(s, "k", b, torch.float64)[see], _states(s, "v", b, torch.float64)[see]
        heads = []
        for h in range(case["heads"]):
            at = h // (case["heads"] // case["kv_heads"])
            z = (q[:, h] @ k[:, at].T) * _scale(case)
            e = (z - z.max(1, keepdim=True).values).exp()
            heads.append((e @ v[:, at]) / e.sum(1, keepdim=True))
        out.append(torch.stack(heads, 1))
    return torch.cat(out)


def _exact_8_bits(x):
    scale = x.abs().amax(-1, keepdim=True).clamp(min=2.0 ** -40) / 448.0
    return (x / scale).to(torch.float8_e4m3fn).double() * scale


def _exact_turn(x, s, way):
    x, half = x.clone(), len(s["axes"])
    for i, a in enumerate(s["axes"]):
        turn = s["positions"][a].double() * 10000.0 ** (-2.0 * i / (2 * half)) * way
        p, q = (2 * i, 2 * i + 1) if s["case"]["interleaved"] else (i, i + half)
        u, w = x[..., p].clone(), x[..., q].clone()
        x[..., p] = u * turn.cos()[:, None] - w * turn.sin()[:, None]
        x[..., q] = w * turn.cos()[:, None] + u * turn.sin()[:, None]
    return x


def _exact_logprob(s):
    case, M = s["case"], s["ids"].numel()
    z = lambda *n: torch.zeros(*n, dtype=torch.float64, device=s["ids"].device)
    lp, entropy, top = z(M), z(M), z(M, case["top"])
    grad = z(*s["logits"].shape) if case["op"] == "logprob_grad" else None
    live = (s["ids"] >= 0).nonzero()[:, 0]
    for at in live.split(max(1, (1 << 27) // case["V"])):
        row = at if s["rows"] is None else s["rows"][at].long()
        a = torch.log_softmax(s["logits"][row].double() / case["T"], 1)
        p = a.exp()
        took = s["ids"][at].long()[:, None]
        lp[at] = a.gather(1, took)[:, 0]
        entropy[at] = torch.special.entr(p).sum(1)
        if case["top"]:
            n = min(case["top"], case["V"])
            top[at] = -math.inf
            top[at, :n] = a.sort(1, descending=True).values[:, :n]
        if grad is not None:
            g, h = s["g_logprob"].double()[at, None], s["g_entropy"].double()[at, None]
            one = torch.zeros_like(p).scatter_(1, took, 1.0)
            dent = torch.special.entr(p) - p * entropy[at, None]          # -p (ln p + H)
            grad[row] = (g * (one - p) + h * dent) / case["T"]
    out = [lp, entropy]
    if case["top"]:
        out += [None, top]
    return out + ([] if grad is None else [grad])
