"""The operators of a hybrid target's attention layers and of sampled
acceptance, as a measured set: what each is given, one pass through it in plain
torch operations or through the library, and its result in 64 bits.

Operators (the case's "op"):
  sample   drafted tokens verified against the target's probabilities, from
           given random numbers (chains and trees, sampled or fixed drafts)
  norm     per-head RMS norm of queries and keys with the rotary embedding, the
           new keys and values written to the paged cache
  attn     attention of a drafted chain or tree over the paged cache
  commit   the accepted root path's rows moved together in the cache
  pages    pages of the cache given back, forked and taken
"""
import random

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # a chain of four sampled drafts on the tiny vocabulary: latency alone
        dict(name="sample_chain_small", op="sample", batch=1, nodes=5, vocab=1024, tree=False, drawn=True),
        # one request's span of 16 with the draft's distributions at the full vocabulary
        dict(name="sample_chain_span16", op="sample", batch=1, nodes=17, vocab=151936, tree=False, drawn=True),
        # sixteen requests' trees of fixed candidates (a greedy or top-k draft)
        dict(name="sample_tree_batch16", op="sample", batch=16, nodes=23, vocab=151936, tree=True, drawn=False),
        # one new token of one request, a quarter of a large head rotated
        dict(name="norm_one_token", op="norm", batch=1, tok=1, h_q=16, h_kv=2, d=256, rot=64, page=16, ctx=500,
             dtype="bf16", tree=False, pairs=False),
        # two prompts of odd length going into the cache
        dict(name="norm_prompt_4001", op="norm", batch=2, tok=4001, h_q=32, h_kv=8, d=128, rot=128, page=64, ctx=37,
             dtype="bf16", tree=False, pairs=False),
        # plain decoding: one token over a short context
        dict(name="attn_one_token_777", op="attn", batch=1, tok=1, h_q=16, h_kv=2, d=128, page=16, ctx=777,
             dtype="bf16", tree=False),
        # one request's tree of 22 drafted nodes over a long context, large heads
        dict(name="attn_tree22_32k", op="attn", batch=1, tok=22, h_q=16, h_kv=2, d=256, page=64, ctx=32501,
             dtype="bf16", tree=True),
        # sixteen requests of different lengths, spans of 16
        dict(name="attn_span16_batch16", op="attn", batch=16, tok=16, h_q=32, h_kv=8, d=128, page=32, ctx=8000,
             dtype="bf16", tree=False),
        # a small tree's accepted path in one f32 layer
        dict(name="commit_small", op="commit", batch=1, nodes=5, layers=1, h_kv=2, d=64, page=16, ctx=100,
             dtype="f32"),
        # sixteen requests' accepted paths through sixteen layers
        dict(name="commit_batch16", op="commit", batch=16, nodes=23, layers=16, h_kv=8, d=128, page=64, ctx=900,
             dtype="bf16"),
        # one request forked once
        dict(name="pages_one_fork", op="pages", forks=1, tok=5, layers=1, h_kv=2, d=128, page=16, ctx=300,
             dtype="bf16"),
        # sixteen requests forked, the losers' pages given back first
        dict(name="pages_16_forks", op="pages", forks=16, tok=22, layers=8, h_kv=4, d=128, page=64, ctx=8000,
             dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(("sample", "sample", "norm", "attn", "attn", "commit", "pages"))
    most = max(_cost(c) for c in listed() if c["op"] == op)
    while True:
        d = rng.choice((64, 128, 256))
        h_kv, group = rng.choice((1, 2, 4, 8)), rng.choice((1, 2, 3, 4, 6, 8))
        dtype = rng.choice(("bf16", "bf16", "f32"))
        page = rng.choice((16, 32, 64, 128))
        if op == "sample":
            c = dict(op=op, batch=_log(rng, 1, 24), nodes=_log(rng, 2, 65), vocab=_log(rng, 700, 151936),
                     tree=rng.random() < 0.5, drawn=rng.random() < 0.5)
        elif op == "norm":
            tok = _log(rng, 1, 6000)
            c = dict(op=op, batch=_log(rng, 1, 32), tok=tok, h_q=h_kv * group, h_kv=h_kv, d=d,
                     rot=rng.choice((d, d // 2, d // 4)), page=page, ctx=_log(rng, 1, 4000), dtype=dtype,
                     tree=tok <= 64 and rng.random() < 0.5, pairs=rng.random() < 0.3)
        elif op == "attn":
            c = dict(op=op, batch=_log(rng, 1, 32), tok=_log(rng, 1, 64), h_q=h_kv * group, h_kv=h_kv, d=d, page=page,
                     ctx=_log(rng, 30, 65000), dtype=dtype, tree=rng.random() < 0.6)
        elif op == "commit":
            c = dict(op=op, batch=_log(rng, 1, 32), nodes=_log(rng, 2, 65), layers=_log(rng, 1, 16), h_kv=h_kv, d=d,
                     page=page, ctx=_log(rng, 10, 2000), dtype=dtype)
        else:
            c = dict(op=op, forks=_log(rng, 1, 32), tok=_log(rng, 1, 64), layers=_log(rng, 1, 8), h_kv=h_kv, d=d,
                     page=page, ctx=_log(rng, 20, 9000), dtype=dtype)
        if _cost(c) <= most and _pool_bytes(c) <= 2.5e9:
            return c


def _cost(c):
    """What a drawn case is held against the listed ones by."""
    w = work(c)
    if c["op"] == "attn":
        slow = 8 if c["dtype"] == "f32" else 1          # 32-bit products run at a fraction of the 16-bit rate
        return max(w["bytes"], w["flops"] * slow / 100)
    return max(w["bytes"], _pool_bytes(c)) if c["op"] in ("commit", "pages") else w["bytes"]


# ---------------------------------------------------------------- shapes

def _lengths(c):
    """Committed tokens of each request: the case's length for the first, other lengths below it."""
    n = 2 * c["forks"] if c["op"] == "pages" else c["batch"]
    r = random.Random(c["ctx"] * 1000 + n)
    return [c["ctx"]] + [r.randint(c["ctx"] // 2, c["ctx"]) for _ in range(n - 1)]


def _new(c):
    return c["nodes"] - 1 if c["op"] == "commit" else c["tok"]


def _width(c):
    return -(-(c["ctx"] + _new(c)) // c["page"])


def _n_pages(c):
    used = sum(-(-(n + _new(c)) // c["page"]) for n in _lengths(c))
    return used + 3


def _pool_bytes(c):
    if c["op"] == "sample":
        return 0
    return 2 * c.get("layers", 1) * _n_pages(c) * c["h_kv"] * c["page"] * c["d"] * (4 if c["dtype"] == "f32" else 2)


def work(c):
    e = 4 if c.get("dtype") == "f32" else 2
    if c["op"] == "sample":
        b, n, v = c["batch"], c["nodes"], c["vocab"]
        read = b * n * v + b * v + (b * v if c["drawn"] else 0) + 3 * b * n
        return {"bytes": 4 * read, "flops": 4 * b * n * v}
    if c["op"] == "norm":
        t = c["batch"] * c["tok"]
        row = (c["h_q"] + 2 * c["h_kv"]) * c["d"]
        return {"bytes": 2 * e * t * row + 4 * t * c["rot"], "flops": 8 * t * row}
    if c["op"] == "attn":
        lens, t, d = _lengths(c), c["tok"], c["d"]
        kv = sum(n + t for n in lens) * c["h_kv"] * d * 2
        pairs = sum(n * t + t * (t + 1) // 2 for n in lens)
        return {"bytes": e * (kv + 2 * c["batch"] * t * c["h_q"] * d), "flops": 4 * pairs * c["h_q"] * d}
    if c["op"] == "commit":
        rows = c["batch"] * max(1, _depth_wanted(c))
        return {"bytes": 4 * e * rows * c["layers"] * c["h_kv"] * c["d"], "flops": 0}
    lens = _lengths(c)[:c["forks"]]
    tail = sum(n % c["page"] for n in lens)
    tables = 8 * sum(-(-n // c["page"]) for n in lens) * 4
    return {"bytes": 4 * e * tail * c["layers"] * c["h_kv"] * c["d"] + tables, "flops": 0}


def _depth_wanted(c):
    return (c["nodes"] - 1) // 2


# ---------------------------------------------------------------- inputs

def _parents(rng, batch, nodes, tree, straight=0.4):
    """Parent arrays as a draft's tree has them: often the node before, else any earlier one."""
    p = np.empty((batch, nodes), np.int32)
    for b in range(batch):
        for i in range(nodes):
            p[b, i] = i - 1 if not tree or rng.random() < straight else rng.randrange(i) if i else -1
    return p


def _dev(x, dtype=None):
    return torch.as_tensor(np.asarray(x), dtype=dtype).cuda()


def _cache(c, seed, g, width=None, live=None):
    """A pool of pages, a table that deals them out at random, and the lengths."""
    rng = random.Random(seed)
    lens = _lengths(c)
    width, total = width or _width(c), _n_pages(c)
    order = list(range(total))
    rng.shuffle(order)
    table = np.full((len(lens), width), -1, np.int32)
    at = 0
    for b, n in enumerate(lens):
        k = -(-(n + (_new(c) if live is None else live)) // c["page"])
        table[b, :k] = order[at:at + k]
        at += k
    dt = TYPES[c["dtype"]]
    shape = (c.get("layers", 1), total, c["h_kv"], c["page"], c["d"])
    return {"k": torch.randn(shape, device="cuda", dtype=dt, generator=g),
            "v": torch.randn(shape, device="cuda", dtype=dt, generator=g),
            "table": _dev(table), "ctx": _dev(lens, torch.int32)}


def prepare(c, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    rng = random.Random(seed)
    s = {"case": dict(c)}

    def normal(*shape, dtype=torch.float32):
        return torch.randn(shape, device="cuda", dtype=dtype, generator=g)

    def uniform(*shape):
        return torch.rand(shape, device="cuda", generator=g)

    if c["op"] == "sample":
        b, n, v = c["batch"], c["nodes"], c["vocab"]
        parent = _parents(rng, b, n, c["tree"])
        s["parent_host"], s["parent"] = parent, _dev(parent)
        s["tree"] = c["tree"]
        up = s["parent"][:, 1:].long()
        logits = normal(b, n, v)
        # a few likely tokens in each row, as a language model's logits have
        top = torch.randint(0, v, (b, n, 6), device="cuda", generator=g)
        logits.scatter_(2, top, 12.0 + 2.0 * normal(b, n, 6))
        s["logits"] = logits
        s["temperature"] = 0.7 + 0.6 * uniform(b)
        if c["drawn"]:
            q = (logits[:, :n - 1] + 0.4 * normal(b, n - 1, v)) / s["temperature"][:, None, None]
            q = torch.exp(q - q.amax(-1, keepdim=True))
            q /= q.sum(-1, keepdim=True)
            s["q"] = q
            tok = torch.empty((b, n - 1), device="cuda", dtype=torch.int64)
            for i in range(n - 1):
                row = q[torch.arange(b, device="cuda"), up[:, i]]
                tok[:, i] = torch.argmax(row / _noise(uniform(b, v)), -1)
        else:
            s["q"] = None
            # candidates from the likely tokens of the parent's row, the likelier the oftener
            row = top[torch.arange(b, device="cuda")[:, None], up]
            score = logits[torch.arange(b, device="cuda")[:, None], up].gather(2, row) / s["temperature"][:, None, None]
            which = torch.argmax(score - torch.log(_noise(uniform(b, n - 1, 6))), -1)
            tok = row.gather(2, which[:, :, None])[:, :, 0]
        s["tokens"] = torch.cat([torch.zeros_like(tok[:, :1]), tok], 1).int().contiguous()
        s["uniforms"] = uniform(b, n)
        s["noise"] = _noise(uniform(b, v))
        s["most_children"] = int(max(np.bincount(p[1:], minlength=1).max() for p in parent))
        return s

    dt = TYPES[c["dtype"]]
    if c["op"] == "norm":
        s.update(_cache(c, seed, g))
        b, t, d = c["batch"], c["tok"], c["d"]
        parent = _parents(rng, b, t + 1, True) if c["tree"] else None
        s["parent"] = None if parent is None else _dev(parent)
        s["qkv"] = normal(b, t, (c["h_q"] + 2 * c["h_kv"]) * d, dtype=dt)
        s["q_norm"], s["k_norm"] = 0.1 * normal(d).to(dt), 0.1 * normal(d).to(dt)
        far = c["ctx"] + t
        inv = 10000.0 ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64) / c["rot"])
        angle = torch.arange(far, dtype=torch.float64)[:, None] * inv
        s["rope"] = torch.cat([angle.cos(), angle.sin()], 1).float().cuda()
        s["out"] = torch.empty((b, t, c["h_q"], d), device="cuda", dtype=dt)
        return s
    if c["op"] == "attn":
        s.update(_cache(c, seed, g))
        b, t = c["batch"], c["tok"]
        parent = _parents(rng, b, t + 1, c["tree"])
        s["tree"], s["parent_host"], s["parent"] = c["tree"], parent, _dev(parent)
        # queries and keys as norms leave them, queries a little longer: peaks as well as flat rows
        s["q"] = (1.5 * normal(b, t, c["h_q"], c["d"])).to(dt)
        s["out"] = torch.empty_like(s["q"])
        return s
    if c["op"] == "commit":
        s.update(_cache(c, seed, g))
        parent = _parents(rng, c["batch"], c["nodes"], True, 0.6)
        s["parent"] = _dev(parent)
        nodes = []
        for p in parent:
            depth = np.zeros(len(p), int)
            for i in range(1, len(p)):
                depth[i] = depth[p[i]] + 1
            nodes.append(int(np.argmin(np.abs(depth - _depth_wanted(c)))))   # about half the tree's nodes deep, where it is
        s["node"] = _dev(nodes, torch.int32)
        s["ctx_out"] = torch.empty_like(s["ctx"])
        return s
    # the first half of the requests are forked into the second half, which hold pages of their own from before
    s.update(_cache(c, seed, g, live=0))
    n = c["forks"]
    ref = torch.zeros(_n_pages(c), dtype=torch.int32)
    ids = s["table"].cpu().flatten()
    ref[ids[ids >= 0].long()] = 1
    s["ref"] = ref.cuda()
    s["src"], s["dst"] = _dev(np.arange(n), torch.int32), _dev(np.arange(n, 2 * n), torch.int32)
    s["give_back"] = _dev([-1] * n + [0] * n, torch.int32)
    s["more"] = c["tok"]
    return s


def _noise(u):
    """Exponential random numbers of uniform ones, never zero."""
    return -torch.log1p(-u.clamp(max=1 - 2.0 ** -24)) + 1e-10


# ---------------------------------------------------------------- plain forms

def _ancestors(parent):
    """[B][N][N]: whether j is on the root path of i (i's own place included)."""
    n = parent.shape[1]
    step = torch.zeros(parent.shape[0], n, n + 1, device=parent.device)
    step.scatter_(2, torch.where(parent < 0, n, parent).long()[:, :, None], 1.0)
    reach = step[:, :, :n] + torch.eye(n, device=parent.device)
    for _ in range(max(1, n - 1).bit_length()):
        reach = ((reach @ reach) > 0).float()
    return reach > 0


def _depths(parent, batch, tok):
    """[B][T]: distance of node t + 1 from the root."""
    if parent is None:
        return torch.arange(1, tok + 1, device="cuda").expand(batch, tok)
    return _ancestors(parent).sum(-1)[:, 1:] - 1


def _plain_sample(s):
    b, n, v = s["logits"].shape
    z = s["logits"] / s["temperature"][:, None, None]
    p = torch.exp(z - z.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    parent = s["parent"].long()
    up, tok, u = parent[:, 1:], s["tokens"][:, 1:].long(), s["uniforms"][:, 1:]
    at = torch.arange(b, device="cuda")
    pt = p[at[:, None], up, tok]
    order = torch.arange(n - 1, device="cuda")
    before = (up[:, :, None] == up[:, None, :]) & (order[None, None, :] < order[None, :, None])   # j an earlier sibling of i
    if s["q"] is None:
        same = tok[:, :, None] == tok[:, None, :]
        left = torch.where((before & same).any(-1), 0.0, pt)
        gone = (before * left[:, None, :]).sum(-1)
        test = u * (1.0 - gone) < left
    else:
        q = s["q"]
        rank = before.sum(-1)
        qt = q[at[:, None], up, tok]
        coef, mass = torch.zeros_like(pt), torch.ones_like(pt)
        # each rejected sibling turns p - c q into p - (c + S) q, S its positive part's sum
        for k in range(1, s["most_children"] + 1):
            prev = (before & (rank[:, None, :] == k - 1)).float()
            c2 = (prev * (coef + mass)[:, None, :]).sum(-1)
            if k < s["most_children"]:
                row = p[at[:, None], up] - c2[:, :, None] * q[at[:, None], up]
                coef = torch.where(rank == k, c2, coef)
                mass = torch.where(rank == k, row.clamp(min=0).sum(-1), mass)
        test = u * qt * mass < (pt - coef * qt).clamp(min=0)
    chosen = test & ~(before & test[:, None, :]).any(-1)
    anc = _ancestors(s["parent"])[:, 1:, 1:]
    reached = ~(anc & ~chosen[:, None, :]).any(-1)
    length = reached.sum(-1)
    node = torch.where(length > 0, (reached * (order + 1)).amax(-1), torch.zeros_like(length))
    pa = p[at, node]
    mine = up == node[:, None]
    if s["q"] is None:
        gone = torch.zeros((b, v), device="cuda").scatter_add_(1, tok, mine.float())
        w = torch.where(gone > 0, 0.0, pa)
    else:
        last = mine & (rank == (rank * mine).amax(-1, keepdim=True))
        c2 = (last * (coef + mass)).sum(-1)
        w = (pa - c2[:, None] * s["q"][at, node.clamp(max=n - 2)]).clamp(min=0)
    w = torch.where(w.amax(-1, keepdim=True) > 0, w, pa)
    token = torch.argmax(w / s["noise"], -1)
    prob = torch.cat([pa.gather(1, token[:, None]), pt], 1)
    return {"accept_len": length.int(), "accept_node": node.int(), "next_token": token.int(), "token_prob": prob}


def _rows_of(table, slot, page):
    """Page and offset of token slots [B][...]."""
    return table.gather(1, (slot // page).clamp(max=table.shape[1] - 1)).long(), slot % page


def _plain_norm(s):
    c = s["case"]
    b, t, d, hq, hk, half = c["batch"], c["tok"], c["d"], c["h_q"], c["h_kv"], c["rot"] // 2
    x = s["qkv"].float().view(b, t, hq + 2 * hk, d)
    w = torch.cat([s["q_norm"].float().expand(hq, d), s["k_norm"].float().expand(hk, d)]) + 1.0
    y = x[:, :, :hq + hk]
    y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6) * w
    slot = s["ctx"].long()[:, None] + torch.arange(t, device="cuda")
    pos = s["ctx"].long()[:, None] + _depths(s["parent"], b, t) - 1
    table = s["rope"][pos][:, :, None]
    cos, sin = table[..., :half], table[..., half:]
    head, tail = y[..., :2 * half], y[..., 2 * half:]
    if c["pairs"]:
        x0, x1 = head[..., 0::2], head[..., 1::2]
        turned = torch.stack([x0 * cos - x1 * sin, x1 * cos + x0 * sin], -1).flatten(-2)
    else:
        x0, x1 = head[..., :half], head[..., half:]
        turned = torch.cat([x0 * cos - x1 * sin, x1 * cos + x0 * sin], -1)
    y = torch.cat([turned, tail], -1)
    s["out"].copy_(y[:, :, :hq])
    page, off = _rows_of(s["table"], slot, c["page"])
    s["k"][0][page, :, off] = y[:, :, hq:].to(s["k"].dtype)
    s["v"][0][page, :, off] = x[:, :, hq + hk:].to(s["v"].dtype)
    return {"q": s["out"], "k": s["k"], "v": s["v"]}


def _plain_attn(s):
    c = s["case"]
    b, t, d, hq, hk = c["batch"], c["tok"], c["d"], c["h_q"], c["h_kv"]
    ids = s["table"].clamp(min=0).long()
    k = s["k"][0][ids].float().permute(0, 2, 1, 3, 4).reshape(b, hk, -1, d)
    v = s["v"][0][ids].float().permute(0, 2, 1, 3, 4).reshape(b, hk, -1, d)
    slots = k.shape[2]
    q = s["q"].float().view(b, t, hk, hq // hk, d).permute(0, 2, 1, 3, 4).reshape(b, hk, -1, d)
    score = (q @ k.transpose(2, 3)).view(b, hk, t, hq // hk, slots) * d ** -0.5
    anc = _ancestors(s["parent"])[:, 1:, 1:]
    rel = torch.arange(slots, device="cuda") - s["ctx"][:, None]
    seen = anc.gather(2, rel.clamp(0, t - 1)[:, None, :].expand(b, t, slots)) & (rel < t)[:, None, :]
    seen = seen | (rel < 0)[:, None, :]
    score = torch.where(seen[:, None, :, None, :], score, float("-inf"))
    p = torch.exp(score - score.amax(-1, keepdim=True))
    o = (p / p.sum(-1, keepdim=True)).view(b, hk, -1, slots) @ v
    return o.view(b, hk, t, hq // hk, d).permute(0, 2, 1, 3, 4).reshape(b, t, hq, d).to(s["q"].dtype)


def _plain_commit(s):
    c = s["case"]
    t = c["nodes"] - 1
    anc = _ancestors(s["parent"])
    depth = anc.sum(-1) - 1
    b = torch.arange(c["batch"], device="cuda")
    node = s["node"].long()
    path, length = anc[b, node], depth[b, node]
    # the node that goes to each of the T drafted slots: the path's at that depth, else the one that is there
    goal = torch.arange(1, t + 1, device="cuda")
    hit = path[:, None, :] & (depth[:, None, :] == goal[None, :, None])
    source = torch.where(goal[None] <= length[:, None], hit.float().argmax(-1), goal[None])
    base = s["ctx"].long()[:, None] - 1
    sp, so = _rows_of(s["table"], base + source, c["page"])
    dp, do = _rows_of(s["table"], base + goal[None], c["page"])
    for pool in (s["k"], s["v"]):
        pool[:, dp, :, do] = pool[:, sp, :, so]
    s["ctx_out"].copy_(s["ctx"] + length)
    return {"k": s["k"], "v": s["v"], "ctx": s["ctx_out"]}


def _free_first(ref):
    return torch.sort((ref != 0).int(), stable=True).indices.int()


def _plain_resize(s, want):
    """Each request's table cut or grown to `want` tokens (below zero: as it is)."""
    table, ref, page = s["table"], s["ref"], s["case"]["page"]
    keep = torch.where(want >= 0, (want + page - 1) // page, table.shape[1])[:, None]
    col = torch.arange(table.shape[1], device="cuda")[None]
    gone = (col >= keep) & (table >= 0)
    ref.index_add_(0, table.clamp(min=0).flatten(), -gone.int().flatten())
    table.masked_fill_(gone, -1)
    need = (col < keep) & (table < 0) & (want >= 0)[:, None]
    rank = torch.cumsum(need.flatten(), 0).view_as(need) - 1
    new = _free_first(ref)[rank.clamp(0, ref.numel() - 1)]
    table.copy_(torch.where(need, new, table))
    ref.index_add_(0, new.flatten(), need.int().flatten())


def _plain_fork(s):
    c = s["case"]
    table, ref, page, src, dst = s["table"], s["ref"], c["page"], s["src"].long(), s["dst"].long()
    n = s["ctx"][src]
    full, tail = n // page, n % page
    col = torch.arange(table.shape[1], device="cuda")[None]
    need = tail > 0
    new = _free_first(ref)[(torch.cumsum(need, 0) - 1).clamp(min=0)]
    old = table[src]
    rows = torch.where(col < full[:, None], old, -1)
    ref.index_add_(0, rows.clamp(min=0).flatten(), (rows >= 0).int().flatten())
    ref.index_add_(0, new, need.int())
    # without a tail nothing is copied: the last full page onto itself
    last = old.gather(1, torch.where(need, full, (full - 1).clamp(min=0)).long()[:, None])[:, 0]
    table[dst] = torch.where((col == full[:, None]) & need[:, None], new[:, None], rows)
    s["ctx"][dst] = n
    live = (torch.arange(page, device="cuda")[None] < tail[:, None])[None, :, None, :, None]
    for pool in (s["k"], s["v"]):
        a, z = last.long(), torch.where(need, new, last).long()
        pool[:, z] = torch.where(live, pool[:, a], pool[:, z])


def _plain_pages(s):
    _plain_resize(s, s["give_back"])
    _plain_fork(s)
    _plain_resize(s, s["ctx"] + s["more"])
    return {"table": s["table"], "ref": s["ref"], "ctx": s["ctx"], "k": s["k"], "v": s["v"]}


# ---------------------------------------------------------------- the library

def _kept(s):
    """What a program keeps beside its data: the dimensions, a workspace, a status word."""
    if "kept" not in s:
        from speculative_decode_hybrid_gb300 import gdnspec as G
        c, kept = s["case"], {"G": G}
        if c["op"] == "sample":
            b, n, _ = s["logits"].shape
            bytes_ = G.spec_accept_sample_workspace_bytes(b, n)
        else:
            rows = s["table"].shape[0]
            kept["dims"] = G.make_attn_dims(rows, c.get("layers", 1), c.get("h_q", c["h_kv"]), c["h_kv"], c["d"], c["page"],
                                            s["k"].shape[1], s["table"].shape[1],
                                            G.GDN_BF16 if c["dtype"] == "bf16" else G.GDN_F32)
            bytes_ = (G.attn_workspace_bytes(kept["dims"], c["tok"]) if c["op"] == "attn" else
                      G.kv_pages_workspace_bytes(kept["dims"]) if c["op"] == "pages" else 0)
        kept["ws_bytes"] = bytes_
        kept["ws"] = torch.zeros(max(bytes_, 1), dtype=torch.uint8, device="cuda")
        kept["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        s["kept"] = kept
    return s["kept"]


def _own_run(s):
    c, kept = s["case"], _kept(s)
    G, ws, wsb, status = kept["G"], kept["ws"], kept["ws_bytes"], kept["status"]
    if c["op"] == "sample":
        b, n, v = s["logits"].shape
        ints = torch.empty((3, b), dtype=torch.int32, device="cuda")
        prob = torch.empty((b, n), dtype=torch.float32, device="cuda")
        G.spec_accept_sample(b, n, v, s["logits"], s["q"], s["tokens"], s["parent"] if s["tree"] else None,
                             s["temperature"], s["uniforms"], s["noise"], ints[0], ints[1], ints[2], prob, ws, wsb, status)
        return {"accept_len": ints[0], "accept_node": ints[1], "next_token": ints[2], "token_prob": prob}
    dims = kept["dims"]
    if c["op"] == "norm":
        G.attn_qk_norm_rope(dims, c["tok"], s["qkv"], s["qkv"].shape[-1], s["q_norm"], s["k_norm"], 1e-6, 1.0, s["rope"],
                            c["rot"], s["rope"].shape[0], s["parent"], s["ctx"], s["table"], s["out"], s["k"], s["v"],
                            status, flags=G.GDN_ROPE_PAIRS if c["pairs"] else 0)
        return {"q": s["out"], "k": s["k"], "v": s["v"]}
    if c["op"] == "attn":
        if s["tree"]:
            G.attn_tree_verify(dims, c["tok"] + 1, s["parent_host"], s["parent"], s["q"], s["k"], s["v"], s["table"],
                               s["ctx"], c["d"] ** -0.5, s["out"], ws, wsb, status)
        else:
            G.attn_verify_span(dims, c["tok"], s["q"], s["k"], s["v"], s["table"], s["ctx"], c["d"] ** -0.5, s["out"],
                               ws, wsb, status)
        return s["out"]
    if c["op"] == "commit":
        G.kv_commit_path(dims, c["nodes"], s["parent"], s["node"], s["ctx"], s["table"], s["k"], s["v"], s["ctx_out"], status)
        return {"k": s["k"], "v": s["v"], "ctx": s["ctx_out"]}
    G.kv_pages_resize(dims, s["give_back"], s["table"], s["ref"], ws, wsb, status)
    G.kv_pages_fork(dims, c["forks"], s["src"], s["dst"], s["table"], s["ctx"], s["ref"], s["k"], s["v"], ws, wsb, status)
    G.kv_pages_resize(dims, s["ctx"] + s["more"], s["table"], s["ref"], ws, wsb, status)
    return {"table": s["table"], "ref": s["ref"], "ctx": s["ctx"], "k": s["k"], "v": s["v"]}


def run(s):
    if own:
        return _own_run(s)
    return {"sample": _plain_sample, "norm": _plain_norm, "attn": _plain_attn, "commit": _plain_commit,
            "pages": _plain_pages}[s["case"]["op"]](s)


# ---------------------------------------------------------------- in 64 bits

def _path(parent, i):
    """Nodes from below the root to i."""
    got = []
    while i > 0:
        got.append(i)
        i = int(parent[i])
    return got[::-1]


def _exact_sample(s):
    b, n, v = s["logits"].shape
    lens, nodes, tokens, probs = [], [], [], []
    for r in range(b):
        p = torch.softmax(s["logits"][r].double() / float(s["temperature"][r]), -1)
        parent, tok = s["parent_host"][r], s["tokens"][r].tolist()
        u = s["uniforms"][r].tolist()
        prob = [0.0] + [float(p[parent[i], tok[i]]) for i in range(1, n)]
        at = depth = 0
        while True:
            rest, hit = p[at].clone(), None
            for i in [j for j in range(1, n) if parent[j] == at]:
                x = tok[i]
                if s["q"] is None:
                    if u[i] < float(rest[x]) / max(float(rest.sum()), 1e-300):
                        hit = i
                        break
                    rest[x] = 0.0
                else:
                    q = s["q"][r, at].double()
                    if u[i] < float(rest[x]) / max(float(q[x]), 1e-300):
                        hit = i
                        break
                    rest = (rest - q).clamp(min=0)
                    rest = rest / rest.sum().clamp(min=1e-300)
            if hit is None:
                break
            at, depth = hit, depth + 1
        rest = rest if float(rest.max()) > 0 else p[at]
        token = int(torch.argmax(rest / s["noise"][r].double()))
        prob[0] = float(p[at, token])
        lens.append(depth), nodes.append(at), tokens.append(token), probs.append(prob)
    return {"accept_len": np.array(lens, np.int32), "accept_node": np.array(nodes, np.int32),
            "next_token": np.array(tokens, np.int32), "token_prob": np.array(probs, np.float64)}


def _exact_norm(s):
    c = s["case"]
    d, hq, hk, half = c["d"], c["h_q"], c["h_kv"], c["rot"] // 2
    out_q, k, v = s["out"].double(), s["k"].double(), s["v"].double()
    for r, n in enumerate(s["ctx"].tolist()):
        parent = None if s["parent"] is None else s["parent"][r].tolist()
        x = s["qkv"][r].double().view(c["tok"], -1, d)
        where = torch.arange(c["tok"], device="cuda") if parent is None else \
            torch.tensor([len(_path(parent, t + 1)) - 1 for t in range(c["tok"])], device="cuda")
        angle = s["rope"].double()[n + where]
        for h in range(hq + hk):
            y = x[:, h]
            y = y / torch.sqrt(y.pow(2).mean(-1, keepdim=True) + 1e-6)
            y = y * (1.0 + (s["q_norm"] if h < hq else s["k_norm"]).double())
            i0 = torch.arange(half, device="cuda") * (2 if c["pairs"] else 1)
            i1 = i0 + (1 if c["pairs"] else half)
            turn = torch.complex(angle[:, :half], angle[:, half:]) * torch.complex(y[:, i0], y[:, i1])
            y[:, i0], y[:, i1] = turn.real, turn.imag
            x[:, h] = y
        out_q[r] = x[:, :hq]
        at = n + torch.arange(c["tok"], device="cuda")
        page = s["table"][r].long()[at // c["page"]]
        k[0, page, :, at % c["page"]] = x[:, hq:hq + hk]
        v[0, page, :, at % c["page"]] = x[:, hq + hk:]
    return {"q": out_q, "k": k, "v": v}


def _exact_attn(s):
    c = s["case"]
    group, out = c["h_q"] // c["h_kv"], torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    for r, n in enumerate(s["ctx"].tolist()):
        at = torch.arange(n + c["tok"], device="cuda")
        page = s["table"][r].long()[at // c["page"]]
        hide = torch.ones((c["tok"], n + c["tok"]), dtype=torch.bool)
        hide[:, :n] = False
        for t in range(c["tok"]):
            hide[t, [n + i - 1 for i in _path(s["parent_host"][r], t + 1)]] = False
        hide = hide.cuda()
        for h in range(c["h_kv"]):
            k, v = (s[m][0, page, h, at % c["page"]].double() for m in "kv")
            for j in range(group):
                a = s["q"][r, :, h * group + j].double() @ k.T / c["d"] ** 0.5
                out[r, :, h * group + j] = torch.softmax(a.masked_fill(hide, float("-inf")), -1) @ v
    return out


def _exact_commit(s):
    page, parent = s["case"]["page"], s["parent"].tolist()
    k, v, ctx = s["k"].double(), s["v"].double(), s["ctx"].tolist()
    for r, node in enumerate(s["node"].tolist()):
        table = s["table"][r].tolist()
        for j, i in enumerate(_path(parent[r], node)):          # a node never moves up: what it leaves is not needed later
            a, z = ctx[r] + i - 1, ctx[r] + j
            for pool in (k, v):
                pool[:, table[z // page], :, z % page] = pool[:, table[a // page], :, a % page]
        ctx[r] += len(_path(parent[r], node))
    return {"k": k, "v": v, "ctx": np.array(ctx, np.int32)}


def _exact_pages(s):
    page, k, v = s["case"]["page"], s["k"].double(), s["v"].double()
    table, ref, ctx = s["table"].tolist(), s["ref"].tolist(), s["ctx"].tolist()

    def take():
        i = ref.index(0)
        ref[i] = 1
        return i

    def resize(want):
        keep = [len([i for i in row if i >= 0]) if w < 0 else -(-w // page) for row, w in zip(table, want)]
        for row, n in zip(table, keep):
            for j in range(n, len(row)):
                if row[j] >= 0:
                    ref[row[j]] -= 1
                    row[j] = -1
        for row, n in zip(table, keep):
            for j in range(n):
                if row[j] < 0:
                    row[j] = take()

    resize(s["give_back"].tolist())
    for a, z in zip(s["src"].tolist(), s["dst"].tolist()):
        full, tail = divmod(ctx[a], page)
        table[z] = table[a][:full] + [-1] * (len(table[a]) - full)
        if tail:
            table[z][full] = take()
            for pool in (k, v):
                pool[:, table[z][full], :, :tail] = pool[:, table[a][full], :, :tail]
        ctx[z] = ctx[a]
    for a in s["src"].tolist():
        for i in table[a][:ctx[a] // page]:
            ref[i] += 1
    resize([n + s["more"] for n in ctx])
    return {"table": np.array(table, np.int32), "ref": np.array(ref, np.int32), "ctx": np.array(ctx, np.int32), "k": k, "v": v}


def exact(c, seed):
    s = prepare(c, seed)
    return {"sample": _exact_sample, "norm": _exact_norm, "attn": _exact_attn, "commit": _exact_commit,
            "pages": _exact_pages}[c["op"]](s)
