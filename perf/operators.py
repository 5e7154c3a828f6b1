"""One round of tree speculation over a KV cache: what is measured of it.

Three operators, as a serving loop calls them one after the other:

* the tree step: a sequence with P cached tokens gets up to n drafted tokens, the nodes of a tree. Node i goes
  into cache row P + i, is rotated at position P + depth[i], and attends to the P cached tokens and to the nodes
  of its mask row (itself and its ancestors);
* verification: from the target's probabilities, the draft's and given random numbers, which nodes stand, and
  the token after the last of them;
* keeping the path: in every layer's cache the rows of the standing nodes move up behind the P cached tokens.

``run`` is one pass through one of them, in elementary torch operations (``own`` false) or through the
framework's entry points (``own`` true); ``exact`` gives the definition in 64 bits.
"""

import math
import random

import numpy as np
import torch

own = False

ROPE_BASE = 10000.0


# ------------------------------------------------------------------ cases
def _tree(name, **kw):
    c = dict(name=name, op="tree", cache="bf16", batch=1, h_q=32, h_kv=8, head_dim=128, prefix=512, prefix_lo=-1, nodes=16,
             ragged=False, page=0, window=0)
    c.update(kw)
    if c["prefix_lo"] < 0:  # every sequence as long
        c["prefix_lo"] = c["prefix"]
    return c


def _verify(name, **kw):
    c = dict(name=name, op="verify", batch=8, nodes=16, vocab=32000, branch=3, dtype="f32", drafted=True, ragged=False)
    c.update(kw)
    return c


def _keep(name, **kw):
    c = dict(name=name, op="keep", cache="bf16", layers=16, batch=8, h_kv=8, head_dim=128, capacity=256, nodes=32, kept=5,
             ragged=False, page=0)
    c.update(kw)
    return c


def listed():
    return [
        # one user, a short conversation, a small tree: latency counts
        _tree("tree one short", prefix=700, nodes=8),
        # a batch at 4096 tokens (the grouped-query workload of the benchmark), a small tree
        _tree("tree gqa4k 16", batch=32, prefix=4080, nodes=16),
        # the same batch with a wide tree: 256 query rows read each key
        _tree("tree gqa4k 64", batch=32, prefix=4032, nodes=64),
        # continuous batching over a page pool, lengths anywhere in 128..16384, every tree of its own size
        _tree("tree paged 32", batch=128, h_q=64, prefix=16352, prefix_lo=96, nodes=32, ragged=True, page=16),
        # few users with very long contexts
        _tree("tree long 32", batch=4, prefix=131040, nodes=32),
        # one key head for all queries, a one-byte cache
        _tree("tree mqa8k e5m2", cache="e5m2", batch=64, h_kv=1, prefix=8184, nodes=8),
        # quantised codes with scales, odd lengths and a group that is no power of two
        _tree("tree u8 odd", cache="u8", batch=24, h_q=28, h_kv=4, prefix=3001, prefix_lo=1777, nodes=13, ragged=True),
        # one user, a small vocabulary, a narrow tree: latency counts
        _verify("verify one", batch=1, nodes=8, vocab=32000, branch=2),
        # a serving batch with a large vocabulary
        _verify("verify batch", batch=32, nodes=16, vocab=128000, branch=3),
        # the largest batch, odd vocabulary, deterministic drafts (no draft probabilities)
        _verify("verify top drafts", batch=64, nodes=32, vocab=100003, branch=4, drafted=False, ragged=True),
        # one layer, as a loop over layers would call it
        _keep("keep one layer", layers=1, batch=4, nodes=16, kept=4),
        # a whole model's caches in one call
        _keep("keep 32 layers paged", layers=32, batch=32, capacity=256, nodes=48, kept=7, ragged=True, page=16),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    case = _drawn(rng)
    del case["name"]
    return case


def _drawn(rng):
    op = rng.choice(["tree", "tree", "tree", "verify", "keep"])
    if op == "tree":
        cache = rng.choice(["bf16", "bf16", "bf16", "e5m2", "u8"])
        h_kv = rng.choice([1, 2, 3, 4, 8])
        group = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
        d = rng.choice([64, 128, 128])
        nodes = _log_int(rng, 1, 64)
        batch = _log_int(rng, 1, 64)
        prefix = _log_int(rng, 1, 32768)
        while batch * prefix * h_kv > 2 ** 22:  # at most half the largest listed case's keys
            batch, prefix = max(1, batch // 2), max(1, prefix * 3 // 4)
        while batch * prefix * h_kv * group * nodes > 2 ** 29:
            nodes = max(1, nodes // 2)
        lo = rng.choice([-1, 0, prefix // 3])
        return _tree("", cache=cache, batch=batch, h_q=h_kv * group, h_kv=h_kv, head_dim=d, prefix=prefix, prefix_lo=lo,
                     nodes=nodes, ragged=rng.random() < 0.5, page=rng.choice([0, 0, 16, 32, 64]),
                     window=rng.choice([0, 0, 0, _log_int(rng, 1, 4096)]))
    if op == "verify":
        nodes, vocab, batch = _log_int(rng, 1, 64), _log_int(rng, 500, 160000), _log_int(rng, 1, 64)
        while batch * nodes * vocab > 2 ** 27:
            batch = max(1, batch // 2)
            nodes = max(1, nodes * 3 // 4)
        return _verify("", batch=batch, nodes=nodes, vocab=vocab, branch=rng.choice([1, 2, 3, 4]),
                       dtype=rng.choice(["f32", "f32", "bf16"]), drafted=rng.random() < 0.7, ragged=rng.random() < 0.5)
    nodes = _log_int(rng, 1, 64)
    layers, batch = _log_int(rng, 1, 48), _log_int(rng, 1, 32)
    return _keep("", cache=rng.choice(["bf16", "bf16", "e5m2", "u8", "f32"]), layers=layers, batch=batch,
                 h_kv=rng.choice([1, 2, 3, 4, 8]), head_dim=rng.choice([64, 128]), capacity=2 * rng.randrange(nodes, 2 * nodes + 64),
                 nodes=nodes, kept=rng.randrange(1, nodes + 1), ragged=rng.random() < 0.5, page=rng.choice([0, 0, 16, 64]))


def work(case):
    b, d = case["batch"], case.get("head_dim", 0)
    if case["op"] == "tree":
        nodes = case["nodes"] * (0.5 if case["ragged"] else 1.0)
        prefix = (case["prefix"] + case["prefix_lo"]) / 2
        keys = (min(prefix, case["window"]) if case["window"] else prefix) + nodes
        row = {"bf16": 2 * d, "e5m2": d, "u8": d + 8}[case["cache"]]
        new = b * nodes * d * (2 * case["h_q"] * 2 + (2 * case["h_kv"] * (2 + 2) if case["cache"] == "bf16" else 0))
        return {"bytes": 2 * b * case["h_kv"] * keys * row + new, "flops": 4.0 * b * case["h_q"] * nodes * keys * d}
    if case["op"] == "verify":
        # the rows of the node at which a sequence's path ends: its next token is drawn from them
        rows = 2 if case["drafted"] else 1
        return {"bytes": b * rows * case["vocab"] * (4 if case["dtype"] == "f32" else 2), "flops": 2.0 * b * rows * case["vocab"]}
    row = {"bf16": 2 * d, "f32": 4 * d, "e5m2": d, "u8": d + 8}[case["cache"]]
    kept = (1 + case["kept"]) / 2 if case["ragged"] else case["kept"]
    return {"bytes": 4.0 * case["layers"] * b * case["h_kv"] * max(kept - 1, 0.5) * row, "flops": 0}


# ----------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 17)
    return g


def _parents(rng, n, branch):
    """A random tree: node 0 the root, every other node below an earlier one that has fewer than `branch` children."""
    par, kids = [-1], [0] * n
    for i in range(1, n):
        a = max(rng.randrange(i), rng.randrange(i)) if branch > 1 else i - 1
        while kids[a] >= branch:
            a += 1  # node i - 1 has no child yet
        par.append(a)
        kids[a] += 1
    return par


def _trees(rng, batch, nodes, branch):
    """parents [batch][nodes], depth and ancestor bits (itself among them) as 32-bit words."""
    parents, depth = [], np.zeros((batch, nodes), np.int32)
    words = np.zeros((batch, nodes, (nodes + 31) // 32), np.uint32)
    for b in range(batch):
        par, bits = _parents(rng, nodes, branch), []
        for i, a in enumerate(par):
            bits.append((bits[a] if i else 0) | 1 << i)
            depth[b, i] = depth[b, a] + 1 if i else 0
            for w in range(words.shape[2]):
                words[b, i, w] = bits[i] >> (32 * w) & 0xFFFFFFFF
        parents.append(par)
    return parents, depth, words


def _num_nodes(rng, case):
    b, n = case["batch"], case["nodes"]
    if not case["ragged"]:
        return [n] * b
    return [n if i == 0 else rng.randrange(0 if i == 1 else 1, n + 1) for i in range(b)]


def _cache(case, shape, g):
    """(values or codes, scale and zero point of each row or None)"""
    if case["cache"] == "u8":
        codes = torch.randint(0, 256, shape, generator=g, device="cuda", dtype=torch.uint8)
        scale = (5.0 + 2.0 * torch.rand(shape[:-1], generator=g, device="cuda")) / 255.0
        zero = torch.randint(100, 156, shape[:-1], generator=g, device="cuda").float()
        return codes, torch.stack([scale, zero], -1).contiguous()
    dt = {"bf16": torch.bfloat16, "f32": torch.float32, "e5m2": torch.bfloat16}[case["cache"]]
    x = torch.randn(shape, generator=g, device="cuda", dtype=dt)
    return (x.to(torch.float8_e5m2) if case["cache"] == "e5m2" else x), None


def _table(rng, need, most):
    """Page numbers of each sequence out of a pool of `most` pages for each, dealt out in random order; unused entries -1."""
    total = len(need) * most
    perm = list(range(total))
    rng.shuffle(perm)
    t = np.full((len(need), most), -1, np.int32)
    at = 0
    for b, k in enumerate(need):
        t[b, :k] = perm[at:at + k]
        at += k
    return torch.from_numpy(t).cuda(), total


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def prepare(case, seed):
    rng, g = random.Random(seed), _gen(seed)
    return {"tree": _prepare_tree, "verify": _prepare_verify, "keep": _prepare_keep}[case["op"]](case, rng, g)


def _prepare_tree(case, rng, g):
    b, n, hq, hk, d = (case[k] for k in ("batch", "nodes", "h_q", "h_kv", "head_dim"))
    parents, depth, words = _trees(rng, b, n, 4)
    num = _num_nodes(rng, case)
    pos = [rng.randint(case["prefix_lo"], case["prefix"]) for _ in range(b)]
    if b > 2:
        pos[0] = case["prefix"]
    s = dict(case=case, parents=parents, depth=_i32(depth), mask=torch.from_numpy(words.view(np.int32)).cuda(), num=_i32(num), pos=_i32(pos),
             most=case["prefix"] + n, table=None, host=(pos, num))
    if case["page"]:
        s["table"], pages = _table(rng, [-(-(p + n) // case["page"]) for p in pos], -(-s["most"] // case["page"]))
        shape = (pages, hk, case["page"], d)
    else:
        shape = (b, hk, (case["prefix"] + n + 1) // 2 * 2, d)
    s["k"], s["ksz"] = _cache(case, shape, g)
    s["v"], s["vsz"] = _cache(case, shape, g)
    s["q_new"] = torch.randn((b, n, hq, d), generator=g, device="cuda", dtype=torch.bfloat16)
    if case["cache"] == "bf16":
        s["k_new"] = torch.randn((b, n, hk, d), generator=g, device="cuda", dtype=torch.bfloat16)
        s["v_new"] = torch.randn((b, n, hk, d), generator=g, device="cuda", dtype=torch.bfloat16)
    s["out"] = torch.zeros((b, n, hq, d), device="cuda", dtype=torch.bfloat16)
    return s


def _prepare_verify(case, rng, g):
    b, n, vocab = case["batch"], case["nodes"], case["vocab"]
    parents, depth, words = _trees(rng, b, n, case["branch"])
    logits = torch.randn((b, n, vocab), generator=g, device="cuda") * 2.5
    p = torch.softmax(logits, -1)
    q = torch.softmax(logits + torch.randn((b, n, vocab), generator=g, device="cuda"), -1)  # a draft model that is near the target
    above = _i32(parents).clamp(min=0).long()
    race = torch.empty((b, n, vocab), device="cuda").exponential_(generator=g)
    tokens = (torch.gather(q, 1, above[..., None].expand(-1, -1, vocab)) / race).argmax(-1).int()
    dt = {"f32": torch.float32, "bf16": torch.bfloat16}[case["dtype"]]
    num = _num_nodes(rng, case)
    return dict(case=case, parents=_i32(parents), mask=torch.from_numpy(words.view(np.int32)).cuda(), num=_i32(num), tokens=tokens,
                p=p.to(dt), q=q.to(dt) if case["drafted"] else None, u=torch.rand((b, n), generator=g, device="cuda"),
                u_next=torch.rand((b,), generator=g, device="cuda"), host=(parents, num))


def _prepare_keep(case, rng, g):
    b, n = case["batch"], case["nodes"]
    most = case["capacity"] - n
    pos = [rng.randint(0, most) for _ in range(b)]
    kept = [rng.randint(1, case["kept"]) if case["ragged"] and i else case["kept"] for i in range(b)]
    path = np.full((b, n), -1, np.int32)
    for i, k in enumerate(kept):
        path[i, :k] = [0] + sorted(rng.sample(range(1, n), k - 1))
    s = dict(case=case, pos=_i32(pos), path=_i32(path), kept=_i32(kept), table=None)
    if case["page"]:
        s["table"], pages = _table(rng, [-(-(p + n) // case["page"]) for p in pos], -(-case["capacity"] // case["page"]))
        shape = (case["layers"], pages, case["h_kv"], case["page"], case["head_dim"])
    else:
        shape = (case["layers"], b, case["h_kv"], case["capacity"], case["head_dim"])
    s["k"], s["ksz"] = _cache(case, shape, g)
    s["v"], s["vsz"] = _cache(case, shape, g)
    return s


# -------------------------------------------------------------------- run
def run(state):
    if own:
        return {"tree": _own_tree, "verify": _own_verify, "keep": _own_keep}[state["case"]["op"]](state)
    return {"tree": _plain_tree, "verify": _plain_verify, "keep": _plain_keep}[state["case"]["op"]](state)


def _rows(x, sz, table):
    """A cache as [batch, h_kv, tokens, head_dim] in 32 bits."""
    if table is not None:
        at = table.clamp(min=0).long()
        x = x.view(torch.uint8)[at].view(x.dtype) if x.dtype == torch.float8_e5m2 else x[at]
        x = x.permute(0, 2, 1, 3, 4).flatten(2, 3)
        sz = None if sz is None else sz[at].permute(0, 2, 1, 3, 4).flatten(2, 3)
    x = x.float()
    return x if sz is None else (x - sz[..., 1:]) * sz[..., :1]


def _bits(words, n):
    """[..., W] 32-bit words as [..., n] truth values."""
    return ((words[..., None] >> torch.arange(32, device=words.device)) & 1).bool().flatten(-2)[..., :n]


def _rotate(x, at):
    """Adjacent pairs turned by at * base^(-2 i / d): angles in 64 bits, x [batch, n, heads, d], at [batch, n]."""
    d = x.shape[-1]
    a = at.double()[..., None] * ROPE_BASE ** (-torch.arange(0, d, 2, device=x.device).double() / d)
    c, s = torch.cos(a)[:, :, None], torch.sin(a)[:, :, None]
    e, o = x[..., 0::2].double(), x[..., 1::2].double()
    return torch.stack([e * c - o * s, e * s + o * c], -1).flatten(-2)


def _plain_tree(s):
    case, n = s["case"], s["case"]["nodes"]
    b, hq, hk, d = (case[k] for k in ("batch", "h_q", "h_kv", "head_dim"))
    pos, depth = s["pos"].long(), s["depth"].long()
    i = torch.arange(n, device="cuda")
    live = i < s["num"][:, None]
    q = s["q_new"].float()
    if case["cache"] == "bf16":
        at = pos[:, None] + depth
        q = _rotate(s["q_new"], at).float()
        slot = pos[:, None] + i
        which, node = torch.nonzero(live, as_tuple=True)
        slot = slot[which, node]
        new = [(s["k"], _rotate(s["k_new"], at).to(torch.bfloat16)[which, node]), (s["v"], s["v_new"][which, node])]
        first, row = (which, slot) if s["table"] is None else (s["table"].long()[which, slot // case["page"]], slot % case["page"])
        new[0][0][first, :, row] = new[0][1]
        new[1][0][first, :, row] = new[1][1]
    k, v = _rows(s["k"], s["ksz"], s["table"]), _rows(s["v"], s["vsz"], s["table"])
    t = torch.arange(k.shape[2], device="cuda")
    node = t - pos[:, None]  # [batch, tokens]: the node of each key, negative for a cached token
    tree = _bits(s["mask"], n) & live[:, None]
    near = torch.ones((), device="cuda", dtype=torch.bool)
    if case["window"]:
        tree = tree & (depth[:, None] > depth[..., None] - case["window"])
        near = t > (pos[:, None] + depth)[..., None] - case["window"]
    inside = (node >= 0) & (node < n)
    seen = torch.gather(tree, 2, node.clamp(0, n - 1)[:, None].expand(-1, n, -1)) & inside[:, None] | (node < 0)[:, None] & near
    rows = q.view(b, n, hk, hq // hk, d).permute(0, 2, 1, 3, 4).flatten(2, 3)
    score = (rows @ k.transpose(2, 3)).mul_(1 / math.sqrt(d)).view(b, hk, n, hq // hk, -1)
    score.masked_fill_(~seen[:, None, :, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = score.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.flatten(2, 3) @ v).view(b, hk, n, hq // hk, d) / torch.where(total == 0, 1.0, total)
    o = o.permute(0, 2, 1, 3, 4).flatten(2, 3)
    s["out"].copy_(torch.where(live[..., None, None], o, s["out"].float()))
    return {"out": s["out"], "k": s["k"], "v": s["v"]} if case["cache"] == "bf16" else {"out": s["out"]}


def _plain_verify(s):
    case, n = s["case"], s["case"]["nodes"]
    live = torch.arange(n, device="cuda") < s["num"][:, None]
    child = live & (s["parents"] >= 0)
    above = s["parents"].clamp(min=0).long()
    p, tok = s["p"].double(), s["tokens"].long()
    same = (above[:, :, None] == above[:, None]) & child[:, :, None] & child[:, None]
    earlier = same & (torch.arange(n, device="cuda") < torch.arange(n, device="cuda")[:, None])
    rank = earlier.sum(-1)  # how many siblings are tried before
    pick = lambda x: x[torch.arange(len(tok), device="cuda")[:, None], above, tok]  # noqa: E731
    px, u = pick(p), s["u"].double()
    if s["q"] is not None:
        q = s["q"].double()
        coef, left = [torch.zeros_like(p[..., 0])], [torch.ones_like(p[..., 0])]
        for _ in range(case["branch"]):  # the residual after each further rejection, at every node
            coef.append(coef[-1] + left[-1])
            left.append((p - coef[-1][..., None] * q).clamp_(min=0).sum(-1))
        coef, left = torch.stack(coef, -1), torch.stack(left, -1)
        of = lambda x: torch.gather(torch.gather(x, 1, above[..., None].expand(-1, -1, x.shape[-1])), 2, rank[..., None])[..., 0]  # noqa: E731
        qx = pick(q)
        good = child & (u * qx * of(left) < (px - of(coef) * qx).clamp(min=0))
    else:
        first = ~(earlier & (tok[:, :, None] == tok[:, None])).any(-1)  # a token that was rejected before has no weight left
        left = 1 - (earlier * (px * first)[:, None]).sum(-1)
        good = child & (u * left < px * first)
    root = live & (s["parents"] < 0)
    good = root | good & ~(earlier & good[:, None]).any(-1)  # the first child that stands
    on = live & ~(_bits(s["mask"], n) & ~good[:, None]).any(-1)
    kept = on.sum(-1)
    path = torch.where(on, torch.arange(n, device="cuda"), n).sort(-1).values
    last = path.gather(1, (kept - 1).clamp(min=0)[:, None])[:, 0].clamp(max=n - 1)
    path = torch.where(path == n, -1, path)
    one = torch.arange(len(tok), device="cuda")
    weight, tried = p[one, last], child & (above == last[:, None])
    if s["q"] is not None:
        weight = (weight - coef[one, last, tried.sum(-1)][:, None] * q[one, last]).clamp_(min=0)
    else:
        weight = weight * (torch.ones_like(weight).scatter_reduce_(1, tok, 1.0 - tried.double(), "amin"))
    cum = weight.cumsum(-1)
    goal = cum[:, -1] * s["u_next"].double()
    drawn = (cum <= goal[:, None]).sum(-1)
    drawn = torch.where(cum[:, -1] > 0, drawn, p[one, last].argmax(-1))
    drawn = torch.where(s["num"] > 0, drawn, -1)
    return {"kept": kept.int(), "path": path.int(), "next": drawn.int()}


def _plain_keep(s):
    case, n = s["case"], s["case"]["nodes"]
    i = torch.arange(n, device="cuda")
    stays = i < s["kept"][:, None]
    src = s["pos"].long()[:, None] + torch.where(stays, s["path"].long(), 0)
    dst = s["pos"].long()[:, None] + torch.where(stays, i, 0)  # the others write row 0 of the tree onto itself
    one = torch.arange(case["batch"], device="cuda")[:, None].expand(-1, n)
    at = lambda r: (one, r) if s["table"] is None else (s["table"].long()[one, r // case["page"]], r % case["page"])  # noqa: E731
    (a, ar), (c, cr) = at(src), at(dst)
    raw = lambda x: x.view(torch.uint8) if x.dtype == torch.float8_e5m2 else x  # noqa: E731
    k, v = raw(s["k"]), raw(s["v"])
    k[:, c, :, cr] = k[:, a, :, ar]
    v[:, c, :, cr] = v[:, a, :, ar]
    if s["ksz"] is not None:
        s["ksz"][:, c, :, cr] = s["ksz"][:, a, :, ar]
        s["vsz"][:, c, :, cr] = s["vsz"][:, a, :, ar]
    return {"k": s["k"], "v": s["v"], "ksz": s["ksz"], "vsz": s["vsz"]}


def _own_tree(s):
    import mqa_decode_attention_gb300 as m

    case, n = s["case"], s["case"]["nodes"]
    if "layout" not in s:  # the layout and the workspace are made once, as a serving loop keeps them
        if case["page"]:
            s["layout"] = m.layout_paged(s["k"], s["v"], s["table"], case["h_q"], case["window"], s["ksz"], s["vsz"])
        else:
            s["layout"] = m.layout_contiguous(s["k"], s["v"], case["h_q"], case["window"], s["ksz"], s["vsz"])
        s["bufs"] = m.TreeBuffers.allocate(s["layout"], n, s["most"])
        s["bufs"].out = s["out"]
    if case["cache"] == "bf16":
        m.tree_step(s["layout"], n, s["q_new"], s["k_new"], s["v_new"], s["pos"], s["depth"], s["mask"], s["most"], s["bufs"], ROPE_BASE,
                    num_nodes=s["num"])
        return {"out": s["out"], "k": s["k"], "v": s["v"]}
    m.gqa_tree_attention(s["layout"], n, s["q_new"], s["pos"], s["depth"], s["mask"], s["most"], 1 / math.sqrt(case["head_dim"]), s["out"],
                         num_nodes=s["num"], workspace=s["bufs"].workspace, err=s["bufs"].err)
    return {"out": s["out"]}


def _own_verify(s):
    import mqa_decode_attention_gb300 as m

    if "bufs" not in s:
        s["bufs"] = m.VerifyBuffers.allocate(s["case"]["batch"], s["case"]["nodes"])
    m.verify_tree(s["p"], s["q"], s["tokens"], s["parents"], s["u"], s["u_next"], s["bufs"], num_nodes=s["num"])
    return {"kept": s["bufs"].num_kept, "path": s["bufs"].path, "next": s["bufs"].next_token}


def _own_keep(s):
    import mqa_decode_attention_gb300 as m

    if "layouts" not in s:
        part = lambda x, i: None if x is None else x[i]  # noqa: E731
        each = range(s["case"]["layers"])
        if s["case"]["page"]:
            s["layouts"] = m.layout_stack([m.layout_paged(s["k"][i], s["v"][i], s["table"], s["case"]["h_kv"], 0, part(s["ksz"], i), part(s["vsz"], i)) for i in each])
        else:
            s["layouts"] = m.layout_stack([m.layout_contiguous(s["k"][i], s["v"][i], s["case"]["h_kv"], 0, part(s["ksz"], i), part(s["vsz"], i)) for i in each])
        s["err"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    m.keep_path(s["layouts"], s["pos"], s["path"], s["kept"], s["err"])
    return {"k": s["k"], "v": s["v"], "ksz": s["ksz"], "vsz": s["vsz"]}


# ------------------------------------------------------------------ exact
def exact(case, seed):
    s = prepare(case, seed)
    return {"tree": _exact_tree, "verify": _exact_verify, "keep": _exact_keep}[case["op"]](s)


def _turned(x, at):
    """x [n, heads, d] as complex pairs times e^(i at base^(-2 i / d)), in 64 bits."""
    d = x.shape[-1]
    freq = torch.pow(torch.tensor(ROPE_BASE, dtype=torch.float64, device="cuda"), -2.0 * torch.arange(d // 2, device="cuda", dtype=torch.float64) / d)
    z = torch.view_as_complex(x.double().reshape(*x.shape[:-1], d // 2, 2).contiguous())
    return torch.view_as_real(z * torch.polar(torch.ones((), device="cuda", dtype=torch.float64), at.double()[:, None, None] * freq)).reshape(x.shape)


def _exact_tree(s):
    """Sequence by sequence: the keys that a node may see are found from its parents, one softmax in 64 bits over them."""
    case = s["case"]
    hq, hk, d, window = case["h_q"], case["h_kv"], case["head_dim"], case["window"]
    step = case["cache"] == "bf16"
    if not step:
        k_all = v_all = None
    else:
        k_all, v_all = s["k"].double(), s["v"].double()
    out = s["out"].double()
    for b, (pos, num) in enumerate(zip(*s["host"])):
        if not num:
            continue
        where = torch.arange(pos + num, device="cuda")
        if s["table"] is None:
            a, r = torch.full_like(where, b), where
        else:
            a, r = s["table"][b].long()[where // case["page"]], where % case["page"]
        q = s["q_new"][b, :num].double()
        if step:
            at = pos + s["depth"][b, :num]
            q = _turned(s["q_new"][b, :num], at)
            k_all[a[pos:], :, r[pos:]] = _turned(s["k_new"][b, :num], at).to(torch.bfloat16).double()
            v_all[a[pos:], :, r[pos:]] = s["v_new"][b, :num].double()
            k, v = k_all[a, :, r], v_all[a, :, r]
        else:
            raw = lambda x: x.view(torch.uint8)[a, :, r].view(x.dtype).double() if x.dtype == torch.float8_e5m2 else x[a, :, r].double()  # noqa: E731
            k, v = raw(s["k"]), raw(s["v"])
            if s["ksz"] is not None:
                k = (k - s["ksz"][a, :, r][..., 1:].double()) * s["ksz"][a, :, r][..., :1].double()
                v = (v - s["vsz"][a, :, r][..., 1:].double()) * s["vsz"][a, :, r][..., :1].double()
        seen = np.zeros((num, pos + num), bool)
        level = [0] * num
        for i in range(num):
            up = i
            while up >= 0:
                level[i] += up != i
                up = s["parents"][b][up]
            seen[i, max(0, pos + level[i] + 1 - window) if window else 0:pos] = True
            up = i
            while up >= 0:
                seen[i, pos + up] = not window or level[up] > level[i] - window
                up = s["parents"][b][up]
        score = torch.einsum("nhgd,thd->hgnt", q.view(num, hk, hq // hk, d), k) / math.sqrt(d)
        w = torch.softmax(score.masked_fill_(~torch.from_numpy(seen).cuda(), -math.inf), -1)
        out[b, :num] = torch.einsum("hgnt,thd->nhgd", w, v).reshape(num, hq, d)
    return {"out": out, "k": k_all, "v": v_all} if step else {"out": out}


def _exact_verify(s):
    """The walk itself, one node after the other."""
    case, n = s["case"], s["case"]["nodes"]
    tokens, u, u_next = s["tokens"].tolist(), s["u"].tolist(), s["u_next"].tolist()
    kept, paths, drawn = [], [], []
    for b, (par, num) in enumerate(zip(*s["host"])):
        at, path, nxt = 0, [0], -1
        while num:
            left = s["p"][b, at].double().cpu().numpy()
            mass, first = 1.0, left
            for c in [c for c in range(1, num) if par[c] == at]:
                x = tokens[b][c]
                if s["q"] is not None:
                    q = s["q"][b, at].double().cpu().numpy()
                    if u[b][c] * q[x] * mass < left[x]:
                        break
                    left = np.maximum(left - mass * q, 0)
                    mass = float(left.sum())
                else:
                    if u[b][c] * mass < left[x]:
                        break
                    mass -= left[x]
                    left = left.copy()
                    left[x] = 0
            else:
                cum = np.cumsum(left)
                nxt = int(np.searchsorted(cum, u_next[b] * cum[-1], side="right")) if cum[-1] > 0 else int(first.argmax())
                break
            at = c
            path.append(c)
        path = path if num else []
        kept.append(len(path))
        paths.append(path + [-1] * (n - len(path)))
        drawn.append(nxt)
    return {"kept": _i32(kept), "path": _i32(paths), "next": _i32(drawn)}


def _exact_keep(s):
    """Row by row, upwards: a row's place is never behind the rows that are still to move."""
    page = s["case"]["page"]
    slot = lambda b, t: (b, t) if s["table"] is None else (int(s["table"][b, t // page]), t % page)  # noqa: E731
    all_of = [s[name] for name in ("k", "v", "ksz", "vsz")]
    for b, (pos, kept) in enumerate(zip(s["pos"].tolist(), s["kept"].tolist())):
        for i, node in enumerate(s["path"][b, :kept].tolist()):
            (a, r), (c, t) = slot(b, pos + node), slot(b, pos + i)
            for x in all_of:
                if x is not None and node != i:
                    x[:, c, :, t] = x[:, a, :, r].clone()
    value = lambda x: x if x is None or x.dtype == torch.uint8 else x.double()  # noqa: E731
    return dict(zip(("k", "v", "ksz", "vsz"), map(value, all_of)))
