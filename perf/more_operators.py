"""A KV cache held in four bits, and the rows on their way into a cache and out of it: what is measured of them.

Three operators, as a serving loop calls them one after the other:

* append: queries and keys of each head are normalised (root mean square, a weight for each dimension), turned by their
  position (one number, or one for each axis of an image or a video), and the key and value rows are written into the
  cache in its type. A row of the 4-bit cache is a code of 0..15 for each value and one bf16 pair (scale s, minimum m):
  the value is m + s * code;
* attention over the 4-bit cache: each new query over every cached token of its sequence, or over the last W of them;
* reading back: rows of a cache of any type as bf16 or fp32 values, in the layout of a cache.

``run`` is one pass through one of them, in elementary torch operations (``own`` false) or through the framework's
entry points (``own`` true); ``exact`` gives the definition in 64 bits.
"""

import math
import random

import numpy as np
import torch

own = False

ROPE_BASE = 10000.0
EPS = 1e-6


# ------------------------------------------------------------------ cases
def _attn(name, **kw):
    c = dict(name=name, op="attn", batch=32, h_q=32, h_kv=8, head_dim=128, tokens=4096, tokens_lo=-1, new=1, page=0, window=0)
    c.update(kw)
    if c["tokens_lo"] < 0:  # every sequence as long
        c["tokens_lo"] = c["tokens"]
    return c


def _append(name, **kw):
    c = dict(name=name, op="append", cache="u4", batch=32, new=1, h_q=32, h_kv=8, head_dim=128, prefix=4096, norm=True, axes=0, page=0)
    c.update(kw)
    return c


def _read(name, **kw):
    c = dict(name=name, op="read", cache="u4", batch=8, h_kv=8, head_dim=128, rows=4096, start=0, ragged=False, page=0, out="bf16")
    c.update(kw)
    return c


def listed():
    return [
        # one user, a short conversation: latency counts
        _attn("attn one short", batch=1, tokens=700),
        # a batch at 4096 tokens, the grouped-query workload of the benchmark
        _attn("attn gqa4k"),
        # the same batch, eight drafted tokens of each sequence checked at once
        _attn("attn gqa4k 8 new", new=8),
        # one key head for all queries
        _attn("attn mqa8k", batch=64, h_kv=1, tokens=8192),
        # continuous batching over a page pool, lengths anywhere in 128..16384
        _attn("attn paged", batch=128, h_q=64, tokens=16384, tokens_lo=128, page=16),
        # few users with very long contexts
        _attn("attn long", batch=4, tokens=131072),
        # odd lengths, a group that is no power of two, small heads, a sliding window
        _attn("attn odd window", batch=24, h_q=28, h_kv=4, head_dim=64, tokens=3001, tokens_lo=777, window=1500),
        # one token of each sequence into a bf16 cache, normalised: latency counts
        _append("append norm bf16", cache="bf16", capacity=256, prefix=255),
        # prompts with images, positions of three axes, into a 4-bit page pool, and the rows as they now stand there
        _append("append prompt 3 axes u4", batch=8, new=4096, prefix=0, axes=3, page=16),
        # odd sizes, an e5m2 cache, no norm
        _append("append odd e5m2", cache="e5m2", batch=7, new=33, h_q=21, h_kv=3, head_dim=64, prefix=1234, norm=False, axes=2),
        # whole cached prompts out of a 4-bit cache, for a prefill that continues them
        _read("read u4"),
        # cached prefixes of many lengths out of a uint8 page pool
        _read("read paged u8", cache="u8", batch=24, h_kv=5, rows=3000, start=777, ragged=True, page=32, out="f32"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    case = _drawn(rng)
    del case["name"]
    return case


def _drawn(rng):
    op = rng.choice(["attn", "attn", "attn", "append", "append", "read"])
    h_kv, d, page = rng.choice([1, 2, 3, 4, 8]), rng.choice([64, 128, 128]), rng.choice([0, 0, 16, 32, 64])
    group = rng.choice([1, 2, 3, 4, 5, 7, 8, 16, 32])
    if op == "attn":
        batch, tokens, new = _log_int(rng, 1, 128), _log_int(rng, 1, 131072), rng.choice([1, 1, 1, _log_int(rng, 2, 32)])
        tokens = max(tokens, new)
        while batch * tokens * h_kv > 2 ** 22:
            batch, tokens = max(1, batch // 2), max(new, tokens * 3 // 4)
        while batch * tokens * h_kv * group * new > 2 ** 28:
            group = max(1, group // 2)
            new = max(1, new // 2)
        return _attn("", batch=batch, h_q=h_kv * group, h_kv=h_kv, head_dim=d, tokens=tokens, tokens_lo=rng.choice([-1, new, max(new, tokens // 3)]),
                     new=new, page=page, window=rng.choice([0, 0, 0, _log_int(rng, 1, 4096)]))
    if op == "append":
        batch, new = _log_int(rng, 1, 64), rng.choice([1, 1, _log_int(rng, 2, 4096)])
        while batch * new * h_kv * (group + 2) > 2 ** 20:
            batch, new = max(1, batch // 2), max(1, new * 3 // 4)
        return _append("", cache=rng.choice(["u4", "u4", "bf16", "u8", "e5m2", "f32"]), batch=batch, new=new, h_q=h_kv * group, h_kv=h_kv,
                       head_dim=d, prefix=rng.choice([0, _log_int(rng, 1, 2048)]), norm=rng.random() < 0.7, axes=rng.choice([0, 0, 2, 3, 4]), page=page)
    batch, rows = _log_int(rng, 1, 64), _log_int(rng, 1, 8192)
    while batch * rows * h_kv > 2 ** 19:
        batch, rows = max(1, batch // 2), max(1, rows * 3 // 4)
    return _read("", cache=rng.choice(["u4", "u4", "bf16", "u8", "e5m2", "f32"]), batch=batch, h_kv=h_kv, head_dim=d, rows=rows,
                 start=rng.choice([0, _log_int(rng, 1, 1000)]), ragged=rng.random() < 0.5, page=page, out=rng.choice(["bf16", "f32"]))


def _row_bytes(cache, d):
    return {"u4": d // 2 + 4, "u8": d + 8, "e5m2": d, "bf16": 2 * d, "f32": 4 * d}[cache]


def work(case):
    b, d, hk = case["batch"], case["head_dim"], case["h_kv"]
    if case["op"] == "attn":
        hq, n = case["h_q"], case["new"]
        tokens = (case["tokens"] + case["tokens_lo"]) / 2
        keys = min(tokens, case["window"] + n - 1) if case["window"] else tokens
        return {"bytes": 2 * b * hk * keys * _row_bytes("u4", d) + b * n * hq * d * (4 + 2), "flops": 4.0 * b * n * hq * keys * d}
    if case["op"] == "append":
        n, hq, size = case["new"], case["h_q"], 4 if case["cache"] == "f32" else 2
        back = 0 if case["cache"] in ("bf16", "f32") else 2 * hk * (_row_bytes(case["cache"], d) + 2 * d)
        return {"bytes": b * n * (hq * d * (size + 4) + 2 * hk * (d * size + _row_bytes(case["cache"], d)) + back), "flops": 10.0 * b * n * (hq + hk) * d}
    rows = case["rows"] * (0.5 if case["ragged"] else 1.0)
    return {"bytes": 2 * b * hk * rows * (_row_bytes(case["cache"], d) + d * (2 if case["out"] == "bf16" else 4)), "flops": 4.0 * b * hk * rows * d}


# ----------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 29)
    return g


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _codes4(shape, g):
    """Codes as rows of a normal distribution have them, two to a byte: the even dimension in the low half."""
    out = torch.empty(shape, dtype=torch.uint8, device="cuda")
    flat = out.view(-1)
    step = 1 << 27
    for at in range(0, flat.numel(), step):
        part = flat[at:at + step]
        low, high = ((torch.randn(part.numel(), generator=g, device="cuda") * 2.9 + 7.5).round_().clamp_(0, 15).to(torch.uint8) for _ in range(2))
        torch.bitwise_or(low, high << 4, out=part)
    return out


def _cache(cache, shape, g):
    """A cache's tensors (codes or values, and a row's scale with its minimum or zero point, or None), shape [..., head_dim]."""
    d = shape[-1]
    if cache == "u4":
        scale = 0.3 + 0.1 * torch.rand(shape[:-1], generator=g, device="cuda")
        low = -scale * (7.0 + torch.rand(shape[:-1], generator=g, device="cuda"))
        return _codes4((*shape[:-1], d // 2), g), torch.stack([scale, low], -1).to(torch.bfloat16)
    if cache == "u8":
        codes = torch.randint(0, 256, shape, generator=g, device="cuda", dtype=torch.uint8)
        scale = (5.0 + 2.0 * torch.rand(shape[:-1], generator=g, device="cuda")) / 255.0
        zero = torch.randint(100, 156, shape[:-1], generator=g, device="cuda").float()
        return codes, torch.stack([scale, zero], -1).contiguous()
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32 if cache == "f32" else torch.bfloat16)
    return (x.to(torch.float8_e5m2) if cache == "e5m2" else x), None


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


def _caches(s, case, lens, most, rng, g):
    """The caches of `most` tokens for each sequence, of which lens[b] are in use."""
    b, hk, d, page = case["batch"], case["h_kv"], case["head_dim"], case["page"]
    s["table"] = None
    if page:
        s["table"], pages = _table(rng, [-(-n // page) for n in lens], -(-most // page))
        shape = (pages, hk, page, d)
    else:
        shape = (b, hk, -(-most // 4) * 4, d)
    cache = case.get("cache", "u4")
    s["k"], s["ksz"] = _cache(cache, shape, g)
    s["v"], s["vsz"] = _cache(cache, shape, g)


def prepare(case, seed):
    rng, g = random.Random(seed), _gen(seed)
    return {"attn": _prepare_attn, "append": _prepare_append, "read": _prepare_read}[case["op"]](case, rng, g)


def _prepare_attn(case, rng, g):
    b, n, hq, d = (case[k] for k in ("batch", "new", "h_q", "head_dim"))
    lens = [rng.randint(case["tokens_lo"], case["tokens"]) for _ in range(b)]
    if b > 2:
        lens[0] = case["tokens"]
    s = dict(case=case, lens=_i32(lens), host=lens)
    _caches(s, case, lens, case["tokens"], rng, g)
    s["q"] = torch.randn((b, n, hq, d), generator=g, device="cuda")  # turned already, fp32 as the append leaves it
    s["out"] = torch.empty((b, n, hq, d), device="cuda", dtype=torch.bfloat16)
    return s


def _sections(case):
    half, axes = case["head_dim"] // 2, case["axes"]
    first = half // (axes + 1)
    rest = (half - first) // (axes - 1)
    return [half - rest * (axes - 1)] + [rest] * (axes - 1)


def _prepare_append(case, rng, g):
    b, n, hq, hk, d = (case[k] for k in ("batch", "new", "h_q", "h_kv", "head_dim"))
    pos = [rng.randint(0, case["prefix"]) for _ in range(b)]
    pos[0] = case["prefix"]
    most = max(case.get("capacity", 0), case["prefix"] + n)
    s = dict(case=case, pos=_i32(pos), host=pos)
    _caches(s, case, [p + n for p in pos], most, rng, g)
    dt = torch.float32 if case["cache"] == "f32" else torch.bfloat16
    for name, heads in (("q_new", hq), ("k_new", hk), ("v_new", hk)):
        s[name] = torch.randn((b, n, heads, d), generator=g, device="cuda", dtype=dt)
    s["qw"] = s["kw"] = s["axis"] = None
    if case["norm"]:
        s["qw"], s["kw"] = ((1.0 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(dt) for _ in range(2))
    if case["axes"]:  # text, where all axes count on together, and here and there an image of 20 patches a line
        i = torch.arange(n, device="cuda").expand(b, n)
        image = torch.rand((b, n), generator=g, device="cuda") < 0.5
        at = torch.tensor(pos, device="cuda")[:, None] + i
        s["axis"] = torch.stack([torch.where(image, (at // 400) * 3 + a, at) + torch.where(image, (i // 20 ** (a % 2)) % 20, 0)
                                 for a in range(case["axes"])]).int()
    widths = _sections(case) if case["axes"] else [d // 2]
    s["pair_axis"] = torch.from_numpy(np.repeat(np.arange(len(widths)), widths)).cuda()
    s["q_rot"] = torch.empty((b, n, hq, d), device="cuda")
    if case["cache"] not in ("bf16", "f32"):
        s["rows"] = [torch.zeros((b, hk, n, d), device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    return s


def _prepare_read(case, rng, g):
    b, hk, d = case["batch"], case["h_kv"], case["head_dim"]
    start = [rng.randint(0, case["start"]) for _ in range(b)]
    rows = [rng.randint(0, case["rows"]) if case["ragged"] and i else case["rows"] for i in range(b)]
    s = dict(case=case, start=_i32(start), rows=_i32(rows), host=(start, rows))
    _caches(s, case, [x + y for x, y in zip(start, rows)], case["start"] + case["rows"], rng, g)
    dt = torch.bfloat16 if case["out"] == "bf16" else torch.float32
    s["out"] = [torch.zeros((b, hk, case["rows"], d), device="cuda", dtype=dt) for _ in range(2)]
    return s


# -------------------------------------------------------------------- run
def run(state):
    if own:
        return {"attn": _own_attn, "append": _own_append, "read": _own_read}[state["case"]["op"]](state)
    return {"attn": _plain_attn, "append": _plain_append, "read": _plain_read}[state["case"]["op"]](state)


def _values(x, sz, cache):
    """Rows of a cache as values in 32 bits."""
    if cache == "u4":
        x = torch.stack([x & 15, x >> 4], -1).flatten(-2).float()
        return x.mul_(sz[..., :1].float()).add_(sz[..., 1:].float())
    x = x.float()
    return (x - sz[..., 1:]) * sz[..., :1] if cache == "u8" else x


def _gathered(x, table):
    """A cache as [batch, h_kv, tokens, ...]."""
    if table is None or x is None:
        return x
    at = table.clamp(min=0).long()
    x = x.view(torch.uint8)[at].view(x.dtype) if x.dtype == torch.float8_e5m2 else x[at]
    return x.transpose(1, 2).flatten(2, 3)


def _plain_attn(s):
    case = s["case"]
    b, n, hq, hk, d = (case[k] for k in ("batch", "new", "h_q", "h_kv", "head_dim"))
    k = _values(_gathered(s["k"], s["table"]), _gathered(s["ksz"], s["table"]), "u4")
    rows = s["q"].view(b, n, hk, hq // hk, d).permute(0, 2, 1, 3, 4).flatten(2, 3)
    score = (rows @ k.transpose(2, 3)).mul_(1 / math.sqrt(d)).view(b, hk, n, hq // hk, -1)
    del k
    t, i = torch.arange(score.shape[-1], device="cuda"), torch.arange(n, device="cuda")
    last = s["lens"].long()[:, None] - n + i  # [batch, new]: the position of each query
    seen = t <= last[..., None]
    if case["window"]:
        seen = seen & (t > last[..., None] - case["window"])
    score.masked_fill_(~seen[:, None, :, None], -math.inf)
    p = score.sub_(score.amax(-1, keepdim=True)).exp_()
    total = p.sum(-1, keepdim=True)
    v = _values(_gathered(s["v"], s["table"]), _gathered(s["vsz"], s["table"]), "u4")
    o = (p.flatten(2, 3) @ v).view(b, hk, n, hq // hk, d) / total
    s["out"].copy_(o.permute(0, 2, 1, 3, 4).flatten(2, 3))
    return {"out": s["out"]}


def _turn(x, at, axis):
    """x [batch, new, heads, d] in 64 bits: adjacent pairs turned by position * base^(-2 i / d); at [axes, batch, new], pair i by axis[i]'s."""
    d = x.shape[-1]
    a = at.double()[axis].permute(1, 2, 0) * ROPE_BASE ** (-torch.arange(0, d, 2, device=x.device).double() / d)
    c, s = torch.cos(a)[:, :, None], torch.sin(a)[:, :, None]
    e, o = x[..., 0::2].double(), x[..., 1::2].double()
    return torch.stack([e * c - o * s, e * s + o * c], -1).flatten(-2)


def _normed(x, w):
    """In 64 bits: what follows rounds to few bits, and a value may lie next to a border."""
    x = x.double()
    return x if w is None else x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.double()


def _encode(x, cache):
    """Rows (bf16; fp32 for an fp32 cache) as a cache holds them."""
    if cache in ("bf16", "f32"):
        return x, None
    if cache == "e5m2":
        return x.float().clamp(-57344, 57344).to(torch.float8_e5m2), None
    low, high = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    if cache == "u8":
        x, low, high = x.float(), low.float(), high.float()
        scale = (high - low) / 255
        scale = torch.where(scale == 0, 1.0, scale)
        zero = (-low / scale).round().clamp(0, 255)
        return (x / scale + zero).round().clamp(0, 255).to(torch.uint8), torch.cat([scale, zero], -1)
    x, low, high = x.double(), low.double(), high.double()
    want = (high - low) / 15  # the scale is the smallest bf16 that reaches the largest value
    scale = want.to(torch.bfloat16)
    above = (scale.view(torch.int16) + 1).view(torch.bfloat16)
    scale = torch.where(scale.double() * 15 < high - low, above, scale).double()
    code = ((x - low) / torch.where(scale == 0, 1.0, scale)).round().clamp(0, 15).to(torch.uint8)
    return code[..., 0::2] | code[..., 1::2] << 4, torch.cat([scale, low], -1).to(torch.bfloat16)


def _places(s, slot):
    """Index of rows `slot` [batch, new] of each sequence: (sequence or page, row), for x[first, :, row] of [first, h_kv, row, ...]."""
    page = s["case"]["page"]
    one = torch.arange(slot.shape[0], device="cuda")[:, None].expand_as(slot)
    return (one, slot) if s["table"] is None else (s["table"].long()[one, slot // page], slot % page)


def _raw(x):
    return x.view(torch.uint8) if x.dtype == torch.float8_e5m2 else x


def _plain_append(s):
    case, i = s["case"], torch.arange(s["case"]["new"], device="cuda")
    cache, slot = case["cache"], s["pos"].long()[:, None] + i
    at = slot[None] if s["axis"] is None else s["axis"]
    s["q_rot"].copy_(_turn(_normed(s["q_new"], s["qw"]), at, s["pair_axis"]))
    k = _turn(_normed(s["k_new"], s["kw"]), at, s["pair_axis"]).to(s["k_new"].dtype)
    first, row = _places(s, slot)
    kc, kz = _encode(k, cache)
    vc, vz = _encode(s["v_new"], cache)
    _raw(s["k"])[first, :, row], _raw(s["v"])[first, :, row] = _raw(kc), _raw(vc)
    if kz is not None:
        s["ksz"][first, :, row], s["vsz"][first, :, row] = kz, vz
    if cache in ("bf16", "f32"):
        return {"q_rot": s["q_rot"], "k": s["k"], "v": s["v"]}
    part = lambda x: None if x is None else _raw(x)[first, :, row].transpose(1, 2).view(x.dtype)  # noqa: E731
    s["rows"][0].copy_(_values(part(s["k"]), part(s["ksz"]), cache))
    s["rows"][1].copy_(_values(part(s["v"]), part(s["vsz"]), cache))
    return {"q_rot": s["q_rot"], "k_rows": s["rows"][0], "v_rows": s["rows"][1]}


def _plain_read(s):
    case, i = s["case"], torch.arange(s["case"]["rows"], device="cuda")
    live = i < s["rows"][:, None]
    first, row = _places(s, torch.where(live, s["start"].long()[:, None] + i, s["start"].long()[:, None].clamp(max=max(case["start"] + case["rows"] - 1, 0))))
    if s["table"] is not None:
        first = first.clamp(min=0)
    for x, sz, out in ((s["k"], s["ksz"], s["out"][0]), (s["v"], s["vsz"], s["out"][1])):
        part = lambda y: None if y is None else _raw(y)[first, :, row].transpose(1, 2).view(y.dtype)  # noqa: E731
        out.copy_(torch.where(live[:, None, :, None], _values(part(x), part(sz), case["cache"]), out.float()))
    return {"k": s["out"][0], "v": s["out"][1]}


def _layout(m, s, h_q, window=0):
    kind = {"cache_dtype": m.MQA_U4} if s["case"].get("cache", "u4") == "u4" else {}
    if s["table"] is not None:
        return m.layout_paged(s["k"], s["v"], s["table"], h_q, window, s["ksz"], s["vsz"], **kind)
    return m.layout_contiguous(s["k"], s["v"], h_q, window, s["ksz"], s["vsz"], **kind)


def _own_attn(s):
    import mqa_decode_attention_gb300 as m

    case = s["case"]
    n, most = case["new"], case["tokens"]
    if "layout" not in s:  # the layout and the workspace are made once, as a serving loop keeps them
        s["layout"] = _layout(m, s, case["h_q"], case["window"])
        s["bufs"] = m.DecodeBuffers.allocate(s["layout"], most, n_new=n)
    m.gqa_decode_attention_multi(s["layout"], n, s["q"], s["lens"], most, 1 / math.sqrt(case["head_dim"]), 0, s["out"],
                                 workspace=s["bufs"].workspace, err=s["bufs"].err)
    return {"out": s["out"]}


def _own_append(s):
    import mqa_decode_attention_gb300 as m

    case = s["case"]
    n = case["new"]
    if "layout" not in s:
        s["layout"] = _layout(m, s, case["h_q"])
        s["err"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    m.kv_append_norm_rope(s["layout"], n, s["q_new"], s["k_new"], s["v_new"], s["pos"], ROPE_BASE, s["q_rot"], s["err"], q_weight=s["qw"],
                          k_weight=s["kw"], eps=EPS, axis_pos=s["axis"], sections=_sections(case) if case["axes"] else None)
    if case["cache"] in ("bf16", "f32"):
        return {"q_rot": s["q_rot"], "k": s["k"], "v": s["v"]}
    m.kv_read_rows(s["layout"], s["pos"], None, s["rows"][0], s["rows"][1], s["err"])
    return {"q_rot": s["q_rot"], "k_rows": s["rows"][0], "v_rows": s["rows"][1]}


def _own_read(s):
    import mqa_decode_attention_gb300 as m

    if "layout" not in s:
        s["layout"] = _layout(m, s, s["case"]["h_kv"])
        s["err"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    m.kv_read_rows(s["layout"], s["start"], s["rows"], s["out"][0], s["out"][1], s["err"])
    return {"k": s["out"][0], "v": s["out"][1]}


# ------------------------------------------------------------------ exact
def exact(case, seed):
    s = prepare(case, seed)
    return {"attn": _exact_attn, "append": _exact_append, "read": _exact_read}[case["op"]](s)


def _stored(s, which, b, t):
    """Rows t of sequence b out of the K or V cache, [len(t), h_kv, d] in 64 bits."""
    x, sz = s[which], s[which + "sz"]
    if s["table"] is None:
        a, r = torch.full_like(t, b), t
    else:
        a, r = s["table"][b].long()[t // s["case"]["page"]], t % s["case"]["page"]
    x = _raw(x)[a, :, r].view(x.dtype)
    kind = s["case"].get("cache", "u4")
    if kind == "u4":
        code = torch.empty((*x.shape[:-1], 2 * x.shape[-1]), dtype=torch.float64, device="cuda")
        code[..., 0::2] = (x % 16).double()
        code[..., 1::2] = torch.div(x, 16, rounding_mode="floor").double()
        pair = sz[a, :, r].double()
        return pair[..., 1:] + pair[..., :1] * code
    if kind == "u8":
        pair = sz[a, :, r].double()
        return (x.double() - pair[..., 1:]) * pair[..., :1]
    return x.double()


def _exact_attn(s):
    """Query by query: one softmax in 64 bits over the keys that it sees."""
    case = s["case"]
    n, hq, hk, d, window = (case[k] for k in ("new", "h_q", "h_kv", "head_dim", "window"))
    out = torch.empty(s["out"].shape, dtype=torch.float64, device="cuda")
    for b, length in enumerate(s["host"]):
        low = max(0, length - n + 1 - window) if window else 0
        t = torch.arange(low, length, device="cuda")
        k, v = _stored(s, "k", b, t), _stored(s, "v", b, t)
        for i in range(n):
            end = length - n + 1 + i
            begin = max(0, end - window) if window else 0
            q = s["q"][b, i].double().view(hk, hq // hk, d)
            score = torch.einsum("hgd,thd->hgt", q, k[begin - low:end - low]) / math.sqrt(d)
            out[b, i] = torch.einsum("hgt,thd->hgd", torch.softmax(score, -1), v[begin - low:end - low]).reshape(hq, d)
    return {"out": out}


def _spun(x, w, angle):
    """x [n, heads, d] normalised, its pairs as complex numbers times e^(i angle), angle [n, d / 2], in 64 bits."""
    x = x.double()
    if w is not None:
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS) * w.double()
    z = torch.view_as_complex(x.reshape(*x.shape[:-1], -1, 2).contiguous()) * torch.polar(torch.ones_like(angle), angle)[:, None]
    return torch.view_as_real(z).reshape(x.shape)


def _kept(x, cache):
    """The values that rows x (bf16 values in 64 bits) have in a cache."""
    if cache == "e5m2":  # three significant bits, the smallest step 2^-16
        step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -14))) - 2)
        return torch.round(x / step) * step
    low, high = x.min(-1, keepdim=True).values, x.max(-1, keepdim=True).values
    if cache == "u8":  # defined by its steps in 32 bits
        low, high = low.float(), high.float()
        scale = (high - low) / 255
        scale[scale == 0] = 1
        zero = torch.clamp(torch.round(-low / scale), 0, 255)
        return ((torch.clamp(torch.round(x.float() / scale + zero), 0, 255) - zero) * scale).double()
    want = ((high - low) / 15).clamp(min=2.0 ** -126)
    unit = torch.exp2(torch.floor(torch.log2(want)) - 7)
    scale = torch.ceil(want / unit) * unit
    scale = torch.where((scale - unit) * 15 >= high - low, scale - unit, scale)
    return low + torch.clamp(torch.round((x - low) / scale), 0, 15) * scale


def _exact_append(s):
    """Sequence by sequence."""
    case, cache = s["case"], s["case"]["cache"]
    n, d, quantised = case["new"], case["head_dim"], case["cache"] not in ("bf16", "f32")
    freq = torch.pow(torch.tensor(ROPE_BASE, dtype=torch.float64, device="cuda"), -2.0 * torch.arange(d // 2, device="cuda", dtype=torch.float64) / d)
    q_rot = torch.empty(s["q_rot"].shape, dtype=torch.float64, device="cuda")
    k_all, v_all = (s["rows"][0].double(), s["rows"][1].double()) if quantised else (s["k"].double(), s["v"].double())
    for b, pos in enumerate(s["host"]):
        t = torch.arange(pos, pos + n, device="cuda")
        if s["axis"] is None:
            angle = t.double()[:, None] * freq
        else:
            ends = np.cumsum(_sections(case))
            angle = torch.cat([s["axis"][a, b].double()[:, None] * freq[e - w:e] for a, (e, w) in enumerate(zip(ends, _sections(case)))], 1)
        q_rot[b] = _spun(s["q_new"][b], s["qw"], angle)
        k = _spun(s["k_new"][b], s["kw"], angle).to(s["k_new"].dtype).double()
        v = s["v_new"][b].double()
        if quantised:
            k_all[b], v_all[b] = _kept(k, cache).transpose(0, 1), _kept(v, cache).transpose(0, 1)
            continue
        a, r = (torch.full_like(t, b), t) if s["table"] is None else (s["table"][b].long()[t // case["page"]], t % case["page"])
        k_all[a, :, r], v_all[a, :, r] = k, v
    return {"q_rot": q_rot, "k_rows": k_all, "v_rows": v_all} if quantised else {"q_rot": q_rot, "k": k_all, "v": v_all}


def _exact_read(s):
    """Sequence by sequence; rows past a sequence's count stay as they were."""
    out = [x.double() for x in s["out"]]
    for b, (start, rows) in enumerate(zip(*s["host"])):
        if rows:
            t = torch.arange(start, start + rows, device="cuda")
            for x, which in zip(out, ("k", "v")):
                x[b, :, :rows] = _stored(s, which, b, t).transpose(0, 1)
    return {"k": out[0], "v": out[1]}
