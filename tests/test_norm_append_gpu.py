"""GPU: the append with normalised queries and keys and positions of several axes, into every cache type, against the
fp64 oracle; reading rows back; both with the attention that follows."""

import math

import numpy as np
import pytest
import torch

import oracle
from u4_cases import deal_pages

pytestmark = pytest.mark.gpu
DEV = "cuda"
BASE = 10000.0
CACHES = ["bf16", "f32", "u8", "e5m2", "u4"]


@pytest.fixture(scope="module")
def m(built_lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import mqa_decode_attention_gb300 as mod

    mod.library()
    return mod


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


class Cache:
    """A cache of any type on the device, with rows of its own to begin with."""

    def __init__(self, m, kind, batch, hkv, d, rows, hq, page=0, seed=0):
        g, rng = torch.Generator().manual_seed(seed), np.random.default_rng(seed)
        self.kind, self.page, self.d = kind, page, d
        self.table = None
        if page:
            table, pages = deal_pages(rng, [-(-rows // page)] * batch)
            self.table = torch.from_numpy(table)
            shape = (pages, hkv, page)
        else:
            shape = (batch, hkv, -(-rows // 4) * 4)
        self.t = {}
        for x in "kv":
            sz = None
            if kind == "u4":
                c = torch.randint(0, 256, (*shape, d // 2), generator=g, dtype=torch.uint8)
                sz = torch.rand(*shape, 2, generator=g).to(torch.bfloat16)
            elif kind == "u8":
                c = torch.randint(0, 256, (*shape, d), generator=g, dtype=torch.uint8)
                sz = torch.stack([torch.rand(shape, generator=g), torch.randint(0, 256, shape, generator=g).float()], -1)
            else:
                c = torch.randn(*shape, d, generator=g).to({"bf16": torch.bfloat16, "f32": torch.float32, "e5m2": torch.float8_e5m2}[kind])
            self.t[x], self.t[x + "sz"] = c.to(DEV), None if sz is None else sz.to(DEV)
        t, more = self.t, {"cache_dtype": m.MQA_U4} if kind == "u4" else {}
        if page:
            self.table_dev = self.table.to(DEV)
            self.layout = m.layout_paged(t["k"], t["v"], self.table_dev, hq, 0, t["ksz"], t["vsz"], **more)
        else:
            self.layout = m.layout_contiguous(t["k"], t["v"], hq, 0, t["ksz"], t["vsz"], **more)

    def slot(self, b, t):
        return (b, slice(None), t) if self.table is None else (int(self.table[b, t // self.page]), slice(None), t % self.page)

    def snapshot(self):
        raw = lambda x: None if x is None else (x.view(torch.uint8) if x.dtype == torch.float8_e5m2 else x).cpu().clone()  # noqa: E731
        return {n: raw(x) for n, x in self.t.items()}

    def row(self, snap, which, b, t):
        """The values of row t of sequence b, [Hkv, d] in 64 bits."""
        x = snap[which][self.slot(b, t)]
        if self.kind == "e5m2":
            return oracle.dequantize_e5m2(x.numpy())
        if self.kind in ("bf16", "f32"):
            return x.double().numpy()
        sz = snap[which + "sz"][self.slot(b, t)].double().numpy()
        if self.kind == "u8":
            return oracle.dequantize_u8(x.numpy(), sz[..., 0], sz[..., 1])
        return oracle.dequantize_u4(oracle.unpack_u4(x.numpy()), sz[..., 0], sz[..., 1])

    def encode(self, rows):
        """rows [Hkv, d] as the cache holds them: (tensor, scale rows or None), as `snapshot` gives them."""
        if self.kind == "bf16":
            return torch.from_numpy(rows).to(torch.bfloat16), None
        if self.kind == "f32":
            return torch.from_numpy(rows).float(), None
        if self.kind == "e5m2":
            return torch.from_numpy(oracle.quantize_e5m2(rows)), None
        if self.kind == "u8":
            c, s, z = oracle.quantize_u8(rows)
            return torch.from_numpy(c), torch.from_numpy(np.stack([s, z], -1))
        c, s, z = oracle.quantize_u4(rows)
        return torch.from_numpy(oracle.pack_u4(c)), torch.from_numpy(np.stack([s, z], -1)).to(torch.bfloat16)


def _inputs(kind, B, n, hq, hkv, d, seed, norm="both", sections=None):
    g = torch.Generator().manual_seed(seed)
    dt = torch.float32 if kind == "f32" else torch.bfloat16
    q, k, v = (torch.randn(B, n, h, d, generator=g).to(dt) for h in (hq, hkv, hkv))
    qw = (1 + 0.3 * torch.randn(d, generator=g)).to(dt) if norm in ("both", "q") else None
    kw = (1 + 0.3 * torch.randn(d, generator=g)).to(dt) if norm in ("both", "k") else None
    axis = None if sections is None else torch.randint(-3, 2000, (len(sections), B, n), generator=g, dtype=torch.int32)
    return q, k, v, qw, kw, axis


def _run(m, c, n, x, pos, eps=1e-6, sections=None, q_rot=None):
    q, k, v, qw, kw, axis = (None if t is None else t.to(DEV) for t in x)
    err = _i32([0])
    q_rot = torch.empty(q.shape, device=DEV) if q_rot is None else q_rot
    m.kv_append_norm_rope(c.layout, n, q, k, v, _i32(pos), BASE, q_rot, err, q_weight=qw, k_weight=kw, eps=eps, axis_pos=axis, sections=sections)
    torch.cuda.synchronize()
    return q_rot, int(err)


def _check(c, before, x, pos, q_rot, eps=1e-6, sections=None, only=None):
    """q_rot within fp32 of the oracle's; the new rows bit for bit the oracle's encoding, but for keys whose 64-bit value
    lies so near a border that the pair of floats (2^-36) may fall on its other side; every other row as it was."""
    q, k, v, qw, kw, axis = x
    eps = float(np.float32(eps))  # the call takes an fp32 number
    B, n, hq, d = q.shape
    f32 = c.kind == "f32"
    after = c.snapshot()
    exp = {name: None if t is None else t.clone() for name, t in before.items()}
    widths = [d // 2] if sections is None else sections
    num = lambda t: None if t is None else t.double().numpy()  # noqa: E731
    for b in range(B):
        for i in range(n):
            at = [pos[b] + i] if axis is None else [int(axis[a, b, i]) for a in range(len(widths))]
            want = oracle.norm_rope(num(q[b, i]), num(qw), eps, at, widths, BASE)
            pair = np.sqrt(want[..., 0::2] ** 2 + want[..., 1::2] ** 2)
            # fp32: sine and cosine 2^-25, two products and a sum 2^-23; norm and weight 2^-21
            assert np.all(np.abs(q_rot[b, i].double().cpu().numpy() - want) <= np.repeat(pair, 2, -1) * 1.5 * 2.0 ** -21 + 1e-37)
            if only is not None and b not in only:
                continue
            key = oracle.norm_rope(num(k[b, i]), num(kw), eps, at, widths, BASE)
            slot = c.slot(b, pos[b] + i)
            rounded = key.astype(np.float32).astype(np.float64) if f32 else oracle.round_bf16(key)
            length = np.repeat(np.sqrt(key[..., 0::2] ** 2 + key[..., 1::2] ** 2), 2, -1)
            near = [(key.astype(np.float64) + s * length * 2.0 ** -36) for s in (-1, 1)]
            near = [t.astype(np.float32).astype(np.float64) if f32 else oracle.round_bf16(t) for t in near]
            open_rows = np.any(near[0] != near[1], -1)  # [Hkv]
            for name, rows in (("k", rounded), ("v", num(v[b, i]))):
                t, sz = c.encode(rows)
                keep = open_rows if name == "k" else np.zeros_like(open_rows)
                for j in range(rows.shape[0]):
                    js = (slot[0], j, slot[2])
                    if keep[j]:
                        got = c.row(after, name, b, pos[b] + i)[j]
                        lim = np.abs(rows[j]).max() * {"f32": 2.0 ** -23, "bf16": 2.0 ** -7, "e5m2": 2.0 ** -1, "u8": 2 / 255, "u4": 2 / 15}[c.kind]
                        assert np.all(np.abs(got - rows[j]) <= lim)
                        exp[name][js] = after[name][js]
                        if sz is not None:
                            exp[name + "sz"][js] = after[name + "sz"][js]
                        continue
                    exp[name][js] = t[j]
                    if sz is not None:
                        exp[name + "sz"][js] = sz[j]
    for name in exp:
        if exp[name] is None:
            continue
        if c.kind in ("bf16", "f32"):  # as numbers: a zero of either sign is the same value
            assert torch.equal(after[name], exp[name]), name
        else:
            assert np.array_equal(after[name].view(torch.uint8).numpy(), exp[name].contiguous().view(torch.uint8).numpy()), name


SHAPES = {
    # name: (hq, hkv, d, pos, n, page, norm, sections)
    "norm": (8, 2, 128, [0, 5, 77], 1, 0, "both", None),
    "norm_paged_several": (6, 3, 64, [0, 13, 40], 5, 16, "both", None),
    "axes3": (8, 2, 128, [0, 9], 3, 0, "both", [24, 20, 20]),
    "axes4_d64": (4, 4, 64, [3, 100], 2, 32, "both", [8, 0, 20, 4]),
    "axes2_no_norm": (21, 3, 64, [1, 64], 4, 0, None, [11, 21]),
    "only_q": (4, 1, 128, [31], 2, 0, "q", None),
    "only_k": (4, 1, 128, [31], 2, 16, "k", [0, 64]),
    "prompt": (5, 1, 128, [0, 3], 150, 64, "both", [16, 24, 24]),
    "long_prompt": (5, 1, 64, [0, 3, 40, 9, 600], 487, 16, "both", [16, 10, 6]),
    "one_head": (1, 1, 64, [0], 1, 0, "both", None),
    "many_heads": (64, 64, 64, [2], 1, 0, "both", None),
}


@pytest.mark.parametrize("kind", CACHES)
@pytest.mark.parametrize("name", list(SHAPES))
def test_append(m, name, kind):
    hq, hkv, d, pos, n, page, norm, sections = SHAPES[name]
    c = Cache(m, kind, len(pos), hkv, d, max(pos) + n, hq, page, seed=len(name))
    x = _inputs(kind, len(pos), n, hq, hkv, d, 7, norm, sections)
    before = c.snapshot()
    q_rot, err = _run(m, c, n, x, pos, sections=sections)
    assert err == 0
    _check(c, before, x, pos, q_rot, sections=sections)


@pytest.mark.parametrize("kind", CACHES)
def test_plain_call_is_the_append(m, kind):
    """Without weights and axes: q_rot and the rows of kv_append_rope (a one-byte cache's key takes a rounding to bf16
    more here: its codes may differ by one step, and its values not at all)."""
    B, n, hq, hkv, d, pos = 3, 4, 8, 2, 128, [0, 30, 200]
    x = _inputs(kind, B, n, hq, hkv, d, 3, None)
    a, b = (Cache(m, kind, B, hkv, d, 204, hq, 16, seed=1) for _ in range(2))
    q_rot, err = _run(m, a, n, x, pos)
    word, other = _i32([0]), torch.empty(B, n, hq, d, device=DEV)
    m.kv_append_rope_multi(b.layout, n, *(t.to(DEV) for t in x[:3]), _i32(pos), BASE, other, word)
    torch.cuda.synchronize()
    assert err == 0 and int(word) == 0
    pair = x[0].double().abs()
    pair = (pair[..., 0::2] + pair[..., 1::2]).repeat_interleave(2, -1)
    assert torch.all((q_rot - other).double().cpu().abs() <= pair * 2.0 ** -21)
    sa, sb = a.snapshot(), b.snapshot()
    same = ["v", "vsz"] + (["k", "ksz"] if kind in ("bf16", "u4") else [])
    for name in same:
        if sa[name] is not None:
            assert np.array_equal(sa[name].view(torch.uint8).numpy(), sb[name].view(torch.uint8).numpy()), name


@pytest.mark.parametrize("eps", [1e-30, 1e-6, 10.0])
def test_sizes_of_values(m, eps):
    """Rows of zeros, of tiny and of huge values: the squares of the last leave the fp32 range."""
    B, n, hq, hkv, d = 8, 1, 4, 4, 128
    c = Cache(m, "bf16", B, hkv, d, 4, hq)
    x = list(_inputs("bf16", B, n, hq, hkv, d, 11))
    size = torch.tensor([0.0, 1e-18, 1e-9, 1e-3, 1e3, 1e15, 1e25, 1e37]).view(B, 1, 1, 1)
    x[0], x[1] = (x[0].float() * size).to(torch.bfloat16), (x[1].float() * size).to(torch.bfloat16)
    before = c.snapshot()
    q_rot, err = _run(m, c, n, x, [1] * B, eps=eps)
    assert err == 0
    _check(c, before, x, [1] * B, q_rot, eps=eps)


def test_far_positions(m):
    """Angles of positions up to the largest and the smallest int32."""
    B, d, ends = 4, 128, [2 ** 31 - 1, -2 ** 31, 10 ** 6 + 1, -1]
    for kind in ("bf16", "u4"):
        c = Cache(m, kind, B, 2, d, 8, 4)
        x = list(_inputs(kind, B, 1, 4, 2, d, 12, "both", [64]))
        x[5] = torch.tensor(ends, dtype=torch.int32).view(1, B, 1)
        before = c.snapshot()
        q_rot, err = _run(m, c, 1, x, [0, 1, 2, 3], sections=[64])
        assert err == 0
        # the angle itself is rounded to 64 bits: 2^31 2^-53 of a turn
        q, k, v, qw, kw, axis = x
        for b in range(B):
            want = oracle.norm_rope(q[b, 0].double().numpy(), qw.double().numpy(), 1e-6, [ends[b]], [64], BASE)
            pair = np.repeat(np.sqrt(want[..., 0::2] ** 2 + want[..., 1::2] ** 2), 2, -1)
            assert np.all(np.abs(q_rot[b, 0].double().cpu().numpy() - want) <= pair * (2.0 ** -20 + 2.0 ** -20))


def test_out_of_range(m):
    for page in (0, 16):
        c = Cache(m, "u4", 4, 2, 128, 40, 4, page, seed=5)
        x = _inputs("u4", 4, 1, 4, 2, 128, 13)
        pos = [39, -1, 4 * 16 if page else 40, 7]
        if page:
            c.table_dev[3, 0] = -7
        before = c.snapshot()
        q_rot, err = _run(m, c, 1, x, pos, q_rot=torch.full((4, 1, 4, 128), 9.0, device=DEV))
        assert err == m.MQA_DEVERR_POS_RANGE | (m.MQA_DEVERR_PAGE_RANGE if page else 0)
        _check(c, before, x, pos, q_rot, only=[0] if page else [0, 3])


@pytest.mark.parametrize("kind", CACHES)
def test_places_of_16_bytes(m, kind):
    """Outputs whose addresses are multiples of 16 bytes, not of 32: the append's query, rows read back."""
    for d, page in ((128, 0), (64, 16)):
        c = Cache(m, kind, 3, 3, d, 70, 9, page, seed=9)
        x = _inputs(kind, 3, 2, 9, 3, d, 19)
        before = c.snapshot()
        memory = torch.full((3 * 2 * 9 * d + 8,), 9.0, device=DEV)
        q_rot, err = _run(m, c, 2, x, [0, 31, 68], q_rot=memory[4:-4].view(3, 2, 9, d))
        assert err == 0 and torch.all(memory[:4] == 9.0) and torch.all(memory[-4:] == 9.0)
        _check(c, before, x, [0, 31, 68], q_rot)
        for dt, step in ((torch.bfloat16, 8), (torch.float32, 4)):
            aligned = [torch.empty(3, 3, 70, d, dtype=dt, device=DEV) for _ in "kv"]
            shifted = [torch.full((3 * 3 * 70 * d + 2 * step,), 9.0, dtype=dt, device=DEV) for _ in "kv"]
            err = _i32([0])
            m.kv_read_rows(c.layout, None, None, *aligned, err)
            m.kv_read_rows(c.layout, None, None, *(t[step:-step].view(3, 3, 70, d) for t in shifted), err)
            torch.cuda.synchronize()
            assert int(err) == 0
            for a, t in zip(aligned, shifted):
                assert torch.equal(t[step:-step].view_as(a).nan_to_num(7.0), a.nan_to_num(7.0))
                assert torch.all(t[:step] == 9.0) and torch.all(t[-step:] == 9.0)


def test_not_finite(m):
    """A key with a value that is not finite: NaN in its row only."""
    c = Cache(m, "bf16", 2, 2, 64, 4, 2)
    x = _inputs("bf16", 2, 1, 2, 2, 64, 14)
    x[1][1, 0, 1, 7] = float("inf")
    x[0][0, 0, 1, 3] = float("nan")
    q_rot, err = _run(m, c, 1, x, [0, 0])
    k = c.t["k"].cpu()
    assert err == 0 and torch.isnan(k[1, 1, 0]).any() and torch.isfinite(k[0, :, 0]).all() and torch.isfinite(k[1, 0, 0]).all()
    assert torch.isnan(q_rot[0, 0, 1]).any() and torch.isfinite(q_rot[0, 0, 0]).all() and torch.isfinite(q_rot[1]).all()


def test_norm_then_attention(m):
    """A decode loop with normalised heads over the 4-bit cache: append, then attention, captured and replayed."""
    B, hq, hkv, d, steps = 2, 8, 2, 128, 12
    c = Cache(m, "u4", B, hkv, d, steps, hq, 16, seed=8)
    bufs = m.DecodeBuffers.allocate(c.layout, steps)
    x = [t.to(DEV) for t in _inputs("u4", B, 1, hq, hkv, d, 15)[:5]]
    axis, pos, lens = torch.zeros(3, B, 1, dtype=torch.int32, device=DEV), _i32([0] * B), _i32([1] * B)

    def step():
        m.kv_append_norm_rope(c.layout, 1, x[0], x[1], x[2], pos, BASE, bufs.q_rot, bufs.err, q_weight=x[3], k_weight=x[4], axis_pos=axis,
                              sections=[16, 24, 24])
        m.gqa_decode_attention(c.layout, bufs.q_rot, lens, steps, 1 / math.sqrt(d), 0, bufs.out, bufs.lse, bufs.workspace, err=bufs.err)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    g = torch.Generator().manual_seed(4)
    K, V = np.zeros((B, hkv, steps, d)), np.zeros((B, hkv, steps, d))
    for t in range(steps):
        new = [torch.randn(y.shape, generator=g).to(torch.bfloat16) for y in x[:3]]
        for y, z in zip(x, new):
            y.copy_(z)
        axis.copy_(torch.tensor([[t], [t // 3], [t % 3]], dtype=torch.int32).view(3, 1, 1).expand(3, B, 1))
        pos.fill_(t)
        lens.fill_(t + 1)
        graph.replay()
        torch.cuda.synchronize()
        assert int(bufs.err) == 0
        snap = c.snapshot()
        for b in range(B):
            K[b, :, t], V[b, :, t] = c.row(snap, "k", b, t), c.row(snap, "v", b, t)
            key = oracle.norm_rope(new[1][b, 0].double().numpy(), x[4].double().cpu().numpy(), 1e-6, [t, t // 3, t % 3], [16, 24, 24], BASE)
            step_of = (key.max(-1) - key.min(-1)) / 15
            assert np.all(np.abs(K[b, :, t] - key) <= step_of[:, None] * 0.52 + np.abs(key).max() * 2.0 ** -7)
            ref, _ = oracle.attention_values(bufs.q_rot[b][None].double().cpu().numpy(), K[b, :, : t + 1], V[b, :, : t + 1], t, 1 / math.sqrt(d))
            got = bufs.out[b].double().cpu().numpy()
            assert np.all(np.abs(got - ref[0]) <= np.abs(ref[0]) * 2.0 ** -8 + 0.05)


# ------------------------------------------------------------ reading back
READ = {
    # name: (hkv, d, start, rows, n, page)
    "whole": (2, 128, None, None, 130, 0),
    "ragged": (3, 64, [0, 5, 100, 7], [130, 0, 1, 64], 130, 0),
    "paged": (2, 128, [0, 15, 33, 64], [100, 50, 17, 1], 100, 16),
    "paged_d64": (5, 64, [1, 2, 3, 4], [63, 64, 65, 200], 200, 64),
    "one": (1, 128, [9, 0, 0, 0], None, 1, 32),
}


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kind", CACHES)
@pytest.mark.parametrize("name", list(READ))
def test_read(m, name, kind, out):
    hkv, d, start, rows, n, page = READ[name]
    B = 4
    most = max((s + r for s, r in zip(start or [0] * B, rows or [n] * B)))
    c = Cache(m, kind, B, hkv, d, most, hkv, page, seed=len(name))
    k, v = (torch.full((B, hkv, n, d), 5.0, dtype=out, device=DEV) for _ in range(2))
    err = _i32([0])
    m.kv_read_rows(c.layout, None if start is None else _i32(start), None if rows is None else _i32(rows), k, v, err)
    torch.cuda.synchronize()
    assert int(err) == 0
    snap = c.snapshot()
    for b in range(B):
        r = n if rows is None else rows[b]
        for got, which in ((k, "k"), (v, "v")):
            x = got[b].double().cpu().numpy()
            assert np.all(x[:, r:] == 5.0)
            for i in range(r):
                want = c.row(snap, which, b, (start[b] if start else 0) + i)
                # one or two fp32 operations, then the rounding to bf16
                tol = np.abs(want) * (2.0 ** -8 * 1.001 if out is torch.bfloat16 else 2.0 ** -23)
                if kind in ("u4", "u8"):
                    tol = tol + np.abs(c.row(snap, which, b, (start[b] if start else 0) + i)).max() * 2.0 ** -22
                if kind in ("bf16", "e5m2") or (kind == "f32" and out is torch.float32):
                    tol = 0.0
                assert np.all(np.abs(x[:, i] - want) <= tol), (b, i)


@pytest.mark.parametrize("kind", CACHES)
def test_read_out_of_range(m, kind):
    """A sequence out of range, and rows of a page outside the pool, are left as they were."""
    for page in (0, 16):
        c = Cache(m, kind, 5, 2, 128, 64, 2, page, seed=2)
        if page:
            c.table_dev[4, 1] = 10 ** 9
        limit = 5 * 16 if page else 64
        start, rows = [-1, limit - 3, 0, 60, 10], [4, 4, 9, 4, 8]
        k, v = (torch.full((5, 2, 8, 128), 5.0, dtype=torch.float32, device=DEV) for _ in range(2))
        err = _i32([0])
        m.kv_read_rows(c.layout, _i32(start), _i32(rows), k, v, err)
        torch.cuda.synchronize()
        want = m.MQA_DEVERR_POS_RANGE | m.MQA_DEVERR_SEQ_LEN | (m.MQA_DEVERR_PAGE_RANGE if page else 0)
        assert int(err) == want
        assert torch.all(k[:3] == 5.0) and torch.all(v[:3] == 5.0)
        snap = c.snapshot()
        for b, r in ((3, range(4)), (4, range(6) if page else range(8))):
            for i in r:
                assert np.allclose(k[b, :, i].double().cpu().numpy(), c.row(snap, "k", b, start[b] + i), rtol=1e-5, atol=1e-4)
        if page:
            assert torch.all(k[4, :, 6:] == 5.0)


def test_read_of_large_caches(m):
    """Offsets past 32 bits: rows of the last head of a contiguous cache of 5 GB."""
    B, hkv, cap, d = 1, 40, 1 << 20, 128
    k = torch.zeros(B, hkv, cap, d, dtype=torch.uint8, device=DEV)
    sz = torch.ones(B, hkv, cap, 2, device=DEV)
    k[0, -1, -5:] = torch.arange(5, dtype=torch.uint8, device=DEV)[:, None] + 1
    lay = m.layout_contiguous(k, k.clone(), hkv, 0, sz, sz)
    out, err = [torch.zeros(B, hkv, 8, d, device=DEV) for _ in range(2)], _i32([0])
    m.kv_read_rows(lay, _i32([cap - 8]), None, *out, err)
    torch.cuda.synchronize()
    assert int(err) == 0
    assert out[0][0, -1, :, 7].tolist() == [-1.0, -1.0, -1.0, 0.0, 1.0, 2.0, 3.0, 4.0]


def test_prefix_in_four_bits_then_prefill(m):
    """A prompt whose prefix lies in the 4-bit cache: its rows are read back as a bf16 cache, the rest of the prompt is
    prefilled over it, and appended to the 4-bit cache as well; the next token is decoded over that."""
    B, hq, hkv, d, prefix, n = 2, 8, 2, 128, 40, 24
    c = Cache(m, "u4", B, hkv, d, 80, hq, 16, seed=21)
    err = _i32([0])
    first = _inputs("u4", B, prefix, hq, hkv, d, 31, None)
    _run(m, c, prefix, first, [0] * B)
    k = torch.zeros(B, hkv, 64, d, dtype=torch.bfloat16, device=DEV)
    v = torch.zeros_like(k)
    m.kv_read_rows(c.layout, None, _i32([prefix] * B), k, v, err)
    snap = c.snapshot()
    lay = m.layout_contiguous(k, v, hq)
    q, kn, vn = (t.to(DEV) for t in _inputs("u4", B, n, hq, hkv, d, 32, None)[:3])
    bufs = m.DecodeBuffers.allocate(lay, prefix + n, num_splits=1, n_new=n)
    m.prefill_step(lay, n, q, kn, vn, _i32([prefix] * B), _i32([prefix + n] * B), prefix + n, bufs)
    q_rot = torch.empty(B, n, hq, d, device=DEV)
    m.kv_append_rope_multi(c.layout, n, q, kn, vn, _i32([prefix] * B), BASE, q_rot, err)
    torch.cuda.synchronize()
    assert int(err) == 0 and int(bufs.err) == 0
    for b in range(B):
        for t in range(prefix):  # the rows read back, each rounded once more to bf16
            want = c.row(snap, "k", b, t)
            assert np.all(np.abs(k[b, :, t].double().cpu().numpy() - want) <= np.abs(want) * 2.0 ** -8 * 1.001 + 1e-6)
        ref, _ = oracle.attention_values(q_rot[b].double().cpu().numpy(), k[b, :, : prefix + n].double().cpu().numpy(),
                                         v[b, :, : prefix + n].double().cpu().numpy(), prefix, 1 / math.sqrt(d))
        assert np.max(np.abs(bufs.out[b].double().cpu().numpy() - ref)) <= 2e-2
    one = [t.to(DEV) for t in _inputs("u4", B, 1, hq, hkv, d, 33, None)[:3]]
    db = m.DecodeBuffers.allocate(c.layout, prefix + n + 1)
    m.decode_step(c.layout, *one, _i32([prefix + n] * B), _i32([prefix + n + 1] * B), prefix + n + 1, db)
    torch.cuda.synchronize()
    assert int(db.err) == 0
    snap = c.snapshot()
    for b in range(B):
        K, V = (np.stack([c.row(snap, w, b, t) for t in range(prefix + n + 1)], 1) for w in "kv")
        ref, _ = oracle.attention_values(db.q_rot[b][None].double().cpu().numpy(), K, V, prefix + n, 1 / math.sqrt(d))
        assert np.max(np.abs(db.out[b].double().cpu().numpy() - ref[0])) <= 2e-2
