"""GPU: the tree step at its edges: the wide append's bits, waits that run out,
many runs of one call, two streams at once, launches without work."""

import math

import numpy as np
import pytest
import torch

import oracle
from test_tree_gpu import check, check_append, check_attention, live, m, run_step  # noqa: F401 (m: fixture)
from tree_cases import TreeCase, raw

pytestmark = pytest.mark.gpu


def step(mod, c, lay, t, bufs):
    mod.tree_step(lay, c.n, t.q_new, t.k_new, t.v_new, t.pos, t.depth, t.mask, c.max_len, bufs, num_nodes=t.num)


# ------------------------------------------------------------------ append

@pytest.mark.parametrize("page", [0, 16])
@pytest.mark.parametrize("hq,hkv,d,n", [(32, 8, 128, 16), (6, 2, 64, 31), (7, 1, 128, 128)])
def test_wide_append_is_the_narrow_one(m, hq, hkv, d, n, page):  # noqa: F811
    """Calls of 256 nodes and more take another kernel: the bytes it leaves are
    those of one call per sequence, NaN and infinite inputs included (every pair
    of theirs takes the kernel's fp64 path, more than it can note at once)."""
    B = 2600 // n
    rng = np.random.default_rng(n)
    pos = [int(x) for x in rng.integers(0, 90000, B)]
    pos[0] = 0
    cap_pos = pos if page else [x % 300 for x in pos]
    nodes = [int(x) for x in rng.integers(0, n + 1, B)]
    nodes[1] = n
    # (paged: the cached tokens' pages all are one page, the nodes' their own)
    c = TreeCase(hq, hkv, d, [0] * B if page else cap_pos, nodes if not page else [n] * B, n, "bf16", page, seed=n + page)
    c.k_new[1, :, 0, : d // 2] = float("inf")
    c.k_new[2, n // 2] = float("nan")
    c.k_new[3, 0] = 0.0
    c.nodes = nodes
    if page:  # positions far out: the table's entries from slot pos / page on are the sequence's pages
        wide = max(pos) // page + c.table.shape[1] + 2
        table = np.zeros((B, wide), np.int32)
        for b in range(B):
            at = pos[b] // page
            own = c.table[b][c.table[b] >= 0]
            table[b, at:at + len(own)] = own
            pos[b] = at * page
        c.table = table
    else:
        pos = cap_pos
    out = []
    for split in (False, True):
        lay, t = c.gpu(m)
        t.pos = torch.tensor(pos, dtype=torch.int32, device="cuda")
        q_rot = torch.full((B, n, hq, d), 3.0, dtype=torch.bfloat16, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        if not split:
            assert B * n >= 256
            m.kv_append_rope_tree(lay, n, t.q_new, t.k_new, t.v_new, t.pos, t.depth, 10000.0, q_rot, err, t.num)
        else:
            for b in range(B):
                s = slice(b, b + 1)
                one = (m.layout_paged(t.k, t.v, t.table[s], hq) if page else m.layout_contiguous(t.k[s], t.v[s], hq))
                m.kv_append_rope_tree(one, n, t.q_new[s], t.k_new[s], t.v_new[s], t.pos[s], t.depth[s], 10000.0, q_rot[s],
                                      err, t.num[s])
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        out.append((t.k, t.v, q_rot))
    for name, a, b in zip("kv", *out):
        nan = a.isnan()
        assert torch.equal(nan, b.isnan()), name
        differ = (a.view(torch.int16) != b.view(torch.int16)) & ~nan
        assert int(differ.sum()) == 0, (name, a[differ][:4], b[differ][:4])
    # q_rot: each the fp32 rotation rounded once, whose products may be fused either way
    rows = live(c)
    want = oracle.tree_rotate(c.q_new, pos, c.depth, 10000.0)[rows]
    step_ = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(want), 2.0 ** -100))) - 7)
    for _, _, q in out:
        assert np.all(np.abs(raw(q)[rows] - want) <= 0.5 * step_ + 1e-6 * np.abs(want).max())
    rows = torch.from_numpy(rows).cuda()
    assert (out[0][2][~rows] == 3.0).all()


def test_wide_append_errors(m):  # noqa: F811
    n, B = 16, 20
    c = TreeCase(8, 2, 128, [20] * B, [n] * B, n)
    bad = dict(nodes=m.MQA_DEVERR_SEQ_LEN, many=m.MQA_DEVERR_SEQ_LEN, depth=m.MQA_DEVERR_TREE, pos=m.MQA_DEVERR_POS_RANGE,
               far=m.MQA_DEVERR_POS_RANGE, page=m.MQA_DEVERR_PAGE_RANGE)
    for page in (0, 16):
        c = TreeCase(8, 2, 128, [20] * B, [n] * B, n, page=page)
        for what, bit in bad.items():
            if what == "page" and not page:
                continue
            lay, t = c.gpu(m)
            before = t.k.clone()
            b = m.TreeBuffers.allocate(lay, n)
            if what == "nodes":
                t.num[3] = -1
            elif what == "many":
                t.num[3] = n + 1
            elif what == "depth":
                t.depth[3, 2] = n
            elif what == "pos":
                t.pos[3] = -2
            elif what == "far":
                t.pos[3] = (t.table.shape[1] * page if page else lay.capacity) - 2
                if page:
                    t.table[3, -1] = int(t.table[3, 0])
            else:
                t.table[3, 1] = 10 ** 6
            m.kv_append_rope_tree(lay, n, t.q_new, t.k_new, t.v_new, t.pos, t.depth, 10000.0, b.q_rot, b.err, t.num)
            torch.cuda.synchronize()
            assert int(b.err.item()) == bit, what
            same = (t.k == before) | (t.k.isnan() & before.isnan())
            if not page and what in ("nodes", "many"):
                assert same[3].all()
            elif not page and what == "pos":
                assert same[3, :, 20:].all()  # (nodes 2.. land in rows 0..)


@pytest.mark.parametrize("d", [64, 128])
def test_wide_step(m, d):  # noqa: F811
    """A step whose append is the wide one, its nodes' rows held to the oracle."""
    rng = np.random.default_rng(5)
    pos = [int(x) for x in rng.integers(0, 300, 30)]
    nodes = [int(x) for x in rng.integers(0, 12, 30)]
    for page in (0, 16):
        check(m, TreeCase(8, 2, d, pos, nodes, 11, "bf16", page, seed=4))


# ---------------------------------------------------------- bounded waits

@pytest.mark.parametrize("cache", ["bf16", "e5m2", "u8"])
@pytest.mark.parametrize("nodes", [8, 64])  # one row tile, two of them
@pytest.mark.parametrize("page", [0, 16])
def test_waits_that_run_out(m, cache, nodes, page):  # noqa: F811
    """With a limit of one nanosecond any wait that is not over at once runs out:
    the launch reports it and comes back, and the next one is as always."""
    c = TreeCase(32, 8, 128, [1500, 300, 900], [nodes, 5, nodes - 3], nodes, cache, page)
    _, ref = run_step(m, c)
    lay, t = c.gpu(m)
    bufs = m.TreeBuffers.allocate(lay, c.n, lse=True)
    for _ in range(3):
        lay.wait_limit_ns = 1
        bufs.err.zero_()
        step(m, c, lay, t, bufs)
        torch.cuda.synchronize()
        assert int(bufs.err.item()) & m.MQA_DEVERR_TIMEOUT
        lay.wait_limit_ns = 0
        bufs.err.zero_()
        bufs.out.fill_(7.0)
        bufs.lse.fill_(7.0)
        step(m, c, lay, t, bufs)
        torch.cuda.synchronize()
        assert int(bufs.err.item()) == 0
        assert torch.equal(bufs.out, ref.out) and torch.equal(bufs.lse, ref.lse)


# --------------------------------------------------------- many runs, streams

@pytest.mark.parametrize("cache", ["bf16", "e5m2", "u8"])
@pytest.mark.parametrize("d", [128, 64])
def test_many_runs_give_the_same_bits(m, cache, d):  # noqa: F811
    """Units of one and two row tiles in runs of several units, 400 times over."""
    rng = np.random.default_rng(9)
    pos = [int(x) for x in rng.integers(0, 1500, 40)]
    nodes = [int(x) for x in rng.integers(0, 33, 40)]
    c = TreeCase(16, 2, d, pos, nodes, 32, cache, 16, seed=2)
    lay, t = c.gpu(m)
    bufs = m.TreeBuffers.allocate(lay, c.n, lse=True)
    bufs.out.fill_(7.0)
    bufs.lse.fill_(7.0)
    step(m, c, lay, t, bufs)
    torch.cuda.synchronize()
    want, want_lse = bufs.out.clone(), bufs.lse.clone()
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(400):
        bufs.out.fill_(7.0)
        bufs.lse.fill_(7.0)
        step(m, c, lay, t, bufs)
        wrong += (bufs.out != want).sum() + (bufs.lse != want_lse).sum()
    torch.cuda.synchronize()
    assert int(bufs.err.item()) == 0
    assert int(wrong.item()) == 0


def test_two_streams_at_once(m):  # noqa: F811
    """Two steps in flight together, each with its own cache and buffers."""
    cases = [TreeCase(32, 8, 128, [2000, 700], [16, 9], 16, "bf16", 16, seed=1),
             TreeCase(32, 8, 128, [900, 1900], [64, 33], 64, "e5m2", 0, seed=2)]
    refs = [run_step(m, c)[1] for c in cases]
    got = []
    for c in cases:
        lay, t = c.gpu(m)
        bufs = m.TreeBuffers.allocate(lay, c.n, lse=True)
        bufs.out.fill_(7.0)
        got.append((c, lay, t, bufs, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(50):
        for c, lay, t, bufs, s in got:
            with torch.cuda.stream(s):
                step(m, c, lay, t, bufs)
    torch.cuda.synchronize()
    for (c, lay, t, bufs, s), ref in zip(got, refs):
        assert int(bufs.err.item()) == 0
        assert torch.equal(bufs.out, ref.out)


@pytest.mark.parametrize("cache", ["bf16", "e5m2", "u8"])
@pytest.mark.parametrize("d", [128, 64])
def test_no_nodes_at_all(m, cache, d):  # noqa: F811
    """A call none of whose sequences drafts anything leaves everything as it was."""
    c = TreeCase(16, 2, d, [300, 0, 70], [0, 0, 0], 7, cache)
    t, bufs = run_step(m, c)
    assert int(bufs.err.item()) == 0
    assert (bufs.out == 7).all() and (bufs.lse == 7).all()
    assert np.array_equal(raw(t.v), raw(c.v), equal_nan=True) and np.array_equal(raw(t.k), raw(c.k), equal_nan=True)


def test_append_without_attention_is_seen_by_the_next_call(m):  # noqa: F811
    """What follows the step in its stream finds the append's rows there, also
    behind a step that had nothing to attend for."""
    c = TreeCase(16, 2, 128, [300, 200], [9, 8], 9, garbage=False)
    lay, t = c.gpu(m)
    bufs = m.TreeBuffers.allocate(lay, c.n)
    step(m, c, lay, t, bufs)
    k = t.k.clone()
    torch.cuda.synchronize()
    check_append(c, t, bufs.q_rot)
    assert torch.equal(k, t.k)


def test_a_scale_of_any_size(m):  # noqa: F811
    """The softmax scale enters the exponent only: a tiny one weighs all keys alike, a large one picks one."""
    c = TreeCase(8, 2, 128, [500], [6], 6, garbage=False)
    lay, t = c.gpu(m)
    b = m.TreeBuffers.allocate(lay, 6)
    m.tree_step(lay, 6, t.q_new, t.k_new, t.v_new, t.pos, t.depth, t.mask, c.max_len, b, scale=1e-30)
    torch.cuda.synchronize()
    att = np.concatenate([np.ones((6, 500), bool), c.bits[0]], 1)
    v = raw(t.v)[0][:, :506]  # [hkv, keys, d]
    got = raw(b.out)[0].reshape(6, 2, 4, 128)
    for i in range(6):
        mean, size = v[:, att[i]].mean(1), np.abs(v[:, att[i]]).mean(1)
        # bf16: the output (P = 1 exactly); fp32: a sum of 506 terms
        bound = 2.0 ** -8 * np.abs(mean) + 520 * 2.0 ** -24 * size * 2
        assert np.all(np.abs(got[i] - mean[:, None]) <= bound[:, None])
    m.tree_step(lay, 6, t.q_new, t.k_new, t.v_new, t.pos, t.depth, t.mask, c.max_len, b, scale=1e4)
    torch.cuda.synchronize()
    assert torch.isfinite(b.out).all()
    q, k = raw(b.q_rot)[0].reshape(6, 2, 4, 128), raw(t.k)[0][:, :506]
    s = np.einsum("ijgd,jtd->ijgt", q, k)
    s[np.broadcast_to(~att[:, None, None], s.shape)] = -np.inf
    two = np.sort(s, -1)[..., -2:]
    clear = (two[..., 1] - two[..., 0]) * 1e4 > 60  # e^-60 of the second
    pick = np.take_along_axis(v[None, :, None], s.argmax(-1)[..., None, None], 3)[..., 0, :]
    got = raw(b.out)[0].reshape(6, 2, 4, 128)
    assert clear.any()
    assert np.all(np.abs(got - pick)[clear] <= 2 * 2.0 ** -8 * np.abs(pick)[clear] + 2.0 ** -22)  # P and the output in bf16
    assert math.isfinite(float(b.out.float().abs().max()))


@pytest.mark.parametrize("d", [128, 64])
def test_u8_every_code_and_zero_point(m, d):  # noqa: F811
    """Every code with zero points from end to end, scales over 2^-20 .. 2^20: an
    exact widening (one row attended: the value itself comes out)."""
    T = 256
    B = 3
    g = torch.Generator().manual_seed(1)
    k = torch.randint(0, 256, (B, 2, T + 2, d), generator=g, dtype=torch.int32).to(torch.uint8)
    v = ((torch.arange(T + 2)[:, None] * 3 + torch.arange(d)) % 256).to(torch.uint8).expand(B, 2, -1, -1).contiguous()
    ksz = torch.ones(B, 2, T + 2, 2)
    ksz[..., 1] = 128
    vsz = torch.ones(B, 2, T + 2, 2)
    vsz[..., 1] = (torch.arange(T + 2) * 7 % 256).float()
    vsz[..., 0] = 2.0 ** (torch.arange(T + 2) % 41 - 20).float()
    k, v, ksz, vsz = (x.cuda().contiguous() for x in (k, v, ksz, vsz))
    lay = m.layout_contiguous(k, v, 4, 0, ksz, vsz)
    q = torch.zeros(B, 1, 4, d, dtype=torch.bfloat16, device="cuda")
    out = torch.zeros(B, 1, 4, d, device="cuda")
    bufs = m.TreeBuffers.allocate(lay, 1)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    for t in range(0, T, 5):  # a window of one: the node attends to itself alone, cache row t
        lay = m.layout_contiguous(k, v, 4, 1, ksz, vsz)
        pos = i32([t, (t + 1) % T, (t + 2) % T])
        m.gqa_tree_attention(lay, 1, q, pos, i32([[0]] * 3), i32([[[1]]] * 3), T + 2, 1.0, out, None, None, bufs.workspace,
                             bufs.err)
        torch.cuda.synchronize()
        assert int(bufs.err.item()) == 0
        for b, at in enumerate(pos.tolist()):
            want = (v[b, 0, at].float() - vsz[b, 0, at, 1]) * vsz[b, 0, at, 0]
            assert torch.equal(out[b, 0], want.expand(4, d))


@pytest.mark.parametrize("cache,d,hq,hkv,nodes", [("bf16", 128, 32, 8, 9), ("bf16", 128, 32, 8, 60), ("bf16", 64, 12, 3, 31),
                                                  ("e5m2", 64, 12, 3, 31), ("u8", 64, 12, 3, 31), ("bf16", 128, 160, 1, 2),
                                                  ("e5m2", 128, 32, 8, 60)])
@pytest.mark.parametrize("page", [0, 16])
def test_probabilities_keep_more_than_a_bf16(m, cache, d, hq, hkv, nodes, page):  # noqa: F811
    """fp32 outputs against the oracle's on the same operands: P as two bf16 terms
    is within 2^-7 (what the first leaves) times 2^-8 (the second's rounding) =
    2^-15 of its value; as an f16 (e5m2, head_dim 128) within 2^-11, or 2^-25 where
    it is below 2^-14 and the row's largest at least 1: 700 keys, 2^-15 at most of
    the largest |v|, which is below 2^3 and over the mean |v| by less than 2^4."""
    c = TreeCase(hq, hkv, d, [600, 37], [nodes, nodes - 1], nodes, cache, page, seed=nodes)
    t, bufs = run_step(m, c, torch.float32)
    assert int(bufs.err.item()) == 0
    p_err = 2.0 ** -15 if cache != "e5m2" or d == 64 else 2.0 ** -11 + 2.0 ** -11
    check_attention(c, t, bufs.q_rot, bufs.out, bufs.lse, p_err=p_err)
