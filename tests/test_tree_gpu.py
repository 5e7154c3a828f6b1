"""GPU: the tree step against the fp64 oracle (oracle/tree.py).

The append is held to the oracle's bytes (V and codes exactly, bf16 K within
one step of the fp64 rotation, q_rot within half a step of it). The attention
is then held to the oracle's on the operands it was given -- its own bf16 q_rot
and the cache rows as they stand -- by the bound its roundings allow, element
by element, with e = 2^-8 (half a bf16 step, relative):
  * P rounded to bf16 (times a V scale, for uint8): e sum w |v|;
  * a score is a sum of d products in fp32 and a scaling: its error is at most
    (d + 2) 2^-24 scale sum |q k| <= (d + 2) 2^-24 reach, which moves every weight
    by that relative amount, once in the sum above the line and once below;
    the exponent's argument scale log2 e (s - m), |.| <= 2 reach, is rounded at
    2^-24 of it, and ex2 is within 2^-22 of its value: 4 more units of reach
    2^-24 and of 2^-22 cover both lines;
  * fp32 accumulation over the keys and the merge of partial results: tiles are
    added one after the other, T keys give at most (T / 64 + 2 * 64) 2^-24 sum w |v|
    beside the exact sum; T <= 8192 here, so 2^-15 sum w |v|;
  * the output rounded to bf16: e |out| (fp32: 2^-24).
lse: the score's error and 2^-20 of max(1, |lse|) for the fp32 logarithm and sums.
"""

import math

import numpy as np
import pytest
import torch

import oracle
from tree_cases import TreeCase, raw

pytestmark = pytest.mark.gpu
E = 2.0 ** -8


@pytest.fixture(scope="module")
def m(built_lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import mqa_decode_attention_gb300 as mod

    mod.library()
    return mod


def run_step(m, c, out_dtype=torch.bfloat16):
    lay, t = c.gpu(m)
    bufs = m.TreeBuffers.allocate(lay, c.n, c.max_len, out_dtype=out_dtype, lse=True)
    bufs.out.fill_(7.0)
    bufs.lse.fill_(7.0)
    bufs.workspace.fill_(255)  # (it need not be cleared)
    m.tree_step(lay, c.n, t.q_new, t.k_new, t.v_new, t.pos, t.depth, t.mask, c.max_len, bufs, num_nodes=t.num)
    torch.cuda.synchronize()
    return t, bufs


def live(c):
    return np.arange(c.n) < np.array(c.nodes)[:, None]


def check_append(c, t, q_rot):
    rows = live(c)
    want = oracle.tree_rotate(c.q_new, c.pos, c.depth, 10000.0)[rows]
    got = raw(q_rot)[rows]
    step = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(want), 2.0 ** -100))) - 7)
    assert np.all(np.abs(got - want) <= 0.5 * step + 1e-6 * np.abs(want).max(initial=1.0))
    k, v, ksz, vsz = oracle.tree_append(raw(c.k), raw(c.v), c.cache, c.k_new, c.v_new, c.pos, c.depth, c.nodes, 10000.0,
                                        c.table, c.page, None if c.ksz is None else raw(c.ksz),
                                        None if c.vsz is None else raw(c.vsz))
    assert np.array_equal(raw(t.v), v, equal_nan=c.cache == "bf16")
    gk = raw(t.k)
    if c.cache == "bf16":
        assert np.array_equal(np.isnan(gk), np.isnan(k))
        fine = ~np.isnan(k)
        step = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(k[fine]), 2.0 ** -100))) - 7)
        assert np.all(np.abs(gk[fine] - k[fine]) <= step)
        assert np.mean(gk[fine] != k[fine]) < 1e-3
    else:  # a value next to a rounding border may take the other code: none here, from the fp64 rotation
        assert np.array_equal(gk, k)
    if c.cache == "u8":
        assert np.array_equal(raw(t.ksz), ksz, equal_nan=True) and np.array_equal(raw(t.vsz), vsz, equal_nan=True)


def check_attention(c, t, q_rot, out, lse, p_err=E):
    scale = 1 / math.sqrt(c.d)
    tokens = c.max_len
    keys = oracle.logical(c.cache, raw(t.k), None if t.ksz is None else raw(t.ksz), c.table, c.page, tokens)
    vals = oracle.logical(c.cache, raw(t.v), None if t.vsz is None else raw(t.vsz), c.table, c.page, tokens)
    ref = oracle.tree_attention(raw(q_rot), keys, vals, c.pos, c.depth, c.nodes, c.bits, scale, c.window)
    rows = live(c)
    got, glse = out.detach().cpu().double().numpy(), None if lse is None else raw(lse)
    assert np.all(got[~rows] == 7.0)  # padding rows are left as they were
    assert glse is None or np.all(glse[~rows] == 7.0)
    want, size, reach = ref["out"][rows], ref["size"][rows], ref["reach"][rows][..., None]
    score = (c.d + 6) * 2.0 ** -24 * reach
    bound = p_err * size + (2 * (score + 2.0 ** -20) + 2.0 ** -15) * size
    bound = bound + (E if out.dtype == torch.bfloat16 else 2.0 ** -24) * (np.abs(want) + bound) + 1e-30
    err = np.abs(got[rows] - want)
    assert np.isfinite(got[rows]).all()
    assert np.all(err <= bound), f"{np.max(err / bound)} of the bound"
    if glse is not None:
        gl, wl = glse[rows], ref["lse"][rows]
        empty = np.isneginf(wl)
        assert np.array_equal(np.isneginf(gl), empty)
        assert np.all(np.abs(gl[~empty] - wl[~empty]) <= score[..., 0][~empty] + 2.0 ** -20 * np.maximum(1, np.abs(wl[~empty])))


def check(m, c, out_dtype=torch.bfloat16):
    t, bufs = run_step(m, c, out_dtype)
    assert int(bufs.err.item()) == 0
    check_append(c, t, bufs.q_rot)
    check_attention(c, t, bufs.q_rot, bufs.out, bufs.lse)
    return t, bufs


# hq, hkv, d, pos, nodes, n
SHAPES = {
    "one token, one node": (8, 2, 128, [1], [1], 1),
    "empty cache": (8, 2, 128, [0, 0], [5, 1], 5),
    "group 1": (4, 4, 128, [130, 63], [7, 7], 7),
    "group 4": (32, 8, 128, [300, 257], [16, 9], 16),
    "group 7, odd": (14, 2, 128, [191, 64, 1], [13, 0, 11], 13),
    "rows past 128": (16, 2, 128, [500, 129], [33, 20], 33),
    "mqa 32": (32, 1, 128, [640, 200], [8, 6], 8),
    "128 nodes": (8, 2, 128, [100, 700], [128, 97], 128),
    "group 48": (96, 2, 128, [70], [5], 5),
    "group 80": (160, 2, 128, [70, 30], [3, 2], 3),
    "group 160": (160, 1, 128, [129], [2], 2),
    "d 64": (12, 3, 64, [200, 33, 64], [10, 31, 31], 31),
    "d 64 mqa": (16, 1, 64, [129, 500], [9, 64], 64),
    "long": (8, 1, 128, [4000, 17], [6, 3], 6),
}


@pytest.mark.parametrize("cache", ["bf16", "e5m2", "u8"])
@pytest.mark.parametrize("page", [0, 16, 64, 256])
@pytest.mark.parametrize("shape", list(SHAPES))
def test_step_matches_oracle(m, shape, page, cache):
    hq, hkv, d, pos, nodes, n = SHAPES[shape]
    check(m, TreeCase(hq, hkv, d, pos, nodes, n, cache, page, seed=len(shape) + page))


@pytest.mark.parametrize("cache", ["bf16", "e5m2", "u8"])
@pytest.mark.parametrize("window", [1, 3, 64, 100, 5000])
@pytest.mark.parametrize("page", [0, 32])
def test_window(m, cache, window, page):
    for d, hq, hkv in ((128, 32, 8), (64, 6, 2)):
        check(m, TreeCase(hq, hkv, d, [333, 2, 64, 0], [20, 20, 11, 4], 20, cache, page, window, seed=window))


@pytest.mark.parametrize("cache", ["bf16", "e5m2", "u8"])
@pytest.mark.parametrize("mask", ["random", "none"])
@pytest.mark.parametrize("pos", [0, 150])
def test_masks_that_are_no_tree(m, cache, mask, pos):
    """Any relation among the nodes; rows that see nothing at all give 0 and -inf."""
    for d, n in ((128, 40), (64, 11), (128, 128)):
        check(m, TreeCase(8, 2, d, [pos, pos], [n, n - 3], n, cache, 0, 0, mask, seed=n))


@pytest.mark.parametrize("page", [0, 16])
def test_fp32_output(m, page):
    check(m, TreeCase(16, 4, 128, [300, 40], [12, 12], 12, page=page), torch.float32)
    check(m, TreeCase(16, 4, 64, [300, 40], [12, 12], 12, page=page), torch.float32)


@pytest.mark.parametrize("cache", ["bf16", "u8"])
def test_many_sequences_of_many_lengths(m, cache):
    """More sequences than lanes, some without nodes: runs that span many units and units that span many runs."""
    rng = np.random.default_rng(3)
    pos = [int(x) for x in rng.integers(0, 400, 70)]
    pos[5], pos[69] = 6000, 3000
    nodes = [int(x) for x in rng.integers(0, 10, 70)]
    nodes[5], nodes[69] = 9, 9
    check(m, TreeCase(4, 1, 128, pos, nodes, 9, cache, 16, seed=1))


@pytest.mark.parametrize("page", [0, 16])
def test_units_of_one_and_of_two_row_tiles(m, page):
    """Trees below and above 128 rows per kv head beside one another, in runs of several units."""
    rng = np.random.default_rng(6)
    pos = [int(x) for x in rng.integers(0, 900, 60)]
    nodes = [int(x) for x in rng.integers(0, 33, 60)]
    check(m, TreeCase(16, 2, 128, pos, nodes, 32, "bf16", page, seed=2))


def test_calls_are_the_step(m):
    """The two calls give the step's bits; so does a second run, on the workspace as the first left it."""
    for d, cache in ((128, "bf16"), (128, "u8"), (64, "e5m2")):
        c = TreeCase(32, 8, d, [700, 257, 1500], [16, 9, 12], 16, cache)
        t, a = run_step(m, c)
        lay, u = c.gpu(m)
        b = m.TreeBuffers.allocate(lay, c.n, lse=True)
        for _ in range(2):
            b.out.fill_(7.0)
            b.lse.fill_(7.0)
            m.kv_append_rope_tree(lay, c.n, u.q_new, u.k_new, u.v_new, u.pos, u.depth, 10000.0, b.q_rot, b.err, u.num)
            m.gqa_tree_attention(lay, c.n, b.q_rot, u.pos, u.depth, u.mask, c.max_len, 1 / math.sqrt(d), b.out, u.num, b.lse,
                                 b.workspace, b.err)
            torch.cuda.synchronize()
            assert torch.equal(a.out, b.out) and torch.equal(a.lse, b.lse)
        assert int(b.err.item()) == 0


def test_num_nodes_none_is_all(m):
    c = TreeCase(32, 8, 128, [300, 257], [10, 10], 10)
    t, a = run_step(m, c)
    lay, u = c.gpu(m)
    b = m.TreeBuffers.allocate(lay, c.n)
    m.tree_step(lay, c.n, u.q_new, u.k_new, u.v_new, u.pos, u.depth, u.mask, c.max_len, b)
    assert torch.equal(a.out, b.out)


def test_chain_is_the_multi_token_step(m):
    """A chain of nodes is what the multi-token step computes, up to the bf16
    rounding of its operands (both within the multi-token tests' 2e-2 of fp64)."""
    from synthetic import make_contiguous_case, workload

    w = workload("gqa4k").with_(batch=2, h_q=32, h_kv=8, seed=5)
    n, lens = 6, [500, 131]
    kc = make_contiguous_case(w, "cuda", seq_lens=torch.tensor(lens, dtype=torch.int32), capacity=500)
    g = torch.Generator(device="cuda").manual_seed(4)
    q, k, v = (torch.randn(2, n, h, 128, generator=g, device="cuda").bfloat16() for h in (32, 8, 8))
    lens_d = torch.tensor(lens, dtype=torch.int32, device="cuda")
    pos = (lens_d - n).int()
    ka, va = kc.k_cache.clone(), kc.v_cache.clone()
    lay = m.layout_contiguous(ka, va, 32)
    bufs = m.DecodeBuffers.allocate(lay, 500, n_new=n)
    m.decode_step_multi(lay, n, q, k, v, pos, lens_d, 500, bufs)
    parents = torch.arange(-1, n - 1, dtype=torch.int32, device="cuda").expand(2, n).contiguous()
    mask, depth = m.tree_mask(parents)
    kb, vb = kc.k_cache.clone(), kc.v_cache.clone()
    lay2 = m.layout_contiguous(kb, vb, 32)
    tb = m.TreeBuffers.allocate(lay2, n)
    m.tree_step(lay2, n, q, k, v, pos, depth, mask, 500, tb)
    assert torch.equal(ka, kb) and torch.equal(va, vb)
    assert (tb.out.float() - bufs.out.float()).abs().max() <= 4e-2


def test_bad_sequences_are_reported_and_skipped(m):
    """A length past the bound, a negative position, too many nodes: the bit, and the others' results as they would be."""
    for cache in ("bf16", "u8"):
        good = TreeCase(8, 2, 128, [300, 257, 90, 10], [8, 0, 0, 5], 8, cache)
        t, a = run_step(m, good)
        lay, u = good.gpu(m)
        b = m.TreeBuffers.allocate(lay, 8, lse=True)
        b.out.fill_(7.0)
        b.lse.fill_(7.0)
        pos = torch.tensor([300, 303, -1, 10], dtype=torch.int32, device="cuda")
        num = torch.tensor([8, 8, 2, 5], dtype=torch.int32, device="cuda")  # 303 + 8 > 308 = max_len
        m.gqa_tree_attention(lay, 8, a.q_rot, pos, u.depth, u.mask, good.max_len, 1 / math.sqrt(128), b.out, num, b.lse,
                             b.workspace, b.err)
        assert int(b.err.item()) == m.MQA_DEVERR_SEQ_LEN
        assert (b.out[1] == 7).all() and (b.out[2] == 7).all()
        num[1] = 9
        m.gqa_tree_attention(lay, 8, a.q_rot, pos, u.depth, u.mask, good.max_len, 1 / math.sqrt(128), b.out, num, b.lse,
                             b.workspace, b.err)
        assert (b.out[1] == 7).all()


def test_append_errors(m):
    c = TreeCase(8, 2, 128, [20, 30], [4, 4], 4)
    lay, t = c.gpu(m)
    b = m.TreeBuffers.allocate(lay, 4)
    before = t.k.clone()
    bad = torch.tensor([5, -1], dtype=torch.int32, device="cuda")
    m.kv_append_rope_tree(lay, 4, t.q_new, t.k_new, t.v_new, t.pos, t.depth, 10000.0, b.q_rot, b.err, bad)
    assert int(b.err.item()) == m.MQA_DEVERR_SEQ_LEN
    assert torch.equal(before.nan_to_num(0), t.k.nan_to_num(0))
    b.err.zero_()
    depth = t.depth.clone()
    depth[0, 2], depth[1, 1] = 4, -1
    m.kv_append_rope_tree(lay, 4, t.q_new, t.k_new, t.v_new, t.pos, depth, 10000.0, b.q_rot, b.err)
    assert int(b.err.item()) == m.MQA_DEVERR_TREE
    b.err.zero_()
    far = torch.tensor([lay.capacity - 2, 30], dtype=torch.int32, device="cuda")
    m.kv_append_rope_tree(lay, 4, t.q_new, t.k_new, t.v_new, far, t.depth, 10000.0, b.q_rot, b.err)
    assert int(b.err.item()) == m.MQA_DEVERR_POS_RANGE


@pytest.mark.parametrize("cache,d", [("bf16", 128), ("u8", 128), ("bf16", 64)])
def test_bad_page_reads_as_zeros(m, cache, d):
    c = TreeCase(32, 8, d, [300, 70], [8, 6], 8, cache, page=16, seed=2)
    t, a = run_step(m, c)
    lay, u = c.gpu(m)
    for name in ("k", "v", "ksz", "vsz"):
        if getattr(u, name) is not None:
            getattr(u, name).copy_(getattr(t, name))  # the nodes' rows are there
    b = m.TreeBuffers.allocate(lay, 8, lse=True)
    b.out.fill_(7.0)
    b.lse.fill_(7.0)
    c.table[0, 3], c.table[0, 7] = -1, 10 ** 6
    u.table.copy_(torch.from_numpy(c.table))
    m.gqa_tree_attention(lay, 8, a.q_rot, u.pos, u.depth, u.mask, c.max_len, 1 / math.sqrt(d), b.out, u.num, b.lse,
                         b.workspace, b.err)
    assert int(b.err.item()) == m.MQA_DEVERR_PAGE_RANGE
    check_attention(c, u, a.q_rot, b.out, b.lse)


def test_graph_replay_and_other_stream(m):
    """Captured and replayed after the inputs changed in place; on a stream of its own; two graphs with a workspace each."""
    for cache, d in (("bf16", 128), ("e5m2", 64)):
        c = TreeCase(32, 8, d, [700, 257], [16, 9], 16, cache, garbage=False)
        t0, ref = run_step(m, c)
        runs = []
        stream = torch.cuda.Stream()
        for _ in range(2):
            lay, t = c.gpu(m)
            bufs = m.TreeBuffers.allocate(lay, c.n, lse=True)
            bufs.out.fill_(7.0)
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.stream(stream):
                m.tree_step(lay, c.n, t.q_new, t.k_new, t.v_new, t.pos, t.depth, t.mask, c.max_len, bufs, num_nodes=t.num)
                with torch.cuda.graph(graph, stream=stream):
                    m.tree_step(lay, c.n, t.q_new, t.k_new, t.v_new, t.pos, t.depth, t.mask, c.max_len, bufs,
                                num_nodes=t.num)
                    m.gqa_tree_attention(lay, c.n, bufs.q_rot, t.pos, t.depth, t.mask, c.max_len, 1 / math.sqrt(d),
                                         bufs.out, t.num, bufs.lse, bufs.workspace, bufs.err)
            runs.append((graph, bufs, lay, t))
        for graph, bufs, lay, t in runs:
            bufs.out.fill_(7.0)
        torch.cuda.synchronize()
        for graph, *_ in runs:
            graph.replay()
        torch.cuda.synchronize()
        for _, bufs, lay, t in runs:
            assert torch.equal(bufs.out, ref.out)
            assert int(bufs.err.item()) == 0


def test_scratch_of_another_call_is_not_kept(m):
    """A larger call's leavings in the same workspace change nothing."""
    big = TreeCase(32, 8, 128, [2000, 1900], [16, 16], 16, seed=8)
    small = TreeCase(32, 8, 128, [140], [3], 3, seed=9)
    t, a = run_step(m, small)
    lay, u = big.gpu(m)
    b = m.TreeBuffers.allocate(lay, 16)
    m.tree_step(lay, 16, u.q_new, u.k_new, u.v_new, u.pos, u.depth, u.mask, big.max_len, b)
    lay2, v = small.gpu(m)
    s = m.TreeBuffers.allocate(lay2, 3)
    s.workspace = b.workspace
    m.tree_step(lay2, 3, v.q_new, v.k_new, v.v_new, v.pos, v.depth, v.mask, small.max_len, s)
    assert torch.equal(s.out, a.out)
