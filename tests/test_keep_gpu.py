"""GPU: keeping an accepted path against oracle/tree.py (bytes, so equal), and
a whole round of speculation: step, verification, path, next step."""


import numpy as np
import pytest
import torch

import oracle
from tree_cases import TreeCase, deal_pages, raw

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m(built_lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import mqa_decode_attention_gb300 as mod

    mod.library()
    return mod


DT = {"bf16": torch.bfloat16, "f32": torch.float32, "u8": torch.uint8, "e5m2": torch.float8_e5m2}


def caches(rng, cache, shape):
    if cache in ("u8", "e5m2"):
        x = torch.from_numpy(rng.integers(0, 256, shape, dtype=np.uint8))
        x = x.view(torch.float8_e5m2) if cache == "e5m2" else x
    else:
        x = torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(DT[cache])
    sz = torch.from_numpy(rng.standard_normal(shape[:-1] + (2,)).astype(np.float32)) if cache == "u8" else None
    return x, sz


def bits(x):
    return x.cpu().view(torch.uint8).numpy() if x.element_size() > 1 else x.cpu().view(torch.uint8).numpy()


@pytest.mark.parametrize("cache", list(DT))
@pytest.mark.parametrize("page", [0, 16, 128])
@pytest.mark.parametrize("B,hkv,d,n,layers", [(1, 1, 64, 1, 1), (3, 2, 128, 16, 2), (2, 3, 64, 128, 3), (4, 8, 128, 40, 70)])
def test_matches_oracle(m, B, hkv, d, n, layers, page, cache):
    rng = np.random.default_rng(n + page)
    pos = rng.integers(0, 60, B)
    kept = rng.integers(0, n + 1, B)
    kept[0] = n if n < 20 else n - 7
    path = np.full((B, n), -5, np.int32)  # (entries past num_kept are not read)
    for b in range(B):
        path[b, :kept[b]] = np.sort(rng.choice(n, kept[b], replace=False))
    if B > 2:
        path[2, :kept[2]] = np.arange(kept[2])  # already in place
    if page:
        table, total = deal_pages(rng, [-(-(int(p) + n) // page) for p in pos], 1)
        shape = (total, hkv, page, d)
    else:
        table, shape = None, (B, hkv, 60 + n + n % 2, d)
    host, dev, lays = [], [], []
    t = None if table is None else torch.from_numpy(table).cuda()
    for _ in range(layers):
        (k, ks), (v, vs) = caches(rng, cache, shape), caches(rng, cache, shape)
        host.append((k, ks, v, vs))
        g = [None if x is None else x.clone().cuda() for x in (k, ks, v, vs)]
        dev.append(g)
        lays.append(m.layout_paged(g[0], g[2], t, hkv, 0, g[1], g[3]) if page else
                    m.layout_contiguous(g[0], g[2], hkv, 0, g[1], g[3]))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")  # noqa: E731
    m.keep_path(m.layout_stack(lays), i32(pos), i32(path), i32(kept), err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    for h, g in zip(host, dev):
        for x, y in zip(h, g):
            if x is not None:
                assert np.array_equal(oracle.keep_path(bits(x), pos, path, kept, table, page), bits(y))


def test_bad_paths_move_nothing(m):
    rng = np.random.default_rng(0)
    k, _ = caches(rng, "bf16", (6, 2, 40, 64))
    g, v = k.clone().cuda(), k.clone().cuda()
    lay = m.layout_contiguous(g, v, 2)
    path = np.array([[0, 2, 5], [2, 1, 3], [0, 3, 3], [0, 2, 8], [-1, 1, 2], [1, 2, 4]], np.int32)
    path = np.pad(path, ((0, 0), (0, 5)), constant_values=-1)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")  # noqa: E731
    pos = [3, 4, 5, 6, 7, 8]
    m.keep_path(lay, i32(pos), i32(path), i32([3] * 6), err)
    assert int(err.item()) == m.MQA_DEVERR_TREE
    want = oracle.keep_path(raw(k), pos, path, [3, 0, 0, 0, 0, 3])
    assert np.array_equal(raw(g), want) and np.array_equal(raw(v), want)
    err.zero_()
    m.keep_path(lay, i32([38, -1, 0, 0, 0, 0]), i32(path), i32([3, 1, 0, 0, 9, -1]), err)
    assert int(err.item()) == m.MQA_DEVERR_TREE | m.MQA_DEVERR_POS_RANGE
    assert np.array_equal(raw(g), want)


@pytest.mark.parametrize("n", [3, 8])
def test_bad_page(m, n):
    """With three nodes, node 4 does not exist; with eight, the second page of the first sequence does not."""
    rng = np.random.default_rng(0)
    k, _ = caches(rng, "bf16", (5, 1, 16, 64))
    g, v = k.clone().cuda(), k.clone().cuda()
    table = np.array([[0, 9], [2, 3]], np.int32)
    lay = m.layout_paged(g, v, torch.from_numpy(table).cuda(), 1)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")  # noqa: E731
    path = [[0, 2, 4] + [-1] * (n - 3)] * 2
    m.keep_path(lay, i32([13, 13]), i32(path), i32([3, 3]), err)
    assert int(err.item()) == (m.MQA_DEVERR_TREE if n == 3 else m.MQA_DEVERR_PAGE_RANGE)
    want = oracle.keep_path(raw(k), [13, 13], path, [0, 0 if n == 3 else 3], table, 16)
    assert np.array_equal(raw(g), want) and np.array_equal(raw(v), want)


@pytest.mark.parametrize("cache", ["bf16", "u8", "e5m2"])
@pytest.mark.parametrize("page", [0, 16])
def test_rounds_of_speculation(m, cache, page):
    """Three rounds as a serving loop runs them, on one graph: the caches and
    the tokens they leave are those of appending the kept tokens one by one."""
    layers, B, hq, hkv, d, n, vocab, rounds = 2, 3, 8, 2, 128, 10, 200, 3
    rng = np.random.default_rng(7)
    g = torch.Generator(device="cuda").manual_seed(1)
    room = 40 + rounds * n
    start = [17, 40, 0]
    if page:
        table, total = deal_pages(rng, [-(-room // page)] * B, 1)
        shape, t = (total, hkv, page, d), torch.from_numpy(table).cuda()
    else:
        shape, t, table = (B, hkv, room, d), None, None
    base = [[*caches(rng, cache, shape), *caches(rng, cache, shape)] for _ in range(layers)]

    def fresh():
        made = []
        for k, ks, v, vs in base:
            x = [None if y is None else y.clone().cuda() for y in (k, ks, v, vs)]
            made.append((x, m.layout_paged(x[0], x[2], t, hq, 0, x[1], x[3]) if page else
                         m.layout_contiguous(x[0], x[2], hq, 0, x[1], x[3])))
        return made

    spec, plain = fresh(), fresh()
    stack = m.layout_stack([lay for _, lay in spec])
    parents = torch.tensor([[-1, 0, 0, 1, 1, 2, 3, 3, 5, 8]] * B, dtype=torch.int32, device="cuda")
    mask, depth = m.tree_mask(parents)
    pos = torch.tensor(start, dtype=torch.int32, device="cuda")
    bufs = [m.TreeBuffers.allocate(lay, n) for _, lay in spec]
    ver = m.VerifyBuffers.allocate(B, n)
    ins = [[torch.empty(B, n, h, d, dtype=torch.bfloat16, device="cuda") for h in (hq, hkv, hkv)] for _ in range(layers)]
    p, q = (torch.empty(B, n, vocab, device="cuda") for _ in "pq")
    tok, u, un = torch.empty(B, n, dtype=torch.int32, device="cuda"), torch.empty(B, n, device="cuda"), torch.empty(B, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def one_round():
        for (x, lay), bf, (qn, kn, vn) in zip(spec, bufs, ins):
            m.tree_step(lay, n, qn, kn, vn, pos, depth, mask, room, bf)
        m.verify_tree(p, q, tok, parents, u, un, ver)
        m.keep_path(stack, pos, ver.path, ver.num_kept, err)
        pos.add_(ver.num_kept)

    def draw():
        for group in ins:
            for x in group:
                x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
        logits = torch.randn(B, n, vocab, generator=g, device="cuda")
        p.copy_(torch.softmax(logits * 2, -1))
        q.copy_(torch.softmax(logits * 2 + 0.5 * torch.randn(B, n, vocab, generator=g, device="cuda"), -1))
        tok.copy_(torch.randint(0, vocab, (B, n), generator=g, device="cuda"))
        tok.copy_(torch.where(torch.rand(B, n, generator=g, device="cuda") < 0.8,
                              q.argmax(-1).gather(1, parents.clamp(min=0).long()).int(), tok))
        u.copy_(torch.rand(B, n, generator=g, device="cuda"))
        un.copy_(torch.rand(B, generator=g, device="cuda"))

    draw()
    keep = [x.clone() for x, in zip([pos])][0]
    one_round()  # warm
    torch.cuda.synchronize()
    for (x, _), (k, ks, v, vs) in zip(spec, base):
        for y, z in zip(x, (k, ks, v, vs)):
            if y is not None:
                y.copy_(z)
    pos.copy_(keep)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        one_round()
    at, moved = list(start), 0
    for _ in range(rounds):
        draw()
        graph.replay()
        torch.cuda.synchronize()
        kept, path = ver.num_kept.tolist(), ver.path.tolist()
        moved += sum(path[b][i] != i for b in range(B) for i in range(kept[b]))
        for (x, lay), (qn, kn, vn) in zip(plain, ins):  # the kept tokens one at a time, at their positions
            sink = torch.empty(B, hq, d, device="cuda")
            for i in range(max(kept)):
                for b in range(B):
                    if i >= kept[b]:
                        continue
                    # (one sequence at a time: the others append out of range and are left alone)
                    where = torch.full((B,), -1, dtype=torch.int32, device="cuda")
                    where[b] = at[b] + i
                    e = torch.zeros(1, dtype=torch.int32, device="cuda")
                    node = path[b][i]
                    m.kv_append_rope(lay, qn[:, node].contiguous(), kn[:, node].contiguous(), vn[:, node].contiguous(), where,
                                     10000.0, sink, e)
        at = [a + k for a, k in zip(at, kept)]
        assert pos.tolist() == at
        for b in range(B):
            for (x, _), (y, _) in zip(spec, plain):
                for a, c in zip(x, y):
                    if a is None:
                        continue
                    a, c = bits(a), bits(c)
                    if page:
                        for tk in range(at[b]):
                            pg = table[b, tk // page]
                            assert np.array_equal(a[pg, :, tk % page], c[pg, :, tk % page])
                    else:
                        assert np.array_equal(a[b, :, :at[b]], c[b, :, :at[b]])
    assert moved > 0 and int(err.item()) == 0 and int(ver.err.item()) == 0 and all(int(x.err.item()) == 0 for x in bufs)
    if cache != "e5m2":  # (8 of the 256 codes the e5m2 caches are drawn from are infinities and NaN)
        assert all(torch.isfinite(x.out).all() for x in bufs)
