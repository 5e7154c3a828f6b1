"""GPU: verification of drafted trees against the fp64 walk of oracle/tree.py.

Every output is a whole number and has to be equal. The oracle's walk and the
kernel's sums are both good to about 2^-44 of a probability, so a decision
could differ only where it lies that close to a tie; the inputs' smallest
margin is asserted to be above 2^-36 (the oracle gives it), which leaves no
doubt about any of them.
"""

import numpy as np
import pytest
import torch

import oracle
from tree_cases import random_parents

pytestmark = pytest.mark.gpu
MARGIN = 2.0 ** -36


@pytest.fixture(scope="module")
def m(built_lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import mqa_decode_attention_gb300 as mod

    mod.library()
    return mod


class Case:
    def __init__(self, B, n, vocab, seed=0, branch=3, dtype=torch.float32, drafted=True, nodes=None, pad=0, spread=2.5, near=1.0):
        rng = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        logits = torch.randn(B, n, vocab, generator=g) * spread
        p = torch.softmax(logits, -1)
        q = torch.softmax(logits + near * torch.randn(B, n, vocab, generator=g), -1)
        self.parents = np.array([random_parents(rng, n, branch) for _ in range(B)], np.int32)
        above = torch.from_numpy(np.maximum(self.parents, 0)).long()
        drawn = torch.gather(q, 1, above[..., None].expand(-1, -1, vocab))
        race = torch.rand(B, n, vocab, generator=g).clamp(min=1e-9).log().neg()
        self.tokens = (drawn / race).argmax(-1).int()
        self.nodes = [n] * B if nodes is None else list(nodes)
        self.u, self.un = torch.rand(B, n, generator=g), torch.rand(B, generator=g)
        wide = vocab + pad

        def rows(x):
            y = torch.full((B, n, wide), float("nan"), dtype=dtype)
            y[..., :vocab] = x.to(dtype)
            return y[..., :vocab]

        self.p, self.q = rows(p), rows(q) if drafted else None
        self.n, self.B = n, B

    def oracle(self):
        f = lambda x: None if x is None else x.double().numpy()  # noqa: E731
        *r, margin = oracle.verify_tree(f(self.p), f(self.q), self.tokens.numpy(), self.parents, self.nodes, self.u.numpy(),
                                        self.un.numpy())
        assert margin > MARGIN
        return r

    def run(self, m):
        cuda = lambda x: None if x is None else torch.as_tensor(x).cuda()  # noqa: E731

        def wide(x):  # keeps the padding
            if x is None:
                return None
            y = torch.empty(x.shape[0], x.shape[1], x.stride(1), dtype=x.dtype, device="cuda").fill_(float("nan"))
            y[..., :x.shape[2]] = x.cuda()
            return y[..., :x.shape[2]]

        bufs = m.VerifyBuffers.allocate(self.B, self.n)
        for t in (bufs.num_kept, bufs.path, bufs.next_token):
            t.fill_(-77)
        m.verify_tree(wide(self.p), wide(self.q), cuda(self.tokens), cuda(self.parents), cuda(self.u), cuda(self.un), bufs,
                      num_nodes=torch.tensor(self.nodes, dtype=torch.int32, device="cuda"))
        torch.cuda.synchronize()
        return bufs

    def check(self, m):
        kept, path, nxt = self.oracle()
        b = self.run(m)
        assert int(b.err.item()) == 0
        assert np.array_equal(b.num_kept.cpu().numpy(), kept)
        assert np.array_equal(b.path.cpu().numpy(), path)
        assert np.array_equal(b.next_token.cpu().numpy(), nxt)
        return kept


@pytest.mark.parametrize("drafted", [True, False])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,n,vocab,branch", [(1, 1, 1, 1), (2, 2, 3, 1), (3, 9, 33, 2), (4, 16, 1000, 3), (2, 40, 4099, 4),
                                              (5, 128, 257, 3), (2, 8, 32000, 2), (3, 8, 50001, 3)])
def test_matches_oracle(m, B, n, vocab, branch, dtype, drafted):
    Case(B, n, vocab, 11 + n, branch, dtype, drafted).check(m)


@pytest.mark.parametrize("pad", [1, 2, 3, 5, 7, 8])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_padded_and_misaligned_rows(m, pad, dtype):
    Case(3, 12, 9001, 5 + pad, 3, dtype, pad=pad).check(m)


def test_ragged_and_empty_trees(m):
    Case(6, 20, 501, 3, nodes=[20, 0, 1, 7, 13, 0]).check(m)


def test_whole_batches(m):
    """As many sequences as leave one, two, four blocks to each; every depth is reached."""
    for B, vocab in ((40, 20001), (160, 9000), (330, 9000), (700, 300)):
        kept = Case(B, 6, vocab, B, 2, near=0.3).check(m)
        assert kept.max() > 2 and kept.min() < 3


def test_draft_equals_target(m):
    """p = q: every first child stands (u < 1), nothing is ever rejected."""
    c = Case(4, 10, 5000, 2, branch=1)
    c.q = c.p.clone()
    kept = c.check(m)
    assert (kept == 10).all()


def test_greedy(m):
    """One-hot probabilities: the walk follows the target's own tokens and ends with the next of them."""
    c = Case(3, 8, 700, 4, branch=1)
    best = c.p.argmax(-1)
    c.p = torch.zeros_like(c.p).scatter_(2, best[..., None], 1.0)
    c.q = None
    c.tokens = torch.cat([torch.zeros(3, 1, dtype=torch.int64), best[:, :-1]], 1).int()
    c.tokens[1, 4] = (c.tokens[1, 4] + 1) % 700
    b = c.run(m)
    assert b.num_kept.tolist() == [8, 4, 8]
    assert b.next_token.tolist() == [int(best[0, 7]), int(best[1, 3]), int(best[2, 7])]


def test_same_token_twice(m):
    """Two children with one token: the second has nothing left (deterministic) or its residual (drawn)."""
    for drafted in (True, False):
        c = Case(4, 5, 64, 6, drafted=drafted)
        c.parents = np.array([[-1, 0, 0, 0, 0]] * 4, np.int32)
        c.tokens[:, 1:] = torch.tensor([3, 3, 9, 9], dtype=torch.int32)
        c.u[:, 1] = c.u[:, 3] = 0.999
        c.check(m)


def test_nothing_left(m):
    """p <= q where it matters: the residual is zero everywhere, the most probable token (lowest of equals) is taken."""
    c = Case(2, 2, 300, 1)
    c.parents = np.array([[-1, 0]] * 2, np.int32)
    c.p[:] = 0.0
    c.p[..., 7] = c.p[..., 250] = 0.25
    c.q[:] = 0.5
    c.tokens[:, 1] = 5
    b = c.run(m)
    assert b.num_kept.tolist() == [1, 1] and b.next_token.tolist() == [7, 7]


def test_nan_probabilities_weigh_nothing(m):
    c = Case(2, 6, 900, 8)
    c.p[..., 100:200] = float("nan")
    clean = Case(2, 6, 900, 8)
    clean.p[..., 100:200] = 0.0
    a, b = c.run(m), clean.run(m)
    for x, y in ((a.path, b.path), (a.next_token, b.next_token), (a.num_kept, b.num_kept)):
        assert torch.equal(x, y)


def test_extreme_random_numbers(m):
    for u in (0.0, 1.0 - 2.0 ** -24):
        c = Case(3, 6, 5001, 9, 2)
        c.u[:] = u
        c.un[:] = u
        f = lambda x: x.double().numpy()  # noqa: E731
        kept, path, nxt, _ = oracle.verify_tree(f(c.p), f(c.q), c.tokens.numpy(), c.parents, c.nodes, c.u.numpy(), c.un.numpy())
        b = c.run(m)
        assert b.num_kept.tolist() == kept.tolist() and b.path.tolist() == path.tolist()
        assert b.next_token.tolist() == nxt.tolist()


def test_bad_nodes_are_reported_and_never_tried(m):
    c = Case(3, 8, 400, 3, 2)
    kept, path, nxt = c.oracle()
    bad = Case(3, 8, 400, 3, 2)
    bad.tokens[1, 5], bad.tokens[1, 6] = 400, -1
    bad.parents[2, 4], bad.parents[2, 7] = 4, 99
    b = bad.run(m)
    assert int(b.err.item()) == m.MQA_DEVERR_TREE
    assert b.num_kept[0].item() == kept[0] and b.next_token[0].item() == nxt[0]
    assert not {5, 6} & set(b.path[1].tolist()) and not {4, 7} & set(b.path[2].tolist())
    bad.nodes = [8, 9, -1]
    b = bad.run(m)
    assert int(b.err.item()) & m.MQA_DEVERR_SEQ_LEN
    assert b.num_kept.tolist()[1:] == [0, 0] and b.next_token.tolist()[1:] == [-1, -1] and (b.path[1:] == -1).all()


def test_graph_replay(m):
    c = Case(4, 16, 20000, 7)
    want = c.run(m)
    cuda = [torch.as_tensor(x).cuda() for x in (c.p.contiguous(), c.q.contiguous(), c.tokens, c.parents, c.u, c.un)]
    bufs = m.VerifyBuffers.allocate(4, 16)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        m.verify_tree(*cuda, bufs)
    for _ in range(2):
        bufs.path.fill_(5)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(bufs.path, want.path) and torch.equal(bufs.next_token, want.next_token)
