"""GPU: verification where little or nothing is left of the target's distribution."""

import numpy as np
import pytest
import torch

import oracle
from test_verify_gpu import m  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu


def run(m, p, tokens, u, un):  # noqa: F811
    """Node 0 with all the others as its children, no draft probabilities."""
    B, n, _ = p.shape
    parents = np.array([[-1] + [0] * (n - 1)] * B, np.int32)
    want = oracle.verify_tree(p.double().numpy(), None, tokens, parents, [n] * B, u, un)[:3]
    bufs = m.VerifyBuffers.allocate(B, n)
    dev = lambda x, t: torch.as_tensor(np.asarray(x), dtype=t).cuda()  # noqa: E731
    m.verify_tree(p.cuda(), None, dev(tokens, torch.int32), dev(parents, torch.int32), dev(u, torch.float32),
                  dev(un, torch.float32), bufs)
    torch.cuda.synchronize()
    assert int(bufs.err.item()) == 0
    got = bufs.num_kept.cpu().numpy(), bufs.path.cpu().numpy(), bufs.next_token.cpu().numpy()
    return want, got


def equal(want, got):
    for a, b in zip(want, got):
        assert np.array_equal(a, b), (a, b)


def test_every_token_rejected_nothing_left(m):  # noqa: F811
    """Four tokens that hold all of p, all rejected: nothing is left, so the most
    probable one is taken. (Their sum as a pair of floats is not exact; taken off
    it again in this order they leave 2^-73.)"""
    p = torch.zeros(1, 5, 300)
    p[0, 0, 4:8] = torch.tensor([float.fromhex(x) for x in ("0x1.2acd58p-21", "0x1.79b9c6p-40", "0x1.e84f16p-52", "0x1.9cc3c4p-53")])
    tokens = [[0, 5, 6, 4, 7]]
    want, got = run(m, p, tokens, [[0.0, 0.9, 0.9, 0.9, 0.9]], [0.5])
    assert want[0][0] == 1 and want[2][0] == 4
    equal(want, got)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab,spread", [(33, 1), (4099, 1), (4099, 100), (50001, 1500)])
@pytest.mark.parametrize("left", [0.0, 2.0 ** -60, 2.0 ** -30])
def test_many_tokens_rejected(m, dtype, vocab, spread, left):  # noqa: F811
    """32 tokens that hold 0.9, all rejected (each weighs less than 0.95 of what is
    left of 1); beside them either nothing, or one token that weighs far less than
    their sum's rounding and is the only one left (vocab 33: in half of the
    sequences it is one of the rejected)."""
    rng = np.random.default_rng(vocab + spread)
    B, n = 64, 33
    p = torch.zeros(B, n, vocab)
    tokens = np.zeros((B, n), np.int64)
    for b in range(B):
        w = rng.random(32) ** 3
        at = 1 + spread * np.arange(32)
        p[b, 0, at] = torch.from_numpy((w / w.sum() * 0.9).astype(np.float32))
        p[b, 0, 0 if b % 2 else vocab - 1] += left
        tokens[b, 1:] = rng.permutation(at)
    p = p.to(dtype)
    un = rng.random(B).astype(np.float32)
    want, got = run(m, p, tokens, np.full((B, n), 0.95, np.float32), un)
    assert (want[0] == 1).all()
    equal(want, got)
