"""GPU: the tree calls at the limits of what they are given: sequences that are
refused, waits that ran out before, scores that span many powers of two, values
that are no numbers."""

import pytest
import torch

from test_tree_gpu import m  # noqa: F401 (fixture)
from tree_cases import TreeCase

pytestmark = pytest.mark.gpu


def same_bits(a, b):
    return a is None or torch.equal(a.view(torch.uint8), b.view(torch.uint8))


# ------------------------------------------------------------------ append

@pytest.mark.parametrize("cache", ["bf16", "e5m2", "u8"])
@pytest.mark.parametrize("B", [4, 20])  # 64 nodes and 320: a bf16 cache takes another kernel from 256 on
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [0, 16])
@pytest.mark.parametrize("whole_step", [False, True])
def test_a_negative_position_appends_nothing(m, cache, B, d, page, whole_step):  # noqa: F811
    """Nodes that would land in rows 0, 1, .. of a sequence at a negative position
    are not written: the caches and q_rot are those of a call in which that
    sequence drafts nothing."""
    n, bad = 16, 3
    c = TreeCase(8, 2, d, [20] * B, [n] * B, n, cache, page, seed=d + B)
    got = []
    for pos, nodes in ((20, 0), (-1, n), (-n, n), (-n - 1, n), (-2 ** 31, n), (-1, 0)):
        lay, t = c.gpu(m)
        t.pos[bad], t.num[bad] = pos, nodes
        bufs = m.TreeBuffers.allocate(lay, n)
        bufs.q_rot.fill_(3.0)
        if whole_step:
            m.tree_step(lay, n, t.q_new, t.k_new, t.v_new, t.pos, t.depth, t.mask, c.max_len, bufs, num_nodes=t.num)
        else:
            m.kv_append_rope_tree(lay, n, t.q_new, t.k_new, t.v_new, t.pos, t.depth, 10000.0, bufs.q_rot, bufs.err, t.num)
        torch.cuda.synchronize()
        want = (m.MQA_DEVERR_POS_RANGE if pos < 0 and nodes else 0) | (m.MQA_DEVERR_SEQ_LEN if pos < 0 and whole_step else 0)
        assert int(bufs.err.item()) == want
        got.append((t.k, t.v, t.ksz, t.vsz, bufs.q_rot))
    assert (got[0][4][bad] == 3.0).all()
    for other in got[1:]:
        assert all(same_bits(a, b) for a, b in zip(got[0], other))
