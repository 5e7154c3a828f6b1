"""GPU: the tree calls at the limits of what they are given: sequences that are
refused, waits that ran out before, scores that span many powers of two, values
that are no numbers."""

import math

import pytest
import torch

from test_tree_gpu import check_attention, m, run_step  # noqa: F401 (m: fixture)
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


# --------------------------------------------------------------- e5m2, wide range

@pytest.mark.parametrize("hq,n", [(8, 1), (32, 5)])  # one row tile, two of them
@pytest.mark.parametrize("first,score", [(True, 17.5), (False, 17.5), (False, 5.5)])
def test_e5m2_light_keys_count(m, hq, n, first, score):  # noqa: F811
    """102400 cached e5m2 keys, 16 of them with a score, the others at 0; values 1
    there, 0 (dims 0 .. 63) or -2 (dims 64 ..) at the 16. The light keys weigh
    e^-17.5 = 2^-25.2 of the heavy ones each, 0.016% in all, which is all of the
    output's first half. (score 5.5, behind the others: below 2^8 of the running
    maximum that was, which stays: the largest P there is.)

    Bound, for weights w relative to the largest: P as an f16 times 2^7 is off by
    2^-11 w, or by 2^-25 2^-7 = 2^-32 where it is subnormal; fp32 sums over T keys by
    (T / 64 + 128) 2^-24 of sum w |v|, in l as in O; the scores (one product, a
    rounding of 2^-24 each in the product, its scaling and the exponent, of up to
    score log2 e < 32 = 2^5, and ex2 2^-22) by 3 * 2^-19 + 2^-22 above and below the
    line. Weights below that are lost to O would be off by all of the first half.

    The caches are one page of each kind, which all sequences share."""
    T, B, ps, d = 102400, 300, 16, 128
    kinds = dict(light=0, heavy=1, nodes=2)
    k = torch.zeros(3, 1, ps, d)
    v = torch.ones(3, 1, ps, d)
    k[kinds["heavy"], :, :, 0] = 1.0
    v[kinds["heavy"], :, :, :64], v[kinds["heavy"], :, :, 64:] = 0.0, -2.0
    k, v = (x.to(torch.float8_e5m2).cuda() for x in (k, v))
    table = torch.zeros(B, T // ps + 1, dtype=torch.int32)
    table[:, 0 if first else T // ps - 1] = kinds["heavy"]
    table[:, T // ps] = kinds["nodes"]
    lay = m.layout_paged(k, v, table.cuda(), hq)
    bufs = m.TreeBuffers.allocate(lay, n, out_dtype=torch.float32, lse=True)
    q = torch.zeros(B, n, hq, d, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = score
    pos = torch.full((B,), T, dtype=torch.int32, device="cuda")
    none = torch.zeros(B, n, 1, dtype=torch.int32, device="cuda")  # the nodes see the cached tokens only
    m.gqa_tree_attention(lay, n, q, pos, None, none, T + n, 1.0, bufs.out, None, bufs.lse, bufs.workspace, bufs.err)
    torch.cuda.synchronize()
    assert int(bufs.err.item()) == 0
    w, N = math.exp(-score), T - ps
    total = ps + w * N
    sums, scores = (T / 64 + 128) * 2.0 ** -24, 2 * (3 * 2.0 ** -19 + 2.0 ** -22)
    for half, value in ((slice(0, 64), 0.0), (slice(64, d), -2.0)):
        want, size = (w * N + ps * value) / total, (w * N + ps * abs(value)) / total
        p_err = (ps * abs(value) * 2.0 ** -11 + N * max(2.0 ** -11 * w, 2.0 ** -32)) / total
        bound = p_err + (2 * sums + scores) * size
        err = (bufs.out[..., half].double() - want).abs().max().item()
        assert err <= bound, (half, err, bound)
        assert value or bound < 0.1 * want  # (the light keys' part is seen)
    want = score + math.log(total)
    assert (bufs.lse.double() - want).abs().max().item() <= sums + scores + 2.0 ** -20 * want


# ---------------------------------------------------------- bounded waits

@pytest.mark.parametrize("cache", ["bf16", "e5m2", "u8"])
@pytest.mark.parametrize("nodes", [8, 64])  # one row tile, two of them
def test_a_call_after_a_timeout_runs_normally(m, cache, nodes):  # noqa: F811
    """The error word keeps the bit of a wait that ran out until the host clears
    it; a call that finds it there computes what it always does."""
    c = TreeCase(32, 8, 128, [1500, 300, 900], [nodes, 5, nodes - 3], nodes, cache)
    _, ref = run_step(m, c)
    lay, t = c.gpu(m)
    bufs = m.TreeBuffers.allocate(lay, c.n, lse=True)
    for limit in (1, 0):
        lay.wait_limit_ns = limit
        bufs.out.fill_(7.0)
        bufs.lse.fill_(7.0)
        m.tree_step(lay, c.n, t.q_new, t.k_new, t.v_new, t.pos, t.depth, t.mask, c.max_len, bufs, num_nodes=t.num)
        torch.cuda.synchronize()
        assert int(bufs.err.item()) == m.MQA_DEVERR_TIMEOUT
    assert torch.equal(bufs.out, ref.out) and torch.equal(bufs.lse, ref.lse)


# ------------------------------------------------------------- NaN attended to

@pytest.mark.parametrize("cache", ["bf16", "e5m2", "u8"])
@pytest.mark.parametrize("hq,hkv,d,n", [(32, 8, 128, 6), (32, 8, 128, 40), (12, 3, 64, 31)])
@pytest.mark.parametrize("where", ["query", "key"])
def test_nan_scores_give_nan(m, cache, hq, hkv, d, n, where):  # noqa: F811
    """A NaN in a row's query, or in a cached key that it attends to, makes that
    row NaN, output and lse, whole or merged of parts; the other rows keep their
    bits."""
    c = TreeCase(hq, hkv, d, [3000, 300, 20, 0], [n, n, n, n], n, cache, seed=n)
    _, ref = run_step(m, c)
    lay, t = c.gpu(m)
    bad = torch.zeros(4, n, hq, dtype=torch.bool, device="cuda")
    if where == "query":
        for b in range(4):
            t.q_new[b, n // 2, b + 1, 10] = float("nan")
            bad[b, n // 2, b + 1] = True
    else:
        for b, at in ((0, 2990), (1, 150), (2, 0)):
            if cache == "u8":
                t.ksz[b, 1, at, 0] = float("nan")
            elif cache == "e5m2":
                t.k.view(torch.uint8)[b, 1, at, 7] = 0x7F
            else:
                t.k[b, 1, at, 7] = float("nan")
            bad[b, :, hq // hkv: 2 * (hq // hkv)] = True
    bufs = m.TreeBuffers.allocate(lay, n, lse=True)
    m.tree_step(lay, n, t.q_new, t.k_new, t.v_new, t.pos, t.depth, t.mask, c.max_len, bufs, num_nodes=t.num)
    torch.cuda.synchronize()
    assert int(bufs.err.item()) == 0
    assert bufs.out[bad].isnan().all() and bufs.lse[bad].isnan().all()
    assert torch.equal(bufs.out[~bad], ref.out[~bad]) and torch.equal(bufs.lse[~bad], ref.lse[~bad])


# ------------------------------------------------------- uint8: probabilities

@pytest.mark.parametrize("hq,hkv,nodes", [(32, 8, 9), (28, 4, 13), (32, 1, 8), (32, 8, 60)])
@pytest.mark.parametrize("page", [0, 16])
def test_u8_probabilities_keep_more_than_a_bf16(m, hq, hkv, nodes, page):  # noqa: F811
    """fp32 outputs over a uint8 cache at head_dim 128: a probability times its V
    scale enters as two bf16 terms, within 2^-15 of its value (2^-7 that the first
    leaves times 2^-8 of the second's rounding)."""
    c = TreeCase(hq, hkv, 128, [600, 37], [nodes, nodes - 1], nodes, "u8", page, seed=nodes)
    t, bufs = run_step(m, c, torch.float32)
    assert int(bufs.err.item()) == 0
    check_attention(c, t, bufs.q_rot, bufs.out, bufs.lse, p_err=2.0 ** -15)
