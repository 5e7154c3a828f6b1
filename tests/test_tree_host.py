"""CPU: refusals of the tree-speculation calls (found before anything is
launched), the host helpers, and pins of their oracle."""

import ctypes

import numpy as np
import pytest
import torch

import oracle
from mqa_decode_attention_gb300 import _abi
from tree_cases import TreeCase, mask_words, raw

FAKE = 0x10000  # 16-byte-aligned stand-in pointer; never dereferenced (the calls fail validation first)


@pytest.fixture(scope="module")
def lib(built_lib):
    return _abi.load()


def _layout(**kw):
    base = dict(cache_dtype=_abi.MQA_BF16, batch=2, h_q=8, h_kv=2, head_dim=128, paged=0, k_cache=FAKE,
                v_cache=FAKE + 4096, capacity=256, page_size=0, num_pages=0, max_pages_per_seq=0, window=0,
                block_table=None)
    base.update(kw)
    return _abi.KVLayout(**base)


def _append(lib, lay, **kw):
    a = dict(n=4, q=FAKE, k=FAKE, v=FAKE, pos=FAKE, depth=FAKE, num=None, base=10000.0, q_rot=FAKE, err=FAKE)
    a.update(kw)
    return lib.kv_append_rope_tree(ctypes.byref(lay), a["n"], a["q"], a["k"], a["v"], a["pos"], a["depth"], a["num"],
                                   a["base"], a["q_rot"], a["err"], None)


def _attention(lib, lay, **kw):
    a = dict(n=4, q=FAKE, pos=FAKE, depth=FAKE, num=None, mask=FAKE, most=100, scale=0.1, out=FAKE, dt=_abi.MQA_BF16,
             lse=None, ws=FAKE, size=1 << 40, err=FAKE)
    a.update(kw)
    return lib.gqa_tree_attention(ctypes.byref(lay), a["n"], a["q"], a["pos"], a["depth"], a["num"], a["mask"],
                                  a["most"], a["scale"], a["out"], a["dt"], a["lse"], a["ws"], a["size"], a["err"], None)


def _step(lib, lay, **kw):
    a = dict(n=4, q=FAKE, k=FAKE, v=FAKE, pos=FAKE, depth=FAKE, num=None, mask=FAKE, most=100, base=1e4, scale=0.1,
             q_rot=FAKE, out=FAKE, dt=_abi.MQA_BF16, lse=None, ws=FAKE, size=1 << 40, err=FAKE)
    a.update(kw)
    return lib.mqa_tree_step(ctypes.byref(lay), a["n"], a["q"], a["k"], a["v"], a["pos"], a["depth"], a["num"],
                             a["mask"], a["most"], a["base"], a["scale"], a["q_rot"], a["out"], a["dt"], a["lse"],
                             a["ws"], a["size"], a["err"], None)


BAD, NOT, WS = _abi.MQA_ERR_INVALID_ARG, _abi.MQA_ERR_UNSUPPORTED, _abi.MQA_ERR_WORKSPACE


@pytest.mark.parametrize("call", [_append, _attention, _step])
def test_layout_and_size_refusals(lib, call):
    assert call(lib, _layout(cache_dtype=_abi.MQA_F32)) == NOT
    assert call(lib, _layout(head_dim=96)) == NOT
    assert call(lib, _layout(h_q=7)) == BAD
    assert call(lib, _layout(cache_dtype=_abi.MQA_U8)) == BAD  # no scales
    assert call(lib, _layout(), n=0) == BAD
    assert call(lib, _layout(), n=129) == BAD
    assert call(lib, _layout(batch=1 << 24), n=128) == BAD  # more rows than an int holds
    for name in ("q", "pos", "err"):
        assert call(lib, _layout(), **{name: None}) == BAD
    assert call(lib, _layout(), q=FAKE + 8) == BAD
    assert call(lib, _layout(), num=FAKE + 2) == BAD


def test_append_refusals(lib):
    for name in ("k", "v", "depth", "q_rot"):
        assert _append(lib, _layout(), **{name: None}) == BAD
    assert _append(lib, _layout(), base=-1.0) == BAD


@pytest.mark.parametrize("call", [_attention, _step])
def test_attention_refusals(lib, call):
    lay = _layout()
    for name in ("mask", "out"):
        assert call(lib, lay, **{name: None}) == BAD
    assert call(lib, lay, most=0) == BAD
    assert call(lib, lay, most=257) == BAD  # past the capacity
    for scale in (0.0, -0.1, float("inf"), float("nan")):
        assert call(lib, lay, scale=scale) == BAD
    assert call(lib, lay, dt=_abi.MQA_U8) == NOT
    assert call(lib, lay, ws=None) == WS
    assert call(lib, lay, size=1000) == WS
    assert call(lib, lay, ws=FAKE + 128) == BAD
    assert call(lib, lay, out=FAKE + 4) == BAD
    assert call(lib, lay, lse=FAKE + 2) == BAD
    assert call(lib, _layout(window=8), depth=None) == BAD  # a window goes by positions


def test_workspace_size(lib):
    assert lib.mqa_tree_workspace_size(ctypes.byref(_layout()), 16) > 0
    assert lib.mqa_tree_workspace_size(ctypes.byref(_layout()), 0) == 0
    assert lib.mqa_tree_workspace_size(ctypes.byref(_layout(cache_dtype=_abi.MQA_F32)), 16) == 0


def _verify(lib, **kw):
    a = dict(B=2, n=4, V=100, p=FAKE, q=FAKE, dt=_abi.MQA_F32, stride=100, tok=FAKE, par=FAKE, num=None, ua=FAKE, un=FAKE,
             kept=FAKE, path=FAKE, nxt=FAKE, err=FAKE)
    a.update(kw)
    return lib.mqa_verify_tree(a["B"], a["n"], a["V"], a["p"], a["q"], a["dt"], a["stride"], a["tok"], a["par"], a["num"],
                               a["ua"], a["un"], a["kept"], a["path"], a["nxt"], a["err"], None)


def test_verify_refusals(lib):
    for name in ("p", "tok", "par", "ua", "un", "kept", "path", "nxt", "err"):
        assert _verify(lib, **{name: None}) == BAD
        assert _verify(lib, **{name: FAKE + 2}) == BAD
    assert _verify(lib, q=FAKE + 4) == BAD
    for kw in (dict(B=0), dict(n=0), dict(n=129), dict(V=0), dict(stride=99), dict(stride=1 << 33)):
        assert _verify(lib, **kw) == BAD
    assert _verify(lib, dt=_abi.MQA_U8) == NOT


def _keep(lib, lays, **kw):
    a = dict(count=len(lays), n=4, pos=FAKE, path=FAKE, kept=FAKE, err=FAKE)
    a.update(kw)
    arr = (_abi.KVLayout * len(lays))(*lays)
    return lib.kv_keep_path(ctypes.byref(arr[0]), a["count"], a["n"], a["pos"], a["path"], a["kept"], a["err"], None)


def test_keep_refusals(lib):
    two = [_layout(), _layout(k_cache=FAKE + 8192)]
    for kw in (dict(count=0), dict(n=0), dict(n=129), dict(pos=None), dict(path=None), dict(kept=None), dict(err=None),
               dict(path=FAKE + 2)):
        assert _keep(lib, two, **kw) == BAD
    assert lib.kv_keep_path(None, 1, 4, FAKE, FAKE, FAKE, FAKE, None) == BAD
    for other in (dict(capacity=258), dict(batch=3), dict(h_kv=4), dict(head_dim=64), dict(cache_dtype=_abi.MQA_F32),
                  dict(paged=1, page_size=16, num_pages=4, max_pages_per_seq=2, block_table=FAKE), dict(v_cache=None)):
        assert _keep(lib, [_layout(), _layout(**other)]) == BAD


def test_binding_refuses_wrong_tensors(built_lib):
    import mqa_decode_attention_gb300 as m

    lay = m.layout_contiguous(torch.zeros(2, 2, 64, 128, dtype=torch.bfloat16), torch.zeros(2, 2, 64, 128, dtype=torch.bfloat16), 8)
    q = torch.zeros(2, 4, 8, 128, dtype=torch.bfloat16)
    kv = torch.zeros(2, 4, 2, 128, dtype=torch.bfloat16)
    pos, depth = torch.zeros(2, dtype=torch.int32), torch.zeros(2, 4, dtype=torch.int32)
    err = torch.zeros(1, dtype=torch.int32)
    ok = dict(q_new=q, k_new=kv, v_new=kv, pos=pos, depth=depth, q_rot=q.clone())
    for name, wrong in (("q_new", q.float()), ("q_new", q.transpose(1, 2)), ("k_new", kv[:, :3]), ("pos", pos.long()),
                        ("depth", depth.t()), ("q_rot", q.float())):
        with pytest.raises(ValueError, match=name):
            a = dict(ok, **{name: wrong})
            m.kv_append_rope_tree(lay, 4, a["q_new"], a["k_new"], a["v_new"], a["pos"], a["depth"], 1e4, a["q_rot"], err,
                                  stream=0)
    bufs = m.VerifyBuffers.allocate(2, 4, "cpu")
    p = torch.zeros(2, 4, 10)
    i, u, un = torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, 4), torch.zeros(2)
    for bad in (dict(p=p.transpose(1, 2)), dict(q=p.bfloat16()), dict(q=p[:, :3]), dict(tok=i.long()), dict(u=u.double()),
                dict(p=p[:, ::2], q=None), dict(p=p[0])):
        a = dict(dict(p=p, q=p, tok=i, u=u), **bad)
        with pytest.raises(ValueError):
            m.verify_tree(a["p"], a["q"], a["tok"], i, a["u"], un, bufs, stream=0)


def test_tree_mask_helper():
    import mqa_decode_attention_gb300 as m

    c = TreeCase(1, 1, 64, [0, 0, 0], [70, 70, 70], 70, garbage=False, seed=4)
    mask, depth = m.tree_mask(torch.from_numpy(c.parents))
    assert np.array_equal(mask.numpy(), c.words) and np.array_equal(depth.numpy(), c.depth)
    assert np.array_equal(oracle.mask_matrix(mask.numpy(), 70), c.bits)
    assert np.array_equal(mask_words(c.bits), c.words)
    for bad in ([[0]], [[-1, 1]], [[-1, -2]]):
        with pytest.raises(ValueError):
            m.tree_mask(torch.tensor(bad))


# ------------------------------------------------------------- oracle pins
def test_oracle_chain_is_multi_token_decode():
    c = TreeCase(4, 2, 64, [20, 3], [5, 5], 5, garbage=False)
    c.parents[:] = np.arange(-1, 4)
    c.depth[:] = np.arange(5)
    c.bits = np.tril(np.ones((2, 5, 5), bool))
    scale = 64 ** -0.5
    for window in (0, 4):
        want = oracle.decode_step_multi(c.k, c.v, c.q_new, c.k_new, c.v_new, [25, 8], 10000.0, scale, "bf16", window=window)
        k, v, _, _ = oracle.tree_append(raw(c.k), raw(c.v), "bf16", c.k_new, c.v_new, c.pos, c.depth, c.nodes, 10000.0)
        assert np.array_equal(k, want["k_cache"]) and np.array_equal(v, want["v_cache"])
        q = oracle.tree_rotate(c.q_new, c.pos, c.depth, 10000.0)
        got = oracle.tree_attention(q, k, v, c.pos, c.depth, c.nodes, c.bits, scale, window)
        assert np.allclose(got["out"], want["out"], atol=1e-12) and np.allclose(got["lse"], want["lse"], atol=1e-12)


def test_oracle_node_equals_its_chain_alone():
    """A node of a tree sees what decoding its chain alone sees."""
    c = TreeCase(4, 2, 64, [9], [8], 8, garbage=False, seed=3)
    scale = 0.2
    q = oracle.tree_rotate(c.q_new, c.pos, c.depth, 10000.0)
    k, v, _, _ = oracle.tree_append(raw(c.k), raw(c.v), "bf16", c.k_new, c.v_new, c.pos, c.depth, c.nodes, 10000.0)
    whole = oracle.tree_attention(q, k, v, c.pos, c.depth, c.nodes, c.bits, scale)
    for i in range(8):
        chain, a = [], i
        while a >= 0:
            chain, a = [a] + chain, c.parents[0][a]
        m = len(chain)
        alone = oracle.decode_step_multi(c.k, c.v, c.q_new[:, chain], c.k_new[:, chain], c.v_new[:, chain], [9 + m], 10000.0,
                                         scale, "bf16")
        assert np.allclose(alone["out"][0, -1], whole["out"][0, i], atol=1e-12)


def test_oracle_verification_follows_the_target():
    """One drafted token: over all drafts and random numbers (a midpoint grid)
    the emitted token follows the target's distribution; without a draft
    distribution likewise for any fixed draft."""
    p = np.array([[[0.5, 0.2, 0.3], [0.1, 0.6, 0.3]]])
    q = np.array([[[0.2, 0.7, 0.1], [1.0, 0.0, 0.0]]])
    grid = (np.arange(60) + 0.5) / 60
    first = np.zeros(3)
    for x in range(3):
        for u in grid:
            for un in grid:
                kept, path, nxt, _ = oracle.verify_tree(p, q, [[0, x]], [[-1, 0]], [2], [[0, u]], [un])
                first[x if kept[0] == 2 else nxt[0]] += q[0, 0, x] / 3600
    assert np.allclose(first, p[0, 0], atol=3 / 60)
    for x in range(3):
        first = np.zeros(3)
        for u in grid:
            for un in grid:
                kept, path, nxt, _ = oracle.verify_tree(p, None, [[0, x]], [[-1, 0]], [2], [[0, u]], [un])
                first[x if kept[0] == 2 else nxt[0]] += 1 / 3600
        assert np.allclose(first, p[0, 0], atol=3 / 60)


def test_oracle_verification_walk():
    """By hand: node 1 rejected, node 2 (its sibling) accepted, its child 3 accepted, then the token after node 3."""
    p = np.zeros((1, 4, 4))
    p[0, 0] = [0.5, 0.5, 0.0, 0.0]
    p[0, 2] = [0.0, 0.0, 1.0, 0.0]
    p[0, 3] = [0.25, 0.25, 0.25, 0.25]
    q = np.full((1, 4, 4), 0.25)
    kept, path, nxt, _ = oracle.verify_tree(p, q, [[0, 2, 1, 2]], [[-1, 0, 0, 2]], [4], [[0, 0.0, 0.9, 0.9]], [0.6])
    assert kept[0] == 3 and list(path[0]) == [0, 2, 3, -1] and nxt[0] == 2
    kept, path, nxt, _ = oracle.verify_tree(p, q, [[0, 2, 1, 2]], [[-1, 0, 0, 2]], [0], [[0, 0, 0.9, 0.9]], [0.6])
    assert kept[0] == 0 and nxt[0] == -1 and (path == -1).all()


def test_oracle_keep_path():
    x = np.arange(2 * 1 * 8 * 1.0).reshape(2, 1, 8, 1)
    y = oracle.keep_path(x, [1, 0], [[0, 2, 3, -1], [1, 4, 5, 7]], [3, 4])
    assert list(y[0, 0, :, 0]) == [0, 1, 3, 4, 4, 5, 6, 7]
    assert list(y[1, 0, :, 0]) == [9, 12, 13, 15, 12, 13, 14, 15]
