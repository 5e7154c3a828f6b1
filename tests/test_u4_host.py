"""CPU: refusals of the 4-bit cache's calls, of the normalised append and of reading back (found before anything is
launched), the binding's checks, and pins of their oracle."""

import ctypes
from fractions import Fraction

import numpy as np
import pytest
import torch

import mqa_decode_attention_gb300 as m
import oracle
from mqa_decode_attention_gb300 import _abi

FAKE = 0x10000  # 16-byte-aligned stand-in pointer; never dereferenced (the calls fail validation first)
BAD, NOT, WS = _abi.MQA_ERR_INVALID_ARG, _abi.MQA_ERR_UNSUPPORTED, _abi.MQA_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib(built_lib):
    return _abi.load()


def _layout(**kw):
    base = dict(cache_dtype=_abi.MQA_U4, batch=2, h_q=8, h_kv=2, head_dim=128, paged=0, k_cache=FAKE,
                v_cache=FAKE + 4096, capacity=256, page_size=0, num_pages=0, max_pages_per_seq=0, window=0,
                block_table=None, k_scale_zero=FAKE, v_scale_zero=FAKE)
    base.update(kw)
    return _abi.KVLayout(**base)


def _attend(lib, lay, **kw):
    a = dict(n=1, q=FAKE, lens=FAKE, most=100, scale=0.1, splits=0, out=FAKE, dt=_abi.MQA_BF16, lse=None, ws=FAKE, size=1 << 40,
             variant=0, err=FAKE)
    a.update(kw)
    return lib.gqa_decode_attention_multi(ctypes.byref(lay), a["n"], a["q"], a["lens"], a["most"], a["scale"], a["splits"], a["out"],
                                          a["dt"], a["lse"], a["ws"], a["size"], a["variant"], a["err"], None)


def _step(lib, lay, **kw):
    a = dict(n=1, q=FAKE, k=FAKE, v=FAKE, pos=FAKE, lens=FAKE, most=100, base=1e4, scale=0.1, splits=0, rot=FAKE, out=FAKE,
             dt=_abi.MQA_BF16, lse=None, ws=FAKE, size=1 << 40, variant=0, err=FAKE)
    a.update(kw)
    return lib.mqa_decode_step_multi(ctypes.byref(lay), a["n"], a["q"], a["k"], a["v"], a["pos"], a["lens"], a["most"], a["base"],
                                     a["scale"], a["splits"], a["rot"], a["out"], a["dt"], a["lse"], a["ws"], a["size"], a["variant"],
                                     a["err"], None)


def _norm(lib, lay, opts=None, **kw):
    a = dict(n=1, q=FAKE, k=FAKE, v=FAKE, pos=FAKE, base=1e4, rot=FAKE, err=FAKE)
    a.update(kw)
    return lib.kv_append_norm_rope(ctypes.byref(lay), a["n"], a["q"], a["k"], a["v"], a["pos"],
                                   None if opts is None else ctypes.byref(opts), a["base"], a["rot"], a["err"], None)


def _read(lib, lay, **kw):
    a = dict(n=10, start=None, rows=None, k=FAKE, v=FAKE, dt=_abi.MQA_BF16, err=FAKE)
    a.update(kw)
    return lib.kv_read_rows(ctypes.byref(lay), a["n"], a["start"], a["rows"], a["k"], a["v"], a["dt"], a["err"], None)


PAGED = _layout(paged=1, capacity=0, page_size=16, num_pages=32, max_pages_per_seq=256, block_table=FAKE)


@pytest.mark.parametrize("call", [_attend, _step, _norm, _read])
def test_layout_refusals(lib, call):
    assert call(lib, _layout(head_dim=96)) == NOT
    assert call(lib, _layout(h_q=7)) == BAD
    assert call(lib, _layout(k_scale_zero=None)) == BAD
    assert call(lib, _layout(v_scale_zero=FAKE + 8)) == BAD
    assert call(lib, _layout(capacity=254)) == NOT  # pairs are copied in units of 16 bytes
    assert call(lib, _layout(capacity=0)) == BAD
    assert call(lib, _layout(capacity=2 ** 31 - 4)) == NOT
    assert call(lib, _layout(paged=1, capacity=0, page_size=16, num_pages=4, max_pages_per_seq=(1 << 27) - 1, block_table=FAKE)) == NOT
    assert call(lib, _layout(k_cache=None)) == BAD
    assert call(lib, _layout(paged=1, page_size=8, num_pages=4, max_pages_per_seq=9, block_table=FAKE)) == NOT
    assert call(lib, _layout(cache_dtype=6)) == NOT


@pytest.mark.parametrize("call", [_attend, _step])
def test_attention_refusals(lib, call):
    for bad in (dict(n=0), dict(n=33), dict(lens=None), dict(most=0), dict(most=257), dict(n=4, most=3), dict(scale=float("nan")),
                dict(splits=-1), dict(out=None), dict(out=FAKE + 8), dict(lse=FAKE + 2), dict(variant=9), dict(err=None),
                dict(splits=2, ws=FAKE + 64)):
        assert call(lib, _layout(), **bad) == BAD, bad
    assert call(lib, _layout(), dt=_abi.MQA_U8) == NOT
    assert call(lib, _layout(), variant=_abi.MQA_VARIANT_CUDA_CORE) == NOT
    for lay, splits in ((_layout(), 2), (PAGED, 3)):
        assert call(lib, lay, splits=splits, ws=None) == WS
        assert call(lib, lay, splits=splits, size=100) == WS


def test_other_calls_refuse_four_bits(lib):
    lay = _layout()
    p = ctypes.byref(lay)
    assert lib.gqa_prefill_attention(p, 64, FAKE, FAKE, 100, 0.1, FAKE, 0, None, FAKE, None) == NOT
    assert lib.mqa_prefill_step(p, 64, FAKE, FAKE, FAKE, FAKE, FAKE, 100, 1e4, 0.1, FAKE, FAKE, 0, None, FAKE, None) == NOT
    assert lib.gqa_tree_attention(p, 4, FAKE, FAKE, FAKE, None, FAKE, 100, 0.1, FAKE, 0, None, FAKE, 1 << 40, FAKE, None) == NOT
    assert lib.kv_append_rope_tree(p, 4, FAKE, FAKE, FAKE, FAKE, FAKE, None, 1e4, FAKE, FAKE, None) == NOT
    assert lib.mqa_tree_workspace_size(p, 4) == 0
    assert lib.kv_keep_path(p, 1, 4, FAKE, FAKE, FAKE, FAKE, None) == NOT


def test_queries(lib):
    """One split needs no workspace, more than one a size whatever their number; the library's choice is one of the two."""
    for lay in (_layout(), PAGED):
        p = ctypes.byref(lay)
        size = [lib.mqa_workspace_size_multi(p, 1, 100, n, 0) for n in (1, 2, 5)]
        assert size[0] == 0 < size[1] == size[2]
        choice = lib.mqa_choose_splits_multi(p, 1, 100, 0)
        assert choice in (1, 2) and lib.mqa_workspace_size_multi(p, 1, 100, 0, 0) == size[choice - 1]
        assert lib.mqa_choose_splits_multi(p, 1, 16 * 256 + 1, 0) == -1
        fused = ctypes.c_int32(7)
        assert lib.mqa_step_launches(p, 1, 100, 0, 0, ctypes.byref(fused)) == 2 and fused.value == 0
        assert lib.mqa_step_launches(p, 1, 100, 0, _abi.MQA_VARIANT_CUDA_CORE, None) == -1


def test_choice_by_length(lib):
    """Short contexts, or windows, need no workspace; long ones of a paged pool are shared."""
    for kw, n, most, choice in ((dict(), 1, 1024, 1), (dict(), 1, 1025, 2), (dict(head_dim=64), 1, 2048, 1), (dict(head_dim=64), 1, 2049, 2),
                                (dict(), 4, 512, 1), (dict(), 4, 513, 2), (dict(), 8, 256, 1), (dict(), 8, 257, 2),
                                (dict(window=960), 1, 4096, 1), (dict(window=962), 1, 4096, 2)):
        lay = _layout(paged=1, capacity=0, page_size=16, num_pages=32, max_pages_per_seq=256, block_table=FAKE, **kw)
        assert lib.mqa_choose_splits_multi(ctypes.byref(lay), n, most, 0) == choice, (kw, n, most)


def _opts(**kw):
    a = dict(q_weight=FAKE, k_weight=FAKE, eps=1e-6, n_axes=0, section=(ctypes.c_int32 * 4)(), axis_pos=None)
    if "section" in kw:
        kw["section"] = (ctypes.c_int32 * 4)(*kw["section"])
    a.update(kw)
    return _abi.NormRope(*[a[k] for k in ("q_weight", "k_weight", "eps", "n_axes", "section", "axis_pos")])


def test_norm_append_refusals(lib):
    for lay in (_layout(), _layout(cache_dtype=_abi.MQA_BF16), _layout(cache_dtype=_abi.MQA_F32)):
        for bad in (dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(q_weight=FAKE + 4),
                    dict(k_weight=FAKE + 8), dict(n_axes=-1), dict(n_axes=5), dict(n_axes=1, section=(64,)),
                    dict(n_axes=2, section=(32, 31), axis_pos=FAKE), dict(n_axes=2, section=(65, -1), axis_pos=FAKE),
                    dict(n_axes=1, section=(64,), axis_pos=FAKE + 2), dict(n_axes=2, section=(2 ** 31 - 1, 2 ** 31 - 1), axis_pos=FAKE)):
            assert _norm(lib, lay, _opts(**bad)) == BAD, bad
        for bad in (dict(n=0), dict(q=None), dict(k=FAKE + 8), dict(pos=None), dict(rot=None), dict(err=None), dict(base=0.0),
                    dict(base=float("inf")), dict(n=2 ** 31 - 1)):
            assert _norm(lib, lay, None, **bad) == BAD, bad


def test_read_refusals(lib):
    for lay in (_layout(), _layout(cache_dtype=_abi.MQA_U8), _layout(cache_dtype=_abi.MQA_FP8_E5M2)):
        for bad in (dict(n=0), dict(n=257), dict(k=None), dict(v=FAKE + 8), dict(start=FAKE + 1), dict(rows=FAKE + 2), dict(err=None)):
            assert _read(lib, lay, **bad) == BAD, bad
        assert _read(lib, lay, dt=_abi.MQA_U8) == NOT
    big = _layout(batch=1 << 20, h_q=1 << 10, h_kv=1 << 10, capacity=1 << 20)
    assert _read(lib, big, n=1 << 20) == BAD


def test_binding_checks():
    k = torch.zeros(2, 2, 8, 64, dtype=torch.uint8)
    sm = torch.zeros(2, 2, 8, 2, dtype=torch.bfloat16)
    lay = m.layout_contiguous(k, k.clone(), 4, 0, sm, sm.clone(), cache_dtype=m.MQA_U4)
    assert lay.cache_dtype == m.MQA_U4 and lay.head_dim == 128
    assert m.layout_contiguous(k, k, 4, 0, sm, sm).cache_dtype == m.MQA_U8  # uint8 alone means bytes
    for bad in (dict(k_scale_zero=None), dict(v_scale_zero=sm.float()), dict(k_scale_zero=sm[:1]), dict(k_scale_zero=sm[..., :1])):
        with pytest.raises(ValueError):
            m.layout_contiguous(k, k, 4, 0, **{**dict(k_scale_zero=sm, v_scale_zero=sm), **bad}, cache_dtype=m.MQA_U4)
    with pytest.raises(ValueError):
        m.layout_contiguous(k.bfloat16(), k.bfloat16(), 4, 0, sm, sm, cache_dtype=m.MQA_U4)
    with pytest.raises(ValueError):
        m.layout_contiguous(k.bfloat16(), k.bfloat16(), 4, cache_dtype=m.MQA_U8)
    q, kv, pos = torch.zeros(2, 3, 4, 128, dtype=torch.bfloat16), torch.zeros(2, 3, 2, 128, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32)
    rot, err = torch.zeros(2, 3, 4, 128), torch.zeros(1, dtype=torch.int32)
    good = dict(q_new=q, k_new=kv, v_new=kv, pos=pos, rope_base=1e4, q_rot=rot, err=err)
    for bad in (dict(q_new=q.float()), dict(k_new=kv[:, :2]), dict(pos=pos.long()), dict(q_rot=rot[:1]), dict(q_weight=torch.zeros(128)),
                dict(k_weight=torch.zeros(64, dtype=torch.bfloat16)), dict(axis_pos=torch.zeros(2, 2, 3, dtype=torch.int32)),
                dict(sections=[64]), dict(axis_pos=torch.zeros(5, 2, 3, dtype=torch.int32), sections=[16, 16, 16, 8, 8]),
                dict(axis_pos=torch.zeros(3, 2, 3, dtype=torch.int32), sections=[32, 32]), dict(err=None)):
        with pytest.raises((ValueError, m.MqaError)):
            m.kv_append_norm_rope(lay, 3, **{**good, **bad}, stream=0)
    out = torch.zeros(2, 2, 5, 128)
    for k_out, v_out in ((out[:1], out), (out, out[:, :, :4]), (out.half(), out.half()), (out, out.bfloat16()), (out[..., :64], out)):
        with pytest.raises((ValueError, TypeError)):
            m.kv_read_rows(lay, None, None, k_out, v_out, err, stream=0)


# ------------------------------------------------------------ the oracle
def test_quantisation_by_fractions():
    """The oracle's scale and codes against exact rational arithmetic."""
    rng = np.random.default_rng(0)
    for t in range(400):
        x = rng.standard_normal(16) * 2.0 ** rng.integers(-30, 30) + (3 * rng.standard_normal() if t % 3 == 0 else 0)
        x = oracle.round_bf16(np.round(x * 4) / 4 if t % 5 == 0 else x)
        codes, scale, low = oracle.quantize_u4(x)
        X = [Fraction(float(v)) for v in x]
        lo, s = min(X), Fraction(float(scale))
        assert Fraction(float(low)) == lo and 15 * s >= max(X) - lo
        bits = int(oracle.bf16_bits(scale))
        assert bits == 0 or 15 * Fraction(float(oracle.bf16_from_bits(bits - 1))) < max(X) - lo
        for v, k in zip(X, codes):
            y = (v - lo) / s if s else Fraction(0)
            f = y.numerator // y.denominator
            assert k == (f if y - f < Fraction(1, 2) else f + 1 if y - f > Fraction(1, 2) else f + (f & 1))
    assert np.array_equal(oracle.unpack_u4(oracle.pack_u4(np.arange(16))), np.arange(16))


def test_norm_rope_pins():
    """A rotation keeps lengths, position 0 turns nothing, the norm's mean square is 1, axes act on their own pairs."""
    rng = np.random.default_rng(1)
    x, w = rng.standard_normal(64), np.ones(64)
    y = oracle.norm_rope(x, w, 0.0, [5], [32], 1e4)
    assert abs(np.mean(y * y) - 1) < 1e-12
    assert np.allclose(oracle.norm_rope(x, None, 0.0, [7], [32], 1e4), oracle.rope_rotate(x, 7, 1e4), atol=1e-12)
    assert np.allclose(oracle.norm_rope(x, None, 0.0, [0, 9], [20, 12], 1e4)[:40], x[:40])
    assert np.allclose(oracle.norm_rope(x, None, 0.0, [0, 9], [20, 12], 1e4)[40:], oracle.rope_rotate(x, 9, 1e4)[40:])


def test_attention_values_is_the_oracles_attention():
    rng = np.random.default_rng(2)
    q, K, V = rng.standard_normal((1, 4, 8)), rng.standard_normal((2, 9, 8)), rng.standard_normal((2, 9, 8))
    out, lse = oracle.attention_values(q, K, V, 8, 0.3)
    want, wl = oracle.gqa_attention(q[0], K, V, 0.3)
    assert np.allclose(out[0], want) and np.allclose(lse[0], wl)
    out, _ = oracle.attention_values(q, K, V, 8, 0.3, window=1)
    assert np.allclose(out[0], np.repeat(V[:, 8], 2, 0))
