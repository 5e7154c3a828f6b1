"""GPU: the normalised append at the ends of its ranges, and its keys where they may differ from kv_append_rope's."""

import numpy as np
import pytest
import torch

import oracle
from test_norm_append_gpu import BASE, CACHES, DEV, Cache, _check, _i32, _inputs, _run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m(built_lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import mqa_decode_attention_gb300 as mod

    mod.library()
    return mod


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("eps", [1e-38, 1e-42])
def test_smallest_eps(m, kind, eps):
    """eps down to the smallest numbers, beside rows of zeros and rows whose squares are smaller still: y = x / sqrt(mean
    x^2 + eps) w has a size of its own all the same."""
    B, hq, hkv, d = 6, 4, 4, 128
    c = Cache(m, kind, B, hkv, d, 4, hq)
    x = list(_inputs(kind, B, 1, hq, hkv, d, 21))
    size = torch.tensor([0.0, 1e-25, 1e-21, 1e-19, 1e-16, 1.0]).view(B, 1, 1, 1)
    x[0], x[1] = (x[0].float() * size).to(x[0].dtype), (x[1].float() * size).to(x[1].dtype)
    before = c.snapshot()
    q_rot, err = _run(m, c, 1, x, [1] * B, eps=eps)
    assert err == 0
    _check(c, before, x, [1] * B, q_rot, eps=eps)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_weights_times_largest_values(m, kind):
    """Rows near the end of the range with weights above 1 (x w alone would leave it), and tiny weights."""
    B, hq, hkv, d = 4, 4, 4, 128
    c = Cache(m, kind, B, hkv, d, 4, hq)
    x = list(_inputs(kind, B, 1, hq, hkv, d, 22))
    size = torch.tensor([1e37, 5e37, 2e19, 1e30]).view(B, 1, 1, 1)
    x[0], x[1] = (x[0].float() * size).to(x[0].dtype), (x[1].float() * size).to(x[1].dtype)
    x[4] = (x[4].float() * 64).to(x[4].dtype)
    before = c.snapshot()
    q_rot, err = _run(m, c, 1, x, [1] * B)
    assert err == 0
    _check(c, before, x, [1] * B, q_rot)


@pytest.mark.parametrize("kind", ["bf16", "f32", "u4"])
def test_keys_at_far_positions(m, kind):
    """Stored keys of positions up to the largest and the smallest int32. The angle is rounded to 64 bits on either side, by
    2^31 2^-53 and the frequency's 2^-53 each: 2^-20 of a pair's length covers both."""
    B, hkv, d, ends = 4, 2, 128, [2 ** 31 - 1, -2 ** 31, 10 ** 9 + 7, -1]
    c = Cache(m, kind, B, hkv, d, 8, 4)
    x = list(_inputs(kind, B, 1, 4, hkv, d, 12, "both", [64]))
    x[5] = torch.tensor(ends, dtype=torch.int32).view(1, B, 1)
    _, err = _run(m, c, 1, x, [0, 1, 2, 3], sections=[64])
    assert err == 0
    after = c.snapshot()
    for b in range(B):
        key = oracle.norm_rope(x[1][b, 0].double().numpy(), x[4].double().numpy(), float(np.float32(1e-6)), [ends[b]], [64], BASE)
        off = np.repeat(np.sqrt(key[..., 0::2] ** 2 + key[..., 1::2] ** 2), 2, -1) * 2.0 ** -20
        got = c.row(after, "k", b, b)
        if kind == "f32":
            assert np.all(np.abs(got - key) <= off + np.abs(key) * 2.0 ** -24)
            continue
        low, high = oracle.round_bf16(key - off), oracle.round_bf16(key + off)
        if kind == "bf16":
            assert np.all((low <= got) & (got <= high))
            continue
        # 4 bits: half a step of the row's scale, at most its largest value's distance to its smallest / 15 and a bf16 step
        step = (high.max(-1) - low.min(-1)) / 15 * (1 + 2.0 ** -7)
        assert np.all((low - 0.5 * step[:, None] * (1 + 2.0 ** -7) <= got) & (got <= high + 0.5 * step[:, None] * (1 + 2.0 ** -7)))


@pytest.mark.parametrize("kind", CACHES)
def test_keys_beside_the_append(m, kind):
    """Without weights and axes the keys are those of kv_append_rope: the same bits in a bf16 and a 4-bit cache, a rounding
    of fp32 apart in an fp32 one, and in a one-byte cache, where a bf16 rounding comes first here, one code at most."""
    B, n, hq, hkv, d, pos = 3, 4, 8, 2, 128, [0, 30, 200]
    x = _inputs(kind, B, n, hq, hkv, d, 3, None)
    a, b = (Cache(m, kind, B, hkv, d, 204, hq, 16, seed=1) for _ in range(2))
    _, err = _run(m, a, n, x, pos)
    word, other = _i32([0]), torch.empty(B, n, hq, d, device=DEV)
    m.kv_append_rope_multi(b.layout, n, *(t.to(DEV) for t in x[:3]), _i32(pos), BASE, other, word)
    torch.cuda.synchronize()
    assert err == 0 and int(word) == 0
    sa, sb = a.snapshot(), b.snapshot()
    if kind in ("bf16", "u4"):
        assert torch.equal(sa["k"], sb["k"])
        return
    if kind == "f32":
        # two roundings of numbers 2^-36 of the pair's length apart
        pair = x[1].double().abs()
        for q in range(B):
            for i in range(n):
                length = (pair[q, i, :, 0::2] + pair[q, i, :, 1::2]).repeat_interleave(2, -1).numpy()
                assert np.all(np.abs(a.row(sa, "k", q, pos[q] + i) - b.row(sb, "k", q, pos[q] + i)) <= length * 2.0 ** -23)
        return
    if kind == "e5m2":
        order = lambda t: torch.where(t >= 128, 128 - t.int(), t.int())  # noqa: E731  (codes of one sign are ordered)
        assert (order(sa["k"]) - order(sb["k"])).abs().max() <= 1
        return
    # uint8: scales of rows whose ends moved by a bf16 rounding, 2^-8 of them, and with them a zero point by one and each
    # code by at most two (one by its value, one by its zero point)
    for q in range(B):
        for i in range(n):
            u, v = a.row(sa, "k", q, pos[q] + i), b.row(sb, "k", q, pos[q] + i)
            span = v.max(-1, keepdims=True) - v.min(-1, keepdims=True)
            # bf16's half step of the value, half a code on either side, the ends' part in the scale
            assert np.all(np.abs(u - v) <= np.abs(v).max(-1, keepdims=True) * 2.0 ** -8 * 2 + span / 255 * 2)
