"""GPU: attention over the 4-bit cache, the append that writes it, and steps, against the fp64 oracle."""

import math

import numpy as np
import pytest
import torch

import oracle
from u4_cases import U4Case, attention_reference, rounding

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def m(built_lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import mqa_decode_attention_gb300 as mod

    mod.library()
    return mod


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _attend(m, c, lay=None, scale=None, splits=0, out_dtype=torch.bfloat16, lens=None, most=None, lse=True, ws=None):
    scale = 1 / math.sqrt(c.d) if scale is None else scale
    lay = c.layout(m) if lay is None else lay
    most = max(c.lens) if most is None else most
    bufs = m.DecodeBuffers.allocate(lay, most, num_splits=splits, out_dtype=out_dtype, n_new=c.n)
    out = torch.full((c.B, c.n, c.hq, c.d), 7.0, dtype=out_dtype, device=DEV)
    ls = torch.full((c.B, c.n, c.hq), 7.0, device=DEV) if lse else None
    if bufs.workspace is not None:
        bufs.workspace.fill_(0xAB)  # need not be cleared
    m.gqa_decode_attention_multi(lay, c.n, c.q.to(DEV), _i32(c.lens if lens is None else lens), most, scale, splits, out, ls,
                                 bufs.workspace, err=bufs.err)
    torch.cuda.synchronize()
    return out, ls, int(bufs.err.item())


def _check(c, out, lse, scale, skip=()):
    for b in range(c.B):
        if b in skip:
            continue
        ref, rl, to, tl = attention_reference(c, b, scale)
        got = out[b].double().cpu().numpy()
        assert np.all(np.isfinite(got)), b
        worst = np.max(np.abs(got - ref) / (to + rounding(ref, out.dtype) * (1 + 1e-3)))
        assert worst <= 1, f"sequence {b}: {worst} of the tolerance"
        if lse is not None:
            d = np.max(np.abs(lse[b].double().cpu().numpy() - rl) / (tl + np.abs(rl) * 2.0 ** -22))
            assert d <= 1, f"sequence {b}: lse {d} of the tolerance"


ATTEND = {
    # name: (hq, hkv, d, lens, n_new, page, window)
    "one_token": (4, 2, 128, [1, 1], 1, 0, 0),
    "tile_borders": (8, 2, 128, [31, 32, 33, 63, 64, 65, 127, 128, 129], 1, 0, 0),
    "d64": (8, 2, 64, [1, 40, 300, 31], 1, 0, 0),
    "mha": (3, 3, 128, [77, 500], 1, 0, 0),
    "group7": (28, 4, 64, [333, 1001, 5], 1, 0, 0),
    "group9": (18, 2, 128, [333, 100], 1, 0, 0),
    "group16": (16, 1, 128, [333, 100, 2000], 1, 0, 0),
    "group17": (17, 1, 64, [200, 64], 1, 0, 0),
    "mqa32": (32, 1, 128, [700, 1], 1, 0, 0),
    "group40": (40, 1, 128, [321], 1, 0, 0),
    "long": (8, 1, 128, [20000], 1, 0, 0),
    "multi2": (8, 2, 128, [2, 50, 333], 2, 0, 0),
    "multi8": (32, 8, 128, [8, 9, 300], 8, 0, 0),
    "multi32": (6, 2, 64, [32, 33, 100], 32, 0, 0),
    "multi5_group3": (3, 1, 128, [5, 64, 200], 5, 0, 0),
    "paged16": (16, 4, 128, [1, 16, 17, 700, 48], 1, 16, 0),
    "paged32_d64": (8, 4, 64, [33, 500], 1, 32, 0),
    "paged64": (8, 8, 128, [65, 64, 1], 1, 64, 0),
    "paged256_multi": (8, 2, 128, [300, 256, 257], 3, 256, 0),
    "window1": (8, 2, 128, [1, 40, 300], 1, 0, 1),
    "window5_multi": (8, 2, 128, [4, 40, 300], 4, 0, 5),
    "window100_paged": (8, 2, 128, [99, 100, 101, 900, 1000], 1, 16, 100),
    "window33_paged_multi": (8, 2, 64, [32, 90, 900], 9, 16, 33),
    "window_over": (8, 2, 128, [300, 20], 1, 0, 1000),
    "many_sequences": (4, 2, 64, [(37 * i) % 150 + 1 for i in range(71)], 1, 16, 0),
    "rows_over_many_blocks": (64, 1, 64, [64, 150], 20, 0, 0),
}


@pytest.mark.parametrize("splits", [0, 1, 4])
@pytest.mark.parametrize("name", list(ATTEND))
def test_attention(m, name, splits):
    hq, hkv, d, lens, n, page, window = ATTEND[name]
    c = U4Case(hq, hkv, d, lens, n, page, window, seed=len(name))
    scale = 1 / math.sqrt(d)
    out, lse, err = _attend(m, c, splits=splits, out_dtype=torch.float32 if splits == 4 else torch.bfloat16)
    assert err == 0
    _check(c, out, lse, scale)


RUNS = {
    # name: (hq, hkv, d, n_new, page, window)
    "rows4": (32, 8, 128, 1, 0, 0),
    "rows8_paged": (64, 8, 128, 1, 16, 0),
    "rows16": (32, 8, 128, 4, 0, 0),
    "rows32_paged_d64": (32, 8, 64, 8, 64, 0),
    "window_d64": (24, 8, 64, 1, 0, 100),
    "rows9_window_paged": (24, 8, 128, 3, 32, 200),
}


@pytest.mark.parametrize("name", list(RUNS))
def test_more_units_than_blocks(m, name):
    """480 units of 1 to 40 tiles: every block takes a run of tiles through several of them."""
    hq, hkv, d, n, page, window = RUNS[name]
    lens = [int(x) for x in np.random.default_rng(50).integers(n, 400, 60)]
    lens[17], lens[18], lens[19], lens[59] = 2500, n, 64, 65
    c = U4Case(hq, hkv, d, lens, n, page, window, seed=51)
    out, lse, err = _attend(m, c, splits=2)
    assert err == 0
    _check(c, out, lse, 1 / math.sqrt(d), skip=set(range(60)) - {0, 1, 16, 17, 18, 19, 20, 37, 58, 59})
    again, lse2, err = _attend(m, c, splits=2)
    assert err == 0 and torch.equal(again, out) and torch.equal(lse2, lse)
    one, lse1, err = _attend(m, c, splits=1)
    assert err == 0
    _check(c, one, lse1, 1 / math.sqrt(d), skip=set(range(60)) - {17, 18, 37})
    # Both round q alike. p s to 11 bits moves either by 2^-11 of the values' range (8 at most here), fp32 sums by 2^-16 of
    # it, and each is rounded to bf16; scores are below 60, their fp32 parts 2^-18 of them.
    assert torch.all((one.float() - out.float()).abs() <= 16 * (2.0 ** -11 + 2.0 ** -16) + 1.01 * 2.0 ** -7 * out.float().abs())
    assert torch.all((lse1 - lse).abs() <= 2 * 61 * 2.0 ** -18)


@pytest.mark.parametrize("scale", [0.0, -0.1, 0.5])
def test_scales(m, scale):
    c = U4Case(8, 2, 128, [50, 3, 200], 2, seed=5)
    for splits in (0, 1):
        out, lse, err = _attend(m, c, scale=scale, splits=splits)
        assert err == 0
        _check(c, out, lse, scale)


def test_every_token_is_found(m):
    """A query that points at one key picks that key's value row: each (token, dimension) comes from its place."""
    L, d = 96, 128
    c = U4Case(L, 1, d, [L], 1, seed=9)
    K, V = c.values(0)
    k = K[0] - K[0].mean(0)
    c.q = torch.from_numpy(k / np.linalg.norm(k, axis=1, keepdims=True) * 40.0).float()[None, None]
    score = (c.q[0, 0].double().numpy() @ K[0].T)
    assert all(np.sort(score[t])[-2] < score[t, t] - 30 for t in range(L))  # the others weigh less than e^-30
    out, _, err = _attend(m, c, scale=1.0, out_dtype=torch.float32)
    assert err == 0
    pair = c.vsm[0, 0].double().numpy()
    # p is a power of e (the reference is only followed when a score passes it by 4), so p s is off by half a step of 11
    # bits, 2^-11, of which the output takes up to 15 s: 2^-11 of a row's range, 1 / 2^7 of a code's step. fp32 sums and
    # the weights of e^-30 add some 2^-20 of the row's values
    step = pair[:, 0] * 15 * 2.0 ** -11 + np.abs(pair).sum(-1) * 16 * 2.0 ** -20
    assert np.all(np.abs(out[0, 0].double().cpu().numpy() - V[0]) <= step[:, None])


def test_wide_scales(m):
    """V rows of very different sizes, and values far from 1: the running exponent follows the largest."""
    for spread, seed in ((1e-30, 1), (1e30, 2), (1e-6, 3)):
        c = U4Case(8, 2, 128, [300, 65], 1, seed=seed)
        c.vsm = (c.vsm.double() * spread).to(torch.bfloat16)
        out, lse, err = _attend(m, c, out_dtype=torch.float32)
        assert err == 0
        _check(c, out, lse, 1 / math.sqrt(128))
    for order in (1, -1):
        c = U4Case(8, 2, 128, [640], 1, seed=4, garbage=False)
        size = torch.logspace(-12 * order, 12 * order, 640, base=2.0)
        c.vsm = (c.vsm.double() * size[None, None, :, None]).to(torch.bfloat16)
        out, lse, err = _attend(m, c, out_dtype=torch.float32)
        assert err == 0
        _check(c, out, lse, 1 / math.sqrt(128))


def test_wide_queries(m):
    """Rows of q of very different sizes beside each other; rows of zeros."""
    c = U4Case(8, 2, 128, [100, 33], 1, seed=6)
    c.q *= torch.tensor([1e-20, 1.0, 0.0, 1e-3, 3.0, 1e-38, 0.5, 0.0])[None, None, :, None]
    out, lse, err = _attend(m, c, out_dtype=torch.float32)
    assert err == 0
    _check(c, out, lse, 1 / math.sqrt(128))


def test_not_finite_stays_in_its_rows(m):
    """A query or a cached row that is not finite gives NaN where it is seen, nowhere else."""
    c = U4Case(8, 2, 128, [100, 70], 2, seed=7)
    c.q[0, 1, 3, 5] = float("inf")
    c.q[1, 0, 6, 0] = float("nan")
    out, _, err = _attend(m, c)
    assert err == 0
    bad = torch.isnan(out).any(-1).cpu()
    want = torch.zeros_like(bad)
    want[0, 1, 3] = want[1, 0, 6] = True
    assert torch.equal(bad, want)
    c = U4Case(8, 2, 128, [100, 70], 1, seed=8)
    c.ksm[1, 1, 33, 0] = float("nan")
    out, _, err = _attend(m, c)
    bad = torch.isnan(out).any(-1).cpu()
    want = torch.zeros_like(bad)
    want[1, 0, 4:] = True
    assert torch.equal(bad, want)


def test_bad_lengths_and_pages(m):
    """Sequences out of range set their bits; the others are right, whatever the split."""
    c = U4Case(8, 2, 128, [100, 60, 33, 200], 1, page=16, seed=11)
    scale = 1 / math.sqrt(128)
    for splits in (0, 1):
        lens = [100, 0, 33, 200]
        out, lse, err = _attend(m, c, splits=splits, lens=lens)
        assert err == m.MQA_DEVERR_SEQ_LEN
        _check(c, out, lse, scale, skip=(1,))
        out, lse, err = _attend(m, c, splits=splits, lens=[-5, 60, 33, 100000])
        assert err == m.MQA_DEVERR_SEQ_LEN
        _check(c, out, lse, scale, skip=(0, 3))
        out, lse, err = _attend(m, c, splits=splits, lens=[0, 0, 0, 0])
        assert err == m.MQA_DEVERR_SEQ_LEN
    c.table[3, 2] = 10 ** 6
    c.table[1, 0] = -1
    for splits in (0, 1):
        out, lse, err = _attend(m, c, splits=splits)
        assert err == m.MQA_DEVERR_PAGE_RANGE
        _check(c, out, lse, scale, skip=(1, 3))


def test_same_call_same_bits(m):
    c = U4Case(32, 4, 128, [5000, 100, 3000 + 7, 1], 1, seed=12, garbage=False)
    first = _attend(m, c)
    for _ in range(3):
        again = _attend(m, c)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def _new_rows(c, seed, kind="randn"):
    g = torch.Generator().manual_seed(seed)
    make = lambda h: torch.randn(c.B, c.n, h, c.d, generator=g).to(torch.bfloat16)  # noqa: E731
    return make(c.hq), make(c.hkv), make(c.hkv)


def _expected_rows(k_new, v_new, pos, base):
    """Codes, scales and minima of the appended K and V rows: [B, n, Hkv, ..]."""
    k = np.empty(k_new.shape)
    for b in range(k.shape[0]):
        for i in range(k.shape[1]):
            k[b, i] = oracle.round_bf16(oracle.rope_rotate(k_new[b, i].double().numpy(), pos[b] + i, base))
    return oracle.quantize_u4(k), oracle.quantize_u4(v_new.double().numpy())


def _check_appended(c, want, pos, only=None):
    """The cache on the device holds the rows of `want`, bit for bit, and elsewhere what it held."""
    for codes, sm, old, old_sm, (wc, ws, wl) in ((c.dev["k"], c.dev["ksm"], c.k, c.ksm, want[0]), (c.dev["v"], c.dev["vsm"], c.v, c.vsm, want[1])):
        exp, exp_sm = old.clone(), old_sm.clone()
        for b in range(c.B):
            if only is not None and b not in only:
                continue
            for i in range(c.n):
                at = c.slot(b, pos[b] + i)
                exp[at] = torch.from_numpy(oracle.pack_u4(wc[b, i]))
                exp_sm[at] = torch.from_numpy(np.stack([ws[b, i], wl[b, i]], -1)).to(torch.bfloat16)
        assert torch.equal(codes.cpu(), exp)
        assert torch.equal(sm.cpu().view(torch.int16), exp_sm.view(torch.int16))


APPEND = {
    "one": (8, 2, 128, [0, 5, 130], 1, 0),
    "one_d64_paged": (8, 2, 64, [0, 15, 16, 200], 1, 16),
    "several": (6, 3, 128, [0, 31, 77], 7, 0),
    "many_heads": (80, 40, 64, [3, 4], 2, 32),
    "prompt": (4, 2, 128, [0, 10], 333, 16),
    "far": (4, 1, 128, [131071, 70000], 1, 64),
}


@pytest.mark.parametrize("name", list(APPEND))
def test_append(m, name):
    hq, hkv, d, pos, n, page = APPEND[name]
    c = U4Case(hq, hkv, d, [p + n for p in pos], n, page, seed=20 + len(name), garbage=False)
    q_new, k_new, v_new = _new_rows(c, 3)
    lay, err = c.layout(m), _i32([0])
    q_rot = torch.empty(c.B, n, hq, d, device=DEV)
    m.kv_append_rope_multi(lay, n, q_new.to(DEV), k_new.to(DEV), v_new.to(DEV), _i32(pos), 10000.0, q_rot, err)
    torch.cuda.synchronize()
    assert int(err) == 0
    _check_appended(c, _expected_rows(k_new, v_new, pos, 10000.0), pos)
    got = q_rot.double().cpu().numpy()
    for b in range(c.B):
        for i in range(n):
            want = oracle.rope_rotate(q_new[b, i].double().numpy(), pos[b] + i, 10000.0)
            x = q_new[b, i].double().abs().numpy()
            pair = np.repeat(x[..., 0::2] + x[..., 1::2], 2, -1)
            assert np.all(np.abs(got[b, i] - want) <= pair * 2.0 ** -22)


def test_append_of_odd_rows(m):
    """Rows with ties, constant rows, zeros, tiny and huge values, one outlier, values that are not finite."""
    d = 128
    rows = [np.zeros(d), -np.zeros(d), np.full(d, 3.25), np.full(d, -1e-3), np.arange(d) % 16, np.arange(d) % 16 / 2 - 3,
            np.arange(d) % 31 / 2, np.where(np.arange(d) == 9, 1000.0, 1e-3 * np.arange(d)), 1e-38 * (np.arange(d) - 60),
            2.0 ** -133 * (np.arange(d) % 7), 1e38 * np.sin(np.arange(d)), np.where(np.arange(d) % 2, 3.3e38, -3.3e38),
            np.where(np.arange(d) == 5, np.inf, 1.0), np.where(np.arange(d) == 5, np.nan, 1.0), np.where(np.arange(d) == 127, -np.inf, 0.0),
            2.0 ** -60 * (np.arange(d) % 16), 1.0 + 2.0 ** -7 * (np.arange(d) % 2), np.where(np.arange(d) == 0, -2.0 ** 100, 2.0 ** -100)]
    rng = np.random.default_rng(5)
    rows += [np.round(rng.standard_normal(d) * 4) / 4 for _ in range(20)] + [2.0 ** rng.uniform(-40, 40, d) for _ in range(10)]
    v_new = torch.tensor(np.array(rows)).to(torch.bfloat16)[:, None, None]  # [B, 1, 1, d]
    c = U4Case(2, 1, d, [1] * len(rows), 1, seed=1, garbage=False)
    lay, err = c.layout(m), _i32([0])
    q = torch.zeros(c.B, 1, 2, d, dtype=torch.bfloat16, device=DEV)
    m.kv_append_rope(lay, q, v_new.to(DEV), v_new.to(DEV), _i32([0] * c.B), 10000.0, torch.empty(c.B, 2, d, device=DEV), err)
    torch.cuda.synchronize()
    want = oracle.quantize_u4(v_new.double().numpy())
    at0 = [t for t in range(c.B) if np.isfinite(np.array(rows[t])).all()]  # (at position 0 the key is the value's row)
    for codes, sm, some in ((c.dev["v"], c.dev["vsm"], range(c.B)), (c.dev["k"], c.dev["ksm"], at0)):
        for t in some:
            assert np.array_equal(codes[t, 0, 0].cpu().numpy(), oracle.pack_u4(want[0][t, 0, 0])), t
            pair = sm[t, 0, 0].double().cpu().numpy()
            assert np.array_equal(pair, [want[1][t, 0, 0], want[2][t, 0, 0]], equal_nan=True), t
    for t in set(range(c.B)) - set(at0):
        assert torch.isnan(c.dev["ksm"][t, 0, 0, 0])


def test_append_out_of_range(m):
    """A position or page out of range sets its bit and leaves the cache as it was; the others are written."""
    for page in (0, 16):
        c = U4Case(4, 2, 128, [40, 40, 40, 40], 1, page, seed=33, garbage=False)
        q_new, k_new, v_new = _new_rows(c, 4)
        cap = 4 * 16 if page else 40
        pos = [39, -1, cap, 7]
        if page:
            c.table[3, 0] = 12345
        lay, err = c.layout(m), _i32([0])
        q_rot = torch.full((c.B, 1, 4, 128), 9.0, device=DEV)
        m.kv_append_rope(lay, q_new.to(DEV), k_new.to(DEV), v_new.to(DEV), _i32(pos), 10000.0, q_rot, err)
        torch.cuda.synchronize()
        assert int(err) == m.MQA_DEVERR_POS_RANGE | (m.MQA_DEVERR_PAGE_RANGE if page else 0)
        want = _expected_rows(k_new, v_new, pos, 10000.0)
        _check_appended(c, want, pos, only=[0] if page else [0, 3])
        assert not torch.any(q_rot == 9.0)


STEP = {
    "gqa": (32, 8, 128, [1, 64, 300, 65], 1, 0, 0),
    "paged_window": (8, 2, 128, [1, 64, 300, 65], 1, 16, 50),
    "multi": (8, 2, 64, [4, 64, 300], 4, 32, 0),
    "mqa": (32, 1, 128, [700, 33], 1, 0, 0),
    "multi32": (16, 4, 128, [32, 100], 32, 0, 0),
}


@pytest.mark.parametrize("splits", [0, 1, 2])
@pytest.mark.parametrize("name", list(STEP))
def test_step(m, name, splits):
    """The step is the append and the attention over what it wrote, bit for bit, in two launches."""
    hq, hkv, d, lens, n, page, window = STEP[name]
    c = U4Case(hq, hkv, d, lens, n, page, window, seed=40 + len(name))
    pos = [x - n for x in lens]
    q_new, k_new, v_new = _new_rows(c, 6)
    lay = c.layout(m)
    bufs = m.DecodeBuffers.allocate(lay, max(lens), num_splits=splits, n_new=n)
    if bufs.workspace is not None:
        bufs.workspace.fill_(0xCD)
    args = (q_new.to(DEV), k_new.to(DEV), v_new.to(DEV), _i32(pos), _i32(lens), max(lens), bufs)
    out = (m.decode_step(lay, *args, num_splits=splits) if n == 1 else m.decode_step_multi(lay, n, *args, num_splits=splits)).clone()
    torch.cuda.synchronize()
    assert int(bufs.err) == 0
    assert m.step_launches(lay, max(lens), splits, n_new=n) == (2, False)
    want = _expected_rows(k_new, v_new, pos, 10000.0)
    _check_appended(c, want, pos)
    # the oracle over the cache as it now stands
    c.k, c.v, c.ksm, c.vsm = (c.dev[x].cpu() for x in ("k", "v", "ksm", "vsm"))
    c.q = bufs.q_rot.cpu().view(c.B, n, hq, d)
    _check(c, out.view(c.B, n, hq, d), bufs.lse.view(c.B, n, hq), 1 / math.sqrt(d))
    again, lse, err = _attend(m, c, lay=lay, splits=splits)
    assert err == 0 and torch.equal(again.view_as(out), out) and torch.equal(lse.view_as(bufs.lse), bufs.lse)


def test_step_leaves_a_workspace_it_does_not_need(m):
    """A step that the library gives one block per unit needs no workspace, and writes none that is passed."""
    c = U4Case(8, 8, 128, [5] * 60, seed=47, garbage=False)
    lay = c.layout(m)
    if m.workspace_size(lay, 5, 0) != 0:
        pytest.skip("more than 960 blocks on this GPU")
    q_new, k_new, v_new = _new_rows(c, 8)
    bufs = m.DecodeBuffers.allocate(lay, 5)
    memory = torch.full((8192,), 0xAB, dtype=torch.uint8, device=DEV)
    bufs.workspace = memory[:256]
    m.decode_step(lay, q_new.to(DEV), k_new.to(DEV), v_new.to(DEV), _i32([4] * 60), _i32(c.lens), 5, bufs)
    torch.cuda.synchronize()
    assert int(bufs.err) == 0 and bool((memory == 0xAB).all())


@pytest.mark.parametrize("splits", [0, 1, 2])
def test_noalloc(m, splits):
    c = U4Case(8, 2, 128, [500, 40], 1, seed=50)
    lay, err = c.layout(m), _i32([0])
    out = torch.empty(2, 8, 128, dtype=torch.bfloat16, device=DEV)
    import ctypes

    fn, vp = m.library().gqa_decode_attention_noalloc, ctypes.c_void_p
    fn.restype, q, lens = ctypes.c_int32, c.q.to(DEV), _i32(c.lens)
    st = fn(ctypes.byref(lay), vp(q.data_ptr()), vp(lens.data_ptr()), ctypes.c_int32(500), ctypes.c_float(1 / math.sqrt(128)),
            ctypes.c_int32(splits), vp(out.data_ptr()), ctypes.c_int32(0), None, ctypes.c_int32(0), vp(err.data_ptr()),
            vp(torch.cuda.current_stream().cuda_stream))
    torch.cuda.synchronize()
    assert st == 0 and int(err) == 0
    _check(c, out.view(2, 1, 8, 128), None, 1 / math.sqrt(128))


@pytest.mark.parametrize("splits", [0, 2])
def test_generation(m, splits):
    """Tokens decoded one after the other into an empty cache, through a captured graph that is replayed: each step's
    result is the attention over the quantised rows so far."""
    B, hq, hkv, d, steps = 2, 8, 2, 128, 40
    c = U4Case(hq, hkv, d, [1] * B, 1, page=16, seed=60, garbage=False)
    c.table = torch.arange(2 * 3, dtype=torch.int32).view(2, 3)
    g = torch.Generator().manual_seed(1)
    c.k, c.ksm = torch.zeros(6, hkv, 16, d // 2, dtype=torch.uint8), torch.zeros(6, hkv, 16, 2, dtype=torch.bfloat16)
    c.v, c.vsm = c.k.clone(), c.ksm.clone()
    lay = c.layout(m)
    bufs = m.DecodeBuffers.allocate(lay, steps, num_splits=splits)
    new = [torch.zeros(B, h, d, dtype=torch.bfloat16, device=DEV) for h in (hq, hkv, hkv)]
    pos, lens = _i32([0] * B), _i32([1] * B)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        m.decode_step(lay, *new, pos, lens, steps, bufs, num_splits=splits)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.decode_step(lay, *new, pos, lens, steps, bufs, num_splits=splits)
    K, V = np.zeros((B, hkv, steps, d)), np.zeros((B, hkv, steps, d))
    for t in range(steps):
        rows = [torch.randn(x.shape, generator=g).to(torch.bfloat16) for x in new]
        for x, y in zip(new, rows):
            x.copy_(y)
        pos.fill_(t)
        lens.fill_(t + 1)
        graph.replay()
        torch.cuda.synchronize()
        assert int(bufs.err) == 0
        k = oracle.round_bf16(oracle.rope_rotate(rows[1].double().numpy(), t, 10000.0))
        K[:, :, t] = oracle.dequantize_u4(*oracle.quantize_u4(k))
        V[:, :, t] = oracle.dequantize_u4(*oracle.quantize_u4(rows[2].double().numpy()))
        c.lens = [t + 1] * B
        c.values = lambda b, upto=None: (K[b, :, : t + 1], V[b, :, : t + 1])
        c.q = bufs.q_rot.cpu().view(B, 1, hq, d)
        _check(c, bufs.out.view(B, 1, hq, d), bufs.lse.view(B, 1, hq), 1 / math.sqrt(d))


def test_two_graphs_share_a_workspace(m):
    """Graphs of calls of different forms over one workspace, replayed one after the other on a stream."""
    cases = [U4Case(16, 2, 128, [3000 + 1, 700], 1, seed=72, garbage=False), U4Case(32, 1, 128, [1300, 90, 2000], 2, 16, seed=73, garbage=False),
             U4Case(8, 8, 64, [int(x) for x in range(1, 600, 10)], 1, seed=74, garbage=False)]
    lays, calls, outs, graphs = [c.layout(m) for c in cases], [], [], []
    ws = torch.empty(max(m.workspace_size(lay, max(c.lens), 2, n_new=c.n) for lay, c in zip(lays, cases)), dtype=torch.uint8, device=DEV)
    err = _i32([0])
    for c, lay in zip(cases, lays):
        out, lse = torch.zeros(c.B, c.n, c.hq, c.d, device=DEV), torch.zeros(c.B, c.n, c.hq, device=DEV)
        q, lens = c.q.to(DEV), _i32(c.lens)
        calls.append(lambda c=c, lay=lay, q=q, lens=lens, out=out, lse=lse: m.gqa_decode_attention_multi(
            lay, c.n, q, lens, max(c.lens), 1 / math.sqrt(c.d), 2, out, lse, ws, err=err))
        outs.append((out, lse))
    for call in calls:
        call()
    torch.cuda.synchronize()
    first = [(o.clone(), l.clone()) for o, l in outs]
    for call in calls:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            call()
    for _ in range(10):
        for o, l in outs:
            o.zero_(), l.zero_()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert int(err) == 0
        for (o, l), (o1, l1) in zip(outs, first):
            assert torch.equal(o, o1) and torch.equal(l, l1)
    for c, (o, l) in list(zip(cases, outs))[:2]:
        _check(c, o, l, 1 / math.sqrt(c.d))


def test_two_streams(m):
    """Calls on two streams at once, a workspace each."""
    cases = [U4Case(16, 2, 128, [3000 + 1, 700], 1, seed=70 + i, garbage=False) for i in range(2)]
    lays = [c.layout(m) for c in cases]
    bufs = [m.DecodeBuffers.allocate(lay, 3001) for lay in lays]
    q, lens = [c.q.to(DEV) for c in cases], [_i32(c.lens) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(20):
        for i, st in enumerate(streams):
            m.gqa_decode_attention(lays[i], q[i], lens[i], 3001, 1 / math.sqrt(128), 0, bufs[i].out, bufs[i].lse, bufs[i].workspace,
                                   err=bufs[i].err, stream=st)
    torch.cuda.synchronize()
    for c, b in zip(cases, bufs):
        assert int(b.err) == 0
        _check(c, b.out.view(2, 1, 16, 128), b.lse.view(2, 1, 16), 1 / math.sqrt(128))


@pytest.mark.parametrize("splits,B,hkv,L", [(2, 8, 2, 40000), (1, 64, 8, 4096), (1, 32, 8, 4096)])
def test_timeout_then_normal_call(m, splits, B, hkv, L):
    """With a limit of 1 ns the waits for tiles run out (runs of many tiles, faster used than loaded): the call comes back,
    says so, and the next one gives what the call before gave."""
    g = torch.Generator(DEV).manual_seed(80)
    codes = [torch.randint(0, 256, (B, hkv, L, 64), generator=g, dtype=torch.uint8, device=DEV) for _ in "kv"]
    pairs = [torch.rand(B, hkv, L, 2, generator=g, device=DEV).to(torch.bfloat16) for _ in "kv"]
    lay = m.layout_contiguous(codes[0], codes[1], 8, 0, pairs[0], pairs[1], cache_dtype=m.MQA_U4)
    q, lens = torch.randn(B, 8, 128, generator=g, device=DEV), _i32([L] * (B - 1) + [L - 77])
    bufs = m.DecodeBuffers.allocate(lay, L, num_splits=splits)

    def call():
        bufs.err.zero_()
        m.gqa_decode_attention(lay, q, lens, L, 0.09, splits, bufs.out, bufs.lse, bufs.workspace, err=bufs.err)
        torch.cuda.synchronize()
        return int(bufs.err), bufs.out.clone()

    err, before = call()
    assert err == 0 and torch.isfinite(before).all()
    lay.wait_limit_ns = 1
    assert call()[0] == m.MQA_DEVERR_TIMEOUT
    lay.wait_limit_ns = 0
    err, after = call()
    assert err == 0 and torch.equal(before, after)


@pytest.mark.parametrize("group", [4, 12, 32])
def test_units_shorter_than_a_block_has_warps(m, group):
    """Thousands of units of one to three tiles, so that the warps of a block are several units apart: the same bits on
    every call, and no wait that runs out."""
    g = torch.Generator(DEV).manual_seed(81)
    B, hkv, L = 400, 8, 190
    codes = [torch.randint(0, 256, (B, hkv, 192, 64), generator=g, dtype=torch.uint8, device=DEV) for _ in "kv"]
    pairs = [torch.rand(B, hkv, 192, 2, generator=g, device=DEV).to(torch.bfloat16) for _ in "kv"]
    lay = m.layout_contiguous(codes[0], codes[1], hkv * group, 0, pairs[0], pairs[1], cache_dtype=m.MQA_U4)
    q, lens = torch.randn(B, hkv * group, 128, generator=g, device=DEV), torch.randint(1, L + 1, (B,), generator=g, dtype=torch.int32, device=DEV)
    bufs, whole = m.DecodeBuffers.allocate(lay, L, num_splits=2), m.DecodeBuffers.allocate(lay, L, num_splits=1)
    m.gqa_decode_attention(lay, q, lens, L, 0.09, 1, whole.out, whole.lse, err=whole.err)
    first = None
    for _ in range(40):
        m.gqa_decode_attention(lay, q, lens, L, 0.09, 2, bufs.out, bufs.lse, bufs.workspace, err=bufs.err)
        torch.cuda.synchronize()
        assert int(bufs.err) == 0 and int(whole.err) == 0
        first = bufs.out.clone() if first is None else first
        assert torch.equal(first, bufs.out)
    # split otherwise the same sums are formed in another order, and the probabilities relative to other maxima: each
    # result is within 2^-10 of the values (2.5 at most here) and a rounding to bf16
    assert torch.all((first.float() - whole.out.float()).abs() <= 2 * (16 * 2.0 ** -10 + 2.0 ** -8 * first.float().abs()))
