"""GPU: attention over a 4-bit cache whose rows, or queries, are of very different sizes beside each other."""

import math

import numpy as np
import pytest
import torch

import oracle
from u4_cases import U4Case, rounding

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def m(built_lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import mqa_decode_attention_gb300 as mod

    mod.library()
    return mod


def _attend(m, c, splits, out_dtype=torch.float32):
    lay, most = c.layout(m), max(c.lens)
    bufs = m.DecodeBuffers.allocate(lay, most, num_splits=splits, out_dtype=out_dtype, n_new=c.n)
    out, lse = torch.empty(c.B, c.n, c.hq, c.d, dtype=out_dtype, device=DEV), torch.empty(c.B, c.n, c.hq, device=DEV)
    lens = torch.tensor(c.lens, dtype=torch.int32, device=DEV)
    m.gqa_decode_attention_multi(lay, c.n, c.q.to(DEV), lens, most, 1 / math.sqrt(c.d), splits, out, lse, bufs.workspace, err=bufs.err)
    torch.cuda.synchronize()
    assert int(bufs.err) == 0
    return out.double().cpu().numpy(), lse.double().cpu().numpy()


def _lse(s):
    return s.max() + np.log(np.exp(s - s.max()).sum())


def _check(c, out, lse):
    """Against 64 bits, with an error that goes by what a query's weights make of each row, not by the largest row.

    Token t's score is off by at most D_t: q is rounded to 11 bits (an even place also by a 16th of its neighbour's half
    step, a value 2^14 below a row's largest by 2^-25 of that), and 2^-18 (1 + its terms) for fp32. Weights that are off by
    factors within exp(+-D_t) move the output by at most sum p_t expm1(D_t) |v_t - out| / sum p_t exp(-D_t). p s is rounded
    by half a step of 11 bits, 2^-11 of itself, of which the output takes the code, -8 to 7 here, and up to 15: 15 2^-11 sum
    p s; and by 2^-30 of a query's largest p s at the least, for each row. Sums of p m, p s c in fp32: 2^-18 of their
    magnitudes."""
    g, scale = c.hq // c.hkv, 1 / math.sqrt(c.d)
    for b in range(c.B):
        K, V = c.values(b)
        q = c.q[b].double().numpy()
        L = c.lens[b]
        pairs = np.stack([c.vsm[c.slot(b, t)].double().numpy() for t in range(L)], 1)  # [Hkv, L, 2]
        for i in range(c.n):
            end = L - c.n + 1 + i
            begin = max(0, end - c.window) if c.window else 0
            for h in range(c.hq):
                k, v, sm = K[h // g, begin:end], V[h // g, begin:end], np.abs(pairs[h // g, begin:end])
                s = scale * (k @ q[i, h])
                top = s.max()
                p = np.exp(s - top)
                total = p.sum()
                p /= total
                want = p @ v
                mag = np.abs(q[i, h])
                mag = mag + mag.reshape(-1, 2)[:, ::-1].reshape(-1) / 16 + mag.max() * 2.0 ** -14
                terms = scale * (np.abs(k) @ mag)
                D = np.minimum(terms * 2.0 ** -11 + (1 + terms) * 2.0 ** -18, 700.0)
                tol = (p * np.expm1(D)) @ np.abs(v - want) / (p @ np.exp(-D))
                ps = p * sm[:, 0]
                tol = tol + 15 * 2.0 ** -11 * ps.sum() + 15 * 2.0 ** -30 * ps.max() * len(p) + 2.0 ** -18 * (15 * ps.sum() + p @ sm[:, 1])
                got = out[b, i, h]
                assert np.all(np.isfinite(got)), (b, i, h)
                worst = np.max(np.abs(got - want) / (tol + rounding(want, torch.float32)))
                assert worst <= 1, f"sequence {b}, token {i}, head {h}: {worst} of the tolerance"
                at = top + np.log(total)
                # ln sum exp(s) is off by no more than it moves when every score does, up or down, by its D_t (which is not cut
                # off here: the exponentials are taken in the logarithm)
                D = terms * 2.0 ** -11 + (1 + terms) * 2.0 ** -18
                up, down = (_lse(s + x) - at for x in (D, -D))
                assert abs(lse[b, i, h] - at) <= max(up, -down) + 2.0 ** -18 + 2.0 ** -20 * abs(at), (b, i, h)


FORMS = {
    # name: (hq, hkv, d, lens, n_new, page, splits)
    "rows4": (8, 2, 128, [300, 700], 1, 0, 1),
    "rows4_shared_paged": (8, 2, 128, [300, 700], 1, 16, 2),
    "rows4_d64": (4, 1, 64, [500], 1, 0, 1),
    "rows16": (8, 2, 128, [300, 520], 4, 0, 2),
    "rows32": (32, 1, 128, [300, 520], 1, 32, 1),
    "rows32_shared": (32, 1, 64, [1500], 1, 0, 2),
}


def _case(name, seed):
    hq, hkv, d, lens, n, page, splits = FORMS[name]
    c = U4Case(hq, hkv, d, lens, n, page, seed=seed, garbage=False)
    # sum(q) of about +-d: a key row of one value then has the score +-d times that value (times the scale)
    g = torch.Generator().manual_seed(seed)
    sign = torch.where(torch.arange(hq) % 3 == 1, -1.0, 1.0)
    c.q = (0.2 * torch.randn(c.B, n, hq, d, generator=g) + sign[None, None, :, None])
    # ordinary keys of mean 0 and small scores
    c.ksm[..., 0], c.ksm[..., 1] = 0.05, -0.375
    return c, splits


def _outlier(c, b, t, score, size):
    """Token t of sequence b: keys of one value, so that the queries of positive sum have this score (and the others its
    negative), and values `size` times as large."""
    at = c.slot(b, t)
    c.ksm[at] = torch.tensor([0.0, score * math.sqrt(c.d) / c.d]).to(torch.bfloat16)
    c.vsm[at] = (c.vsm[at].float() * size).to(torch.bfloat16)


@pytest.mark.parametrize("size", [2.0 ** 25, 2.0 ** 33, 2.0 ** 40])
@pytest.mark.parametrize("name", list(FORMS))
def test_a_large_row_that_some_queries_do_not_see(m, name, size):
    """One value row far larger than the others, of weight e^-140 for most queries and of weight 1 for the others of its
    kv head: first, in the middle, last, and beside a row that counts."""
    for where in (0, 70, 131, -1):
        c, splits = _case(name, 3)
        for b in range(c.B):
            _outlier(c, b, where if where >= 0 else c.lens[b] - c.n, -140.0, size)
        _check(c, *_attend(m, c, splits))


@pytest.mark.parametrize("name", list(FORMS))
def test_a_large_row_that_a_later_one_outweighs(m, name):
    """A query meets a large row first, with the highest score so far, and then a small one that leaves it nothing."""
    c, splits = _case(name, 4)
    for b in range(c.B):
        _outlier(c, b, 5, 60.0, 2.0 ** 38)
        _outlier(c, b, 200, 160.0, 1.0)
    _check(c, *_attend(m, c, splits))


@pytest.mark.parametrize("name", ["rows4", "rows16", "rows32_shared"])
def test_sizes_all_over(m, name):
    """Rows of sizes spread over 2^+-20, zero rows and constant rows among them."""
    c, splits = _case(name, 5)
    g = torch.Generator().manual_seed(6)
    size = 2.0 ** (40 * torch.rand(c.vsm.shape[:-1], generator=g) - 20)
    size[torch.rand(size.shape, generator=g) < 0.05] = 0.0
    c.vsm = (c.vsm.float() * size[..., None]).to(torch.bfloat16)
    flat = torch.rand(size.shape, generator=g) < 0.05
    c.vsm[..., 0][flat] = 0.0
    c.ksm[..., 0], c.ksm[..., 1] = 1.0, -7.5  # scores of many sizes
    _check(c, *_attend(m, c, splits))


@pytest.mark.parametrize("name", ["rows4", "rows32"])
def test_constant_rows_alone(m, name):
    """Value rows without a scale: zeros first, then constants of many sizes."""
    c, splits = _case(name, 7)
    c.vsm[..., 0] = 0.0
    for b in range(c.B):
        for t in range(c.lens[b]):
            c.vsm[c.slot(b, t)][..., 1] = 0.0 if t < 100 else 2.0 ** ((37 * t) % 80 - 40)
    c.ksm[..., 0], c.ksm[..., 1] = 1.0, -7.5
    _check(c, *_attend(m, c, splits))


@pytest.mark.parametrize("name", ["rows4", "rows16", "rows32"])
def test_queries_of_very_different_sizes(m, name):
    """Heads of one kv head whose queries are 2^36 apart: each keeps its bits."""
    c, splits = _case(name, 8)
    c.q = torch.randn(c.q.shape, generator=torch.Generator().manual_seed(9))
    c.q *= torch.where(torch.arange(c.hq) % 4 == 2, 2.0 ** 36, 1.0)[None, None, :, None]
    c.ksm[..., 0], c.ksm[..., 1] = 0.35, -2.6
    _check(c, *_attend(m, c, splits))
